"""Cross attention forward in the forms that few shapes take: CTAs with two tiles of query rows over ragged entries, alone
and as the two-CTA clusters of a tail that leaves SMs idle.  Each test asserts the form that its shape takes (launches and
workspace), so that a change of the rule cannot leave it without the kernel that it is about."""
import pytest

from parity_util import need_gpu
from test_cross import _case, _check
from test_timeout_cross import _check as _check_timeout

# 64 heads of 700 (600) rows are 192 pairs of tiles: a full wave of 152, and 40 clusters, of entries 25 (the second head's
# third pair) to 31.  The third pair of a head has 188 (88) rows: a second tile of 60 rows (none).
CLUSTERS = dict(B=32, Hq=2, Hk=2, Nk=700)
LENS = [700, 0, 1, 127, 128, 129, 255, 256, 257, 500, 699, 640, 641] + [700] * 12 + [0, 1, 128, 129, 257, 699, 700]


def _routes(fa, call, launches, workspace):
    before = fa.fa_kernel_launches()
    call()
    assert fa.fa_kernel_launches() - before == launches and (workspace > 0) == (launches == 3)


def _tensors(case):
    import torch
    q, k, v, _, lens = case
    return q.cuda(), k.cuda(), v.cuda(), None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [600, 700])
def test_clusters_of_two_tiles(Nq, d):
    fa = need_gpu()
    s = CLUSTERS
    for lens in (None, LENS):
        case = _case(Nq + d, s["B"], s["Hq"], s["Hk"], Nq, s["Nk"], d, lens)
        t = _tensors(case)
        _routes(fa, lambda: fa.fa_cross_fwd(*t), 2, fa.fa_cross_fwd_workspace_size(s["B"], s["Hq"], s["Hk"], Nq, s["Nk"], d))
        _check(fa, case, backward=False)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_clusters_of_grouped_heads(d):
    """Two query heads of 300 rows a key head: the same pairs of tiles, of rows of both."""
    fa = need_gpu()
    case = _case(d, 32, 4, 2, 300, 700, d, LENS)
    t = _tensors(case)
    _routes(fa, lambda: fa.fa_cross_fwd(*t), 2, fa.fa_cross_fwd_workspace_size(32, 4, 2, 300, 700, d))
    _check(fa, case, backward=False)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_pairs_of_two_tiles(d):
    """80 heads of 300 rows over three key blocks: 160 pairs, the second of a head with one tile."""
    fa = need_gpu()
    for lens in (None, [300, 0, 1, 128, 129, 299, 256, 257] * 5):
        case = _case(d + 1, 40, 2, 2, 300, 300, d, lens)
        t = _tensors(case)
        _routes(fa, lambda: fa.fa_cross_fwd(*t), 1, fa.fa_cross_fwd_workspace_size(40, 2, 2, 300, 300, d))
        _check(fa, case, backward=False)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Nq,Nk,launches", [(40, 300, 300, 1), (32, 700, 700, 2), (32, 600, 700, 2)])
def test_waits_run_out(B, Nq, Nk, launches, d):
    """The bounded waits of both forms: the kernels wind down by themselves, and both CTAs of a cluster reach its barriers."""
    fa = need_gpu()
    t = _tensors(_case(d, B, 2, 2, Nq, Nk, d, ([Nk, Nk - 3, 1, 0] * B)[:B]))
    _routes(fa, lambda: fa.fa_cross_fwd(*t), launches, fa.fa_cross_fwd_workspace_size(B, 2, 2, Nq, Nk, d))
    _check_timeout(fa, lambda: fa.fa_cross_fwd(*t))
