"""Attention of whole prompts and chunks of them over the cache: many new tokens a request, several row tiles a key head, on
both forms of the call.  Against the oracle, with the tolerances of test_cache.py."""
import pytest

from parity_util import need_gpu
from test_cache import _cache_case, _check_cache, _wide


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hk,N,lens", [(4, 1, 150, [150, 149, 151, 700]), (2, 2, 300, [300, 0, 1, 431]),
                                          (3, 1, 129, [129, 128, 257, 64])])
def test_prompts(Hq, Hk, N, lens, wide, d):
    """Prompts into an empty cache, shorter ones in the same call, and chunks behind earlier tokens."""
    fa = need_gpu()
    bs = 16 if d == 64 else 64
    _check_cache(fa, _cache_case(N + d, len(lens), Hq, Hk, N, d, bs, lens, extra_columns=_wide(len(lens), Hk, bs) if wide else 1))
