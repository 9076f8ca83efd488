"""Attention over a cache whose value scales lie far apart, against the oracle's plain form.

Tolerances: those of test_cache.py, and what f16 drops.  A probability enters the product with the values as f16, times
its value scale, relative to the largest such product T of the row so far: 2^12 of it in the streams, 2^7 in the tiles.
Below 2^-14 a step of f16 is 2^-24, so a term p s code is off by at most half of one, 2^-37 or 2^-32 of T, times its code."""
import math

import numpy as np
import pytest

from oracle import lengths as ol
from parity_util import need_gpu, np64
from test_cache import _cache_case, _check_attention, _run_cache, _wide

ONE = 0x38                                   # the code of 1.0
SCALE = 0.125


def _check(fa, case):
    q, kc, vc, ks, vs, table, lens = case
    o, lse, mag, bound, spread = ol.cache_forward(np64(q), kc, vc, ks, vs, table, lens, SCALE)
    weights = ol.cache_forward(np64(q), kc, np.full_like(vc, ONE), ks, vs, table, lens, SCALE)[0]   # sum p s >= T
    d, rows = q.shape[-1], q.shape[1] // kc.shape[1] * q.shape[2]
    dropped = 2.0 ** (-32 if rows > 32 else -37) * weights * 448 * max(1, int(max(lens)))
    # Both are relative to sums over the keys; _check_attention takes 2^-11 of the first.
    _check_attention(_run_cache(fa, case, SCALE), (o, lse, mag + dropped * 2.0 ** 11, bound, spread), d, 2.0 ** -11)


def _balanced(case, lo, hi, seed):
    """Value scales of 2^lo .. 2^hi, and keys that give each block a weight of about the inverse: every block counts."""
    q, kc, vc, ks, vs, table, lens = case
    a = np.random.default_rng(seed).integers(lo, hi + 1, vs.shape)
    a.flat[:2] = lo, hi
    ks[:], vs[:] = 2.0 ** -6, 2.0 ** a
    q[..., 0] = 64.0
    kc[..., 0] = ol.to_e4m3(np.repeat((-a * math.log(2) / (64 * SCALE * 2.0 ** -6))[..., None], kc.shape[2], -1))
    return case


SHAPES = [(1, 1, 1), (8, 2, 1), (16, 1, 1), (6, 2, 5), (26, 1, 1), (40, 1, 1), (64, 1, 1), (50, 1, 2), (100, 1, 1), (130, 1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk,N", SHAPES)
def test_blocks_of_unlike_scales_that_all_count(Hq, Hk, N, d):
    fa = need_gpu()
    for bs, lens, lo, hi in ((16, [700, 33, 0, 1], -40, 20), (64, [500, 90, 65, 301], -20, 10)):
        case = _cache_case(Hq + N + d + bs, 4, Hq, Hk, N, d, bs, lens, extra_columns=_wide(4, Hk, bs) if Hq * N > 32 * Hk else 1)
        _check(fa, _balanced(case, lo, hi, Hq + d))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk,N", [(2, 1, 3), (8, 2, 4), (5, 1, 3), (2, 2, 20), (20, 1, 3), (9, 1, 8), (50, 1, 2), (1, 1, 128)])
def test_an_unseen_block_of_large_values_changes_nothing(Hq, Hk, N, d):
    """The newest token begins a block whose values are 2^48 times the others': the rows before it do not see it."""
    fa = need_gpu()
    for bs, lens in ((16, [65, 17, 129, 161]), (32, [33, 97, 1, 257])):
        case = _cache_case(Hq + N + d + bs, 4, Hq, Hk, N, d, bs, lens, extra_columns=_wide(4, Hk, bs) if Hq * N > 32 * Hk else 1)
        _, _, _, ks, vs, table, _ = case
        ks[:], vs[:] = 2.0 ** -6, 2.0 ** -8
        for b, n in enumerate(lens):
            vs[table[b, (n - 1) // bs]] = 2.0 ** 40
        _check(fa, case)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [4, 16, 40, 100])
def test_the_ends_of_the_scales_range(Hq, d):
    """Blocks of nothing (2^-100) among others, the largest scale under no weight, and requests of one of the two."""
    fa = need_gpu()
    case = _cache_case(Hq + d, 4, Hq, 1, 1, d, 16, [300, 40, 16, 200], extra_columns=_wide(4, 1, 16) if Hq > 32 else 1)
    q, kc, vc, ks, vs, table, _ = case
    ks[:], vs[:] = 2.0 ** -6, 2.0 ** -8
    q[..., 0], kc[..., 0] = 64.0, 0x7e
    for b, j in ((0, 0), (0, 7), (1, 1), (2, 0), (3, 12)):
        vs[table[b, j]], vc[table[b, j]] = 2.0 ** -100, 0
    for b, j in ((0, 3), (1, 0), (3, 0)):                      # about e^-112 of the others' weights
        vs[table[b, j]], kc[table[b, j], ..., 0] = 2.0 ** 117, 0xfe
    _check(fa, case)
