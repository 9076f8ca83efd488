"""Strides that a call never uses: those of the token dimension of one token, of the head dimension of one head."""
import pytest
import torch

from parity_util import need_gpu


def _append(fa, x, d, bs=16):
    T, H = x.shape[:2]
    cache = [torch.zeros(3, H, bs, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scale = [torch.ones(3, H, device="cuda") for _ in range(2)]
    slots = torch.arange(20, 20 + T, device="cuda")
    fa.fa_cache_append(x, x, slots, *cache, *scale)
    return [c.view(torch.uint8) for c in cache] + scale


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,H,strides", [(1, 5, (3, 128)), (9, 1, (128, 1)), (1, 1, (7, 5)), (1, 1, (1, 1))])
def test_append_ignores_strides_of_single_tokens_and_heads(T, H, strides, d):
    fa = need_gpu()
    base = torch.randn(T * H * 128, generator=torch.Generator().manual_seed(d)).bfloat16().cuda()
    x = base.as_strided((T, H, d), (*strides, 1))
    assert x.stride() == (*strides, 1)
    for got, want in zip(_append(fa, x, d), _append(fa, x.contiguous().clone(), d)):
        assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,strides", [(2, 3, (12, 64)), (2, 3, (256, 4)), (2, 1, (4, 64)), (1, 2, (64, 4))])
def test_append_refuses_strides_that_it_would_use(T, H, strides):
    fa = need_gpu()
    x = torch.zeros(1024, dtype=torch.bfloat16, device="cuda").as_strided((T, H, 64), (*strides, 1))
    with pytest.raises(fa.FAError) as err:
        _append(fa, x, 64)
    assert err.value.status == fa.FA_ERR_INVALID_ARG
