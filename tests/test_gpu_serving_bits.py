"""Appending without norm, rotation or 8-bit codes keeps every value's bits."""
import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_value_is_stored_unchanged(dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    T, Hk, D, page = 64, 8, 128, 16
    bits = torch.arange(-2 ** 15, 2 ** 15).to(torch.int16).view(T, Hk, D).cuda()
    k, v = bits.view(dtype), bits.flip(0).contiguous().view(dtype)
    kc = torch.zeros(T // page, Hk, page, D, dtype=dtype, device="cuda")
    vc, q_out, k_out = torch.zeros_like(kc), torch.empty_like(k), torch.empty_like(k)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    h.kv_append(k, v, kc, vc, slots)
    h.qk_norm_rope(k, v, q_out, k_out)
    torch.cuda.synchronize()
    for cache, x, copy in ((kc, k, q_out), (vc, v, k_out)):
        for got in (cache.transpose(1, 2).reshape(T, Hk, D), copy):
            nan = x.isnan()
            assert torch.equal(got.isnan(), nan)
            assert torch.equal(got.view(torch.int16)[~nan], x.view(torch.int16)[~nan])
    h.close()
