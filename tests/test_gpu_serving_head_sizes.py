"""Norms of heads of every size that their type holds, with any eps."""
import pytest
import torch

import serving_ref as ref

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


@pytest.mark.parametrize("dtype,low,high", [(torch.bfloat16, -125, 126), (torch.float16, -13, 14)])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-36, 1e-30, 1e-6, 1.0])
@pytest.mark.parametrize("D", [16, 80, 128, 256])
@pytest.mark.parametrize("T", [1, 600])
def test_norms_of_any_size(handle, dtype, low, high, eps, D, T):
    # one head of a token ordinary, the others of sizes from the type's least
    # normal to its largest values
    Hq, Hk = 13, 4
    print(f"[heads size] {dtype} eps={eps} D={D} T={T}", flush=True)
    g = torch.Generator().manual_seed(D)
    size = torch.randint(low, high + 1, (T, Hq + Hk, 1), generator=g)
    size[:, 3] = 0
    size[0, :4, 0] = torch.tensor([low, high, low + 1, 0])
    x = torch.rand(T, Hq + Hk, D, generator=g, dtype=torch.float64) + 0.5
    x = (x * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0) * 2.0 ** size.double()).to(dtype)
    assert x.isfinite().all() and (x != 0).all()
    q, k = x[:, :Hq].contiguous(), x[:, Hq:].contiguous()
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype)
    qo, ko = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
    handle.qk_norm_rope(q.cuda(), k.cuda(), qo, ko, q_weight=w.cuda(), k_weight=w.cuda(), eps=eps)
    torch.cuda.synchronize()
    held = float(torch.tensor(eps, dtype=torch.float32))  # eps as the kernel holds it
    for src, got in ((q, qo), (k, ko)):
        y, sz = ref.heads(src, w, held, None, None, 0, False)
        # half a step of the result, in the subnormal range of the type's least
        tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
        bound = ref.heads_bound(y, sz, D, dtype) + tiny
        off = (got.cpu().double() - y).abs()
        assert (off <= bound).all(), (int((off > bound).sum()), float((off / bound).nan_to_num(1e9).max()))


def test_heads_that_have_no_norm(handle):
    # zeros without eps are 0 / 0; infinities and NaN spoil their own head
    x = torch.randn(1, 5, 64).bfloat16()
    x[0, 0] = 0
    x[0, 1, 7] = float("inf")
    x[0, 2, 9] = float("nan")
    x[0, 3] *= 1e-25
    out, ko = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    w = torch.ones(64, dtype=torch.bfloat16)
    handle.qk_norm_rope(x.cuda(), x.cuda(), out, ko, q_weight=w.cuda(), eps=0.0)
    torch.cuda.synchronize()
    got = out.cpu().float()[0]
    assert got[0].isnan().all() and got[1, 7].isnan() and got[2].isnan().all()
    y, size = ref.heads(x[:, 3:], w, 0.0, None, None, 0, False)
    assert ((got[3:].double() - y[0]).abs() <= ref.heads_bound(y, size, 64, torch.bfloat16)[0]).all()
