"""Rows whose largest logit lies far from zero, as where an additive mask
covers every token: the distribution is that of the differences."""
import math

import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


@pytest.mark.parametrize("T,V", [(2, 40), (3, 5003), (2, 131072), (300, 40009)])
@pytest.mark.parametrize("base", [-1e8, -1e9, -1e10, -1e12, -1e20, -1e30, 1e9, 1e11, 1e25])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_far_from_zero(handle, T, V, base, dtype, temperature):
    print(f"[score far] {dtype} base={base} T={T} V={V} temperature={temperature}", flush=True)
    top = 20
    x = torch.full((T, V), base).to(dtype)
    best = float(x[0, 0])
    step = abs(best) * torch.finfo(dtype).eps * 2   # two steps of the type at most
    # row 0: every logit the same.  Row 1: a third of them, spread over the
    # row, so far below that they weigh nothing.  Row 2: a NaN-free mixture of
    # a few ordinary logits among the masked ones.
    x[1, ::3] = torch.tensor(best - max(1e4, 4 * step)).to(dtype)
    if T > 2 and base < 0:
        x[2, 7::V // 4] = torch.tensor(0.5).to(dtype)
    lp = torch.full((T,), 77.0, device="cuda")
    en = torch.full((T,), 77.0, device="cuda")
    ids = torch.full((T, top), -7, dtype=torch.int32, device="cuda")
    tl = torch.full((T, top), 77.0, device="cuda")
    tok = torch.ones(T, dtype=torch.int32)
    handle.token_logprobs(x.cuda(), tok.cuda(), lp, entropy=en, top_ids=ids, top_logprobs=tl,
                          temperature=temperature)
    torch.cuda.synchronize()
    # differences of logits are exact or a few steps off; a sum of n equal
    # terms is off by V / 64 + 64 steps (a lane adds them one after the other),
    # and where exponents are taken relative to a rounded product, all of them
    # by the same amount: 2^-24 of its size, of which there are a few dozen
    bound = (V / 64 + 64) * U32 + 64 * U32 * 4
    logp = torch.log_softmax(x.double() / temperature, -1)
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(-1)
    want = logp[:, 1]
    off = (lp.cpu().double() - want).abs()
    assert (off <= bound * (1 + want.abs())).all(), (lp.cpu()[:3], want[:3])
    assert ((en.cpu().double() - entropy).abs() <= 4 * bound * (1 + math.log(V))).all(), (en[:3], entropy[:3])
    order = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(ids.cpu().long(), order)
    wt = logp.gather(1, order)
    assert ((tl.cpu().double() - wt).abs() <= bound * (1 + wt.abs())).all()
