"""Attention rows whose weight lies almost whole on one position, over fp16
caches: the other positions together can still be what a row's result is
made of, however small each of their weights is."""
import math

import pytest
import torch

import serving_ref as ref
from test_gpu_serving_attention import BF16, E4M3, FP16, Case, compare

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


def sink_case(D, G, n, ctx, dtype, cache, gap, seed):
    """A first position `gap` (in powers of two) above the others for every
    row, with values of zero; the others hold values around 1000 (200 as
    e4m3 codes), so that the result is far above the type's smallest."""
    c = Case([ctx], [n], 1, G, D, 16, dtype, cache, mask="none", seed=seed)
    c.q *= 0.25
    c.q[..., 0] = 16.0
    c.k[..., 0] = torch.zeros(()).to(c.k.dtype)
    big = 200.0 if cache is E4M3 else 1000.0
    c.v = ((c.v.float() * 0.1 + 1.0) * big).to(c.v.dtype)
    first = int(c.table[0, 0])
    key = torch.zeros(D)
    ks = 1.0 if c.ks is None else float(c.ks[0])
    key[0] = gap * math.log(2) / (16.0 * c.scale * ks)
    c.k[first, 0, 0] = key.to(c.k.dtype)
    c.v[first, 0, 0] = torch.zeros(D).to(c.v.dtype)
    return c


# 4, 80 and 320 rows of a key head: the streaming kernel and both tiles, in one
# and in several splits.
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n,ctx", [(4, 1, 900), (4, 1, 5000), (4, 20, 900), (4, 20, 5000), (16, 20, 900)])
@pytest.mark.parametrize("dtype,cache", [(FP16, None), (FP16, E4M3), (BF16, None)])
@pytest.mark.parametrize("gap", [20, 26])
def test_small_weights_add_up(handle, D, G, n, ctx, dtype, cache, gap):
    print(f"[attend] D={D} G={G} n={n} ctx={ctx} {dtype} {cache} gap={gap}", flush=True)
    c = sink_case(D, G, n, ctx, dtype, cache, gap, seed=D + n)
    out, lse = c.run(handle)
    wout, tol, wlse, ltol = c.ref()
    # the output's own smallest step, which the relative bound leaves out
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    # a weight is held to half a step, its product and the result to another
    compare((out, lse), (wout, tol + tiny, wlse, ltol))
    assert (wout.abs() > 100 * tiny).all()
