"""Attention where scores are as large as finite heads can make them: the rows
are still made of their largest scores, in equal parts where several tie."""
import math

import pytest
import torch

import serving_ref as ref
from test_gpu_serving_attention import BF16, E4M3, FP16, Case

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


# The sizes of queries and keys, as multiples that every type holds exactly, and
# how many values of a head are not zero.  The products with scale and log2 e
# reach from 2^20 to beyond 2^100.
SIZES = [(FP16, None, 2.0 ** 11, 2.0 ** 12, 1), (FP16, None, 2.0 ** 13, 2.0 ** 14, 1),
         (FP16, None, 61440.0, 61440.0, 1), (FP16, None, 61440.0, 57344.0, 64),
         (FP16, E4M3, 61440.0, 448.0, 64), (BF16, None, 2.0 ** 12, 2.0 ** 13, 1),
         (BF16, None, 1.5 * 2.0 ** 16, 1.25 * 2.0 ** 17, 3), (BF16, None, 2.0 ** 40, 2.0 ** 45, 64)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n,ctx", [(4, 1, 300), (4, 1, 5000), (4, 20, 300), (4, 20, 5000), (16, 20, 300)])
@pytest.mark.parametrize("dtype,cache,a,b,wide", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_scores_share_the_row(handle, D, G, n, ctx, dtype, cache, a, b, wide, sign):
    print(f"[attend far] D={D} G={G} n={n} ctx={ctx} {dtype} {cache} {a}x{b} wide={wide} {sign}", flush=True)
    c = Case([ctx], [n], 1, G, D, 16, dtype, cache, mask="none", seed=D + n)
    c.ks = None if c.ks is None else torch.ones_like(c.ks)
    g = torch.Generator().manual_seed(ctx)
    length = ctx + n
    if sign > 0:  # most scores far below; ties at some positions of the context
        key = torch.full((length,), -b / 2)
        best = torch.randperm(ctx, generator=g)[:max(1, ctx // 97)]
        key[best] = b
    else:         # every score at the same place far below zero
        key = torch.full((length,), -b)
    c.q = torch.zeros_like(c.q)
    c.q[..., :wide] = a
    for pos in range(length):
        row = torch.zeros(D)
        row[:wide] = key[pos]
        c.k[int(c.table[0, pos // 16]), 0, pos % 16] = row.to(c.k.dtype)
    out, lse = c.run(handle)
    v = ref.gather_cache(c.v, c.vs, c.table[0], length, 0)
    step = ref.half_step(dtype)
    top = float(key.max()) * a * wide * c.scale
    for i in range(n):
        seen = torch.arange(length) <= ctx + i
        tied = seen & (key == key.max())
        want = v[tied].mean(0)
        # weights of one and their sum are exact; the sums of the products and
        # the division are not, nor is the rounding of the result
        tol = step * want.abs() * (1 + 2.0 ** -7) + (256 + 2 * length ** 0.5) * ref.U32 * v[tied].abs().mean(0) + 1e-30
        # a smaller maximum before the largest leaves at most a rescaled zero
        off = (out[i].double() - want).abs()
        assert (off <= tol).all(), (i, float((off / tol).nan_to_num(1e9).max()))
        wl = top + math.log(int(tied.sum()))
        # scale, log2 e and the products with them: four roundings of the score
        assert ((lse[i].double() - wl).abs() <= 8 * ref.U32 * abs(wl) + 1e-5).all(), (lse[i], wl)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n,ctx", [(4, 1, 900), (4, 1, 5000), (4, 20, 900), (16, 20, 900)])
@pytest.mark.parametrize("dtype,cache", [(FP16, None), (FP16, E4M3), (BF16, None), (BF16, E4M3)])
@pytest.mark.parametrize("value", [0.0, math.inf])
def test_a_far_beginning_leaves_nothing(handle, D, G, n, ctx, dtype, cache, value):
    # The first 600 positions lie far below zero for every second head: their
    # weights are exact zeros.  The heads in between score them as any other.
    print(f"[attend far] beginning D={D} G={G} n={n} ctx={ctx} {dtype} {cache} {value}", flush=True)
    c = Case([ctx], [n], 1, G, D, 16, dtype, cache, mask="none", seed=D + ctx)
    c.ks = None if c.ks is None else torch.ones_like(c.ks)
    length, far = ctx + n, 600
    far_q, far_k = (61440.0, 448.0) if cache is E4M3 else (61440.0, 57344.0)
    if dtype is BF16:
        far_q *= 2.0 ** 20
    zero = torch.zeros(()).to(c.k.dtype)
    c.k[..., 0] = zero                      # only the first positions meet q[0]
    for pos in range(far):
        c.k[int(c.table[0, pos // 16]), 0, pos % 16, 0] = torch.tensor(-far_k).to(c.k.dtype)
    c.q[..., 0] = 0.0
    c.q[:, ::2, 0] = far_q
    if value != 0.0 and cache is None:      # of a position without weight, in one value: the others stay
        c.v[int(c.table[0, 1]), 0, 3, 0] = value
    out, lse = c.run(handle)
    k, v = (ref.gather_cache(x, s, c.table[0], length, 0) for x, s in ((c.k, c.ks), (c.v, c.vs)))
    step = ref.half_step(dtype)
    for h in range(G):
        for i in range(n):
            first = far if h % 2 == 0 else 0
            at = slice(first, ctx + i + 1)
            q = c.q[i, h].double()
            z = (k[at] @ q) * c.scale
            big = float((k[at].abs() @ q.abs()).max() * c.scale)
            p = torch.softmax(z, 0)
            dims = slice(1, D) if value != 0.0 else slice(0, D)
            r, size = (p @ v[at])[dims], (p @ v[at].abs())[dims]
            rel = 2 * (D + 8) * ref.U32 * big + (256 + 2 * length ** 0.5) * ref.U32
            tol = step * r.abs() * (1 + 2.0 ** -7) + (step + rel) * size + 1e-30
            off = (out[i, h, dims].double() - r).abs()
            assert (off <= tol).all(), (h, i, float((off / tol).nan_to_num(1e9).max()))
            wl = float(torch.logsumexp(z, 0))
            assert abs(float(lse[i, h]) - wl) <= rel + 16 * ref.U32 * (1 + abs(wl))
