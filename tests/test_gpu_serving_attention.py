"""Attention of new tokens over a paged cache on the GPU against 64 bits, at
the lengths, masks and layouts where it can go wrong."""
import math
import random

import pytest
import torch

import serving_ref as ref

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu

BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


class Case:
    """Tensors on the CPU; run() moves them, ref() keeps them here."""

    def __init__(self, ctx, nodes, Hk=2, G=4, D=128, page=16, dtype=BF16, cache=None, mask="tree",
                 seed=0, q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        self.ctx, self.nodes, self.D, self.G, self.Hk = ctx, nodes, D, G, Hk
        B, T = len(ctx), sum(nodes)
        self.dtype, cdt = dtype, cache or dtype
        need = [(c + n + page - 1) // page for c, n in zip(ctx, nodes)]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)  # never-used entries
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.k = torch.randn(pages, Hk, page, D, generator=g).to(cdt)
        self.v = torch.randn(pages, Hk, page, D, generator=g).to(cdt)
        self.q = (q_scale * torch.randn(T, Hk * G, D, generator=g)).to(dtype)
        self.ks = torch.rand(Hk, generator=g) + 0.5 if cdt == E4M3 else None
        self.vs = torch.rand(Hk, generator=g) + 0.5 if cdt == E4M3 else None
        self.context = torch.tensor(ctx, dtype=torch.int32)
        self.offsets = torch.tensor([sum(nodes[:b]) for b in range(B + 1)], dtype=torch.int32)
        self.mask = None
        if mask == "tree":
            self.mask, _ = lg.tree_mask([[rng.randint(max(-1, i - 4), i - 1) if i else -1
                                          for i in range(n)] for n in nodes], device="cpu")
        elif mask == "random":  # any pattern, empty rows among them
            words = (max(nodes) + 63) // 64
            self.mask = torch.randint(-2 ** 63, 2 ** 63 - 1, (T, words), generator=g)
            self.mask[::3] = 0
        self.scale = 1.0 / math.sqrt(D)

    def run(self, h, max_context=None, max_nodes=None, q=None, k=None, v=None, lse=True, table=None):
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        T = self.q.shape[0]
        out = torch.full(self.q.shape, 7.0, dtype=self.dtype, device="cuda")
        l = torch.full((T, self.q.shape[1]), 77.0, device="cuda") if lse else None
        h.tree_attention(dev(self.q) if q is None else q, dev(self.k) if k is None else k,
                         dev(self.v) if v is None else v, out,
                         dev(self.table) if table is None else table, dev(self.context),
                         dev(self.offsets),
                         max_context=max(self.ctx) if max_context is None else max_context,
                         max_nodes=max(self.nodes) if max_nodes is None else max_nodes,
                         mask=dev(self.mask), scale=self.scale, k_scale=dev(self.ks),
                         v_scale=dev(self.vs), lse=l)
        torch.cuda.synchronize()
        return out.cpu(), None if l is None else l.cpu()

    def ref(self):
        return ref.attention(self.q, self.k, self.v, self.table, self.context, self.offsets,
                             self.mask, self.scale, self.ks, self.vs)

    def check(self, h, **kw):
        compare(self.run(h, **kw), self.ref())


def compare(got, want):
    out, lse = got
    wout, tol, wlse, ltol = want
    off = (out.double() - wout).abs()
    ok = (off <= tol) | (out.double().isnan() & wout.isnan())
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()} outputs, worst " \
                     f"{float((off / tol).nan_to_num(1e9).max()):.3g} of the bound"
    if lse is not None:
        off = (lse.double() - wlse).abs()
        ok = (off <= ltol) | (lse.double() == wlse) | (lse.isnan() & wlse.isnan())
        assert ok.all(), f"lse: worst {float(off.nan_to_num(1e9).max()):.3g}"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [(BF16, None), (FP16, None), (BF16, E4M3), (FP16, E4M3)])
@pytest.mark.parametrize("ctx,nodes,Hk,G,page", [
    ([1], [1], 1, 1, 16), ([0], [1], 2, 4, 16), ([127, 128, 129, 31, 32, 0], [1] * 6, 2, 4, 16),
    ([300, 5], [5, 7], 2, 3, 8), ([64, 700, 0], [12, 1, 20], 1, 4, 64), ([200], [40], 2, 8, 32),
    ([1000, 63], [9, 16], 3, 1, 1)])
def test_trees(handle, D, dtype, cache, ctx, nodes, Hk, G, page):
    print(f"[attend] D={D} {dtype} {cache} ctx={ctx} nodes={nodes} {Hk}x{G} page={page}", flush=True)
    Case(ctx, nodes, Hk, G, D, page, dtype, cache, seed=len(ctx) + D).check(handle)


@pytest.mark.parametrize("ctx,nodes,mask", [([500, 30], [70, 130], "tree"), ([90, 0], [65, 3], "random"),
                                            ([40], [64], "random"), ([77, 200], [1, 2], "random"),
                                            ([0, 0], [33, 150], "none"), ([250, 17], [90, 33], "none")])
@pytest.mark.parametrize("G", [1, 5])
def test_masks(handle, ctx, nodes, mask, G):
    print(f"[attend] ctx={ctx} nodes={nodes} {mask} G={G}", flush=True)
    Case(ctx, nodes, 2, G, 64, 16, BF16, mask=mask, seed=3).check(handle)


def test_rows_that_see_nothing(handle):
    c = Case([0, 0, 40], [3, 70, 2], 1, 2, 64, mask="random", seed=5)
    c.mask[:] = 0
    out, lse = c.run(handle)
    assert (out[:73] == 0).all() and (lse[:73] == -math.inf).all()
    compare((out, lse), c.ref())


@pytest.mark.parametrize("G,n", [(1, 1), (4, 12), (8, 20)])
@pytest.mark.parametrize("dtype,cache", [(BF16, None), (FP16, E4M3)])
def test_long_contexts_in_splits(handle, G, n, dtype, cache):
    print(f"[attend] splits G={G} n={n} {dtype} {cache}", flush=True)
    Case([5003, 0, 2222], [n, 1, n], 1, G, 128, 16, dtype, cache, seed=7, q_scale=2.0).check(handle)


@pytest.mark.parametrize("ctx_bound,node_bound", [(0, 1), (100, 3), (10 ** 6, 500)])
@pytest.mark.parametrize("mask", ["tree", "none"])
def test_bounds_shape_the_launch_only(handle, ctx_bound, node_bound, mask):
    c = Case([3000, 10], [70, 41], 1, 2, 64, mask=mask, seed=8)
    if mask == "tree":
        node_bound = min(node_bound, 64 * c.mask.shape[1])
    c.check(handle, max_context=ctx_bound, max_nodes=node_bound)


def bad_value(dtype, kind):
    return {"nan": math.nan, "inf": math.inf, "-inf": -math.inf}[kind]


@pytest.mark.parametrize("kind", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("n,G", [(9, 2), (40, 4)])
@pytest.mark.parametrize("ctx", [20, 128, 600])
def test_masked_places_may_hold_anything(handle, kind, n, G, ctx):
    # NaN and infinities in the keys and values of one drafted node, in unused
    # slots of the last page and in pages of nobody: rows that do not see
    # them are as if they were not there
    c = Case([ctx], [n], 1, G, 64, 64, FP16, seed=11)
    clean = Case([ctx], [n], 1, G, 64, 64, FP16, seed=11)
    bad = n // 2
    pos = ctx + bad
    pg, at = int(c.table[0, pos // 64]), pos % 64
    for t in (c.k, c.v):
        t[pg, 0, at, ::3] = bad_value(FP16, kind)
    used = set(c.table[0][c.table[0] >= 0].tolist())
    for p in range(c.k.shape[0]):
        if p not in used:
            c.k[p] = c.v[p] = math.nan
    last = int(c.table[0, (ctx + n - 1) // 64])
    if (ctx + n) % 64:
        c.k[last, 0, (ctx + n) % 64:] = math.nan
        c.v[last, 0, (ctx + n) % 64:] = math.nan
    out, lse = c.run(handle)
    sees = (c.mask[:, 0] >> bad) & 1 == 1
    assert sees.any() and not sees.all()
    wout, tol, wlse, ltol = clean.ref()
    compare((out[~sees], lse[~sees]), (wout[~sees], tol[~sees], wlse[~sees], ltol[~sees]))
    if kind == "nan":
        assert out[sees][..., ::3].isnan().all()


def test_infinite_scores(handle):
    # a key that gives one row +inf: that row is not a number, others are fine;
    # one that gives -inf weighs nothing
    c = Case([30], [1], 1, 2, 64, dtype=BF16, seed=12)
    clean = Case([30], [1], 1, 2, 64, dtype=BF16, seed=12)
    pg, at = int(c.table[0, 0]), 5
    c.q[0, 0, 0], c.q[0, 1, 0] = 1.0, -1.0
    clean.q[0, 0, 0], clean.q[0, 1, 0] = 1.0, -1.0
    c.k[pg, 0, at, 0] = -math.inf
    out, lse = c.run(handle)
    assert out[0, 1].isnan().all() and lse[0, 1].isnan()
    clean.k[pg, 0, at] = 0
    clean.k[pg, 0, at, 0] = -3e38  # as good as not there for head 0
    wout, tol, wlse, ltol = clean.ref()
    compare((out[:, :1], lse[:, :1]), (wout[:, :1], tol[:, :1], wlse[:, :1], ltol[:, :1]))


def test_strides(handle):
    # queries as a part of a QKV product; caches token-major, and side by side
    c = Case([150, 33], [6, 4], 2, 3, 64, 16, BF16, seed=13)
    T, Hq = c.q.shape[:2]
    wide = torch.zeros(T, (Hq + 4) * 64, dtype=BF16, device="cuda")
    wide[:, 128:128 + Hq * 64] = c.q.reshape(T, -1).cuda()
    q = wide[:, 128:128 + Hq * 64].view(T, Hq, 64)
    k = c.k.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    both = torch.stack([c.v, c.v + 1], 1).cuda()
    table = torch.full((2, c.table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table.cuda()
    c.check(handle, q=q, k=k, v=both[:, 0], table=table[:, :c.table.shape[1]])


def test_extra_rows_are_not_touched(handle):
    c = Case([50, 700], [3, 2], 1, 2, 64, mask="none", seed=14)
    for extra_ctx in (0, 5000):          # without and with splits
        more = torch.zeros(8, 2, 64, dtype=BF16)
        more[:5] = c.q
        out = torch.full_like(more, 7.0).cuda()
        handle.tree_attention(more.cuda(), c.k.cuda(), c.v.cuda(), out, c.table.cuda(),
                              c.context.cuda(), c.offsets.cuda(), max_context=700 + extra_ctx,
                              max_nodes=3)
        torch.cuda.synchronize()
        assert (out[5:] == 7).all()
        compare((out[:5].cpu(), None), c.ref())


def test_lengths_cut_at_the_table(handle):
    # a context longer than the page table has pages for reads what is there
    c = Case([100], [2], 1, 1, 64, 16, mask="none", seed=15)
    c.context[0] = 4000
    out, lse = c.run(handle, max_context=4000)
    room = c.table.shape[1] * 16
    c.table[0, -1] = 0                   # the unused entry reads a page in range
    k = ref.gather_cache(c.k, None, c.table[0], room, 0)
    v = ref.gather_cache(c.v, None, c.table[0], room, 0)
    p = torch.softmax(c.q[:, 0].double() @ k.t() * c.scale, 1)
    assert ((out[:, 0].double() - p @ v).abs() <= 2.0 ** -6 * (1e-2 + p @ v.abs())).all()


@pytest.mark.parametrize("mask", ["none", "tree"])
@pytest.mark.parametrize("n,G,bound", [(2, 1, 100), (2, 1, 5000), (40, 4, 100), (70, 4, 5000)])
def test_a_context_up_to_the_largest_integer(handle, n, G, bound, mask):
    # what the table has no pages for is cut off, however long it is said to be
    c = Case([300], [n], 2, G, 128, 16, mask=mask, seed=20)
    c.table[0, -1] = 0
    room = c.table.shape[1] * 16
    results = []
    for ctx in (room, 2 ** 31 - 1, 2 ** 31 - n):
        c.context[0] = ctx
        results.append(c.run(handle, max_context=bound))
    assert results[0][0].isfinite().all()
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])


def test_empty_calls(handle):
    c = Case([40, 9], [2, 3], 1, 2, 64, mask="none", seed=16)
    e = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    handle.tree_attention(e, c.k.cuda(), c.v.cuda(), torch.empty_like(e), c.table.cuda(),
                          c.context.cuda(), z, max_context=40, max_nodes=0)
    # a sequence without nodes between others
    c = Case([40, 9, 20], [2, 0, 3], 1, 2, 64, mask="none", seed=17)
    c.check(handle)


def test_a_cache_past_32_bit_offsets(handle):
    Hk, page, D = 4, 64, 256
    pages = 2 ** 31 // (Hk * page * D) + 2
    k = torch.zeros(pages, Hk, page, D, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    c = Case([90], [3], Hk, 2, D, page, BF16, seed=18)
    far = [pages - 1, 0]
    table = torch.tensor([far], dtype=torch.int32, device="cuda")
    for i, p in enumerate(far):
        k[p], v[p] = c.k[c.table[0, i]].cuda(), c.v[c.table[0, i]].cuda()
    c.check(handle, k=k, v=v, table=table)


def test_repeats_are_equal(handle):
    c = Case([3000, 700], [20, 9], 2, 4, 128, seed=19)
    a, b = c.run(handle), c.run(handle)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
