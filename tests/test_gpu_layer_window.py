"""window_attention against the formula in 64 bits."""
import random

import pytest
import torch

import layer_ref as ref

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
    """Sequences with contexts `ctx` and `cnt` nodes, in shuffled pages."""

    def __init__(self, ctx, cnt, window, sinks, H=4, K=2, D=128, dtype=BF16, cache=None, page=16, tree=False,
                 seed=0, spare=3):
        g = torch.Generator().manual_seed(seed + sum(ctx) + 31 * sum(cnt) + window)
        rng = random.Random(seed)
        cache = dtype if cache is None else cache
        self.window, self.sinks, self.page = window, sinks, page
        need = [(x + n + page - 1) // page for x, n in zip(ctx, cnt)]
        order = list(range(sum(need) + spare))
        rng.shuffle(order)
        self.table = torch.zeros(len(ctx), max(max(need), 1), dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[sum(need[:b]):sum(need[:b + 1])], dtype=torch.int32)
        shape = (sum(need) + spare, K, page, D)
        self.k_cache = torch.randn(shape, generator=g).to(cache)
        self.v_cache = torch.randn(shape, generator=g).to(cache)
        self.k_scale = self.v_scale = None
        if cache is E4M3:
            self.k_scale, self.v_scale = torch.rand(K, generator=g) + 0.5, torch.rand(K, generator=g) + 0.5
        T = sum(cnt)
        self.q = torch.randn(T, H, D, generator=g).to(dtype)
        self.context = torch.tensor(ctx, dtype=torch.int32)
        self.offsets = torch.tensor([sum(cnt[:b]) for b in range(len(cnt) + 1)], dtype=torch.int32)
        self.mask = self.positions = None
        if tree:
            parents = [[rng.randint(max(0, i - 4), i - 1) if i else -1 for i in range(n)] for n in cnt]
            self.mask, depth = lg.tree_mask(parents, device="cpu")
            self.positions = (torch.repeat_interleave(self.context, torch.tensor(cnt)) + depth).to(torch.int32)
        self.max_context, self.max_nodes = max(ctx), max(cnt)

    NAMES = ("q", "k_cache", "v_cache", "table", "context", "offsets", "mask", "positions", "k_scale", "v_scale")

    def on_gpu(self):
        return {n: None if getattr(self, n) is None else getattr(self, n).cuda() for n in self.NAMES}

    def call(self, h, d, out, lse, **kw):
        return h.window_attention(
            d["q"], d["k_cache"], d["v_cache"], out, d["table"], d["context"], d["offsets"],
            max_context=kw.get("max_context", self.max_context), max_nodes=kw.get("max_nodes", self.max_nodes),
            window=self.window, sinks=self.sinks, mask=d["mask"], positions=d["positions"], scale=kw.get("scale"),
            k_scale=d["k_scale"], v_scale=d["v_scale"], lse=lse)

    def run(self, h, **kw):
        d = self.on_gpu()
        out = torch.full_like(d["q"], 7.0)
        lse = torch.full(d["q"].shape[:2], 7.0, device="cuda")
        assert self.call(h, d, out, lse, **kw) is out
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu()

    def check(self, got, **kw):
        out, tol, lse, ltol = ref.window_attention(
            self.q, self.k_cache, self.v_cache, self.table, self.context, self.offsets, self.window, self.sinks,
            self.mask, self.positions, k_scale=self.k_scale, v_scale=self.v_scale, **kw)
        assert ((got[0].double() - out).abs() <= tol).all()
        none = lse == -float("inf")
        assert torch.equal(got[1] == -float("inf"), none)
        assert ((got[1].double() - lse).abs()[~none] <= ltol[~none]).all()


SHAPES = [  # contexts, nodes, window, sinks
    ([0], [1], 1, 0), ([40], [1], 16, 0), ([700, 3, 0, 129], [1, 1, 1, 1], 100, 4),
    ([2000, 31], [1, 1], 333, 70), ([1500], [1], 5000, 2), ([100], [1], 1, 40),
    ([900, 10, 500], [5, 1, 3], 64, 1), ([1000, 0], [70, 33], 200, 5), ([300], [200], 50, 0),
    ([300], [200], 1, 3), ([64, 0, 5], [0, 300, 17], 130, 129), ([1300], [90], 700, 300)]


@pytest.mark.parametrize("ctx,cnt,window,sinks", SHAPES)
@pytest.mark.parametrize("D,dtype,cache,page", [
    (128, BF16, BF16, 16), (128, FP16, E4M3, 64), (64, FP16, FP16, 8), (64, BF16, E4M3, 1), (256, BF16, BF16, 32),
    (256, FP16, E4M3, 128)])
def test_nodes_after_the_context(handle, ctx, cnt, window, sinks, D, dtype, cache, page):
    c = Case(ctx, cnt, window, sinks, D=D, dtype=dtype, cache=cache, page=page)
    c.check(c.run(handle))


@pytest.mark.parametrize("ctx,cnt,window,sinks", [
    ([700, 3, 0, 129], [3, 9, 5, 1], 100, 4), ([900], [40], 8, 0), ([900, 200], [150, 66], 64, 70),
    ([50], [64], 1, 3), ([513, 30], [20, 33], 40, 0), ([1100], [100], 2000, 5)])
@pytest.mark.parametrize("D,dtype,cache", [(128, BF16, BF16), (128, BF16, E4M3), (64, FP16, FP16), (256, FP16, FP16)])
def test_trees(handle, ctx, cnt, window, sinks, D, dtype, cache):
    c = Case(ctx, cnt, window, sinks, D=D, dtype=dtype, cache=cache, tree=True)
    c.check(c.run(handle))


@pytest.mark.parametrize("H,K", [(1, 1), (8, 1), (5, 5), (12, 2), (24, 2)])
def test_head_groups(handle, H, K):
    for cnt in ([1, 1], [7, 20], [90, 3]):
        c = Case([400, 77], cnt, 90, 3, H=H, K=K)
        c.check(c.run(handle))


@pytest.mark.parametrize("tree", [False, True])
def test_long_contexts_are_split(handle, tree):
    for cnt, window in (([1], 6000), ([3, 20], 4000), ([150, 1], 3000)):
        c = Case([9000, 7001][:len(cnt)], cnt, window, 9, tree=tree, page=64)
        c.check(c.run(handle))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cnt", [1, 20, 130])
def test_what_lies_outside_the_window_does_not_reach_a_row(handle, D, cnt):
    # infinities and NaN before the window, where blocks are shared with visible positions too
    for window, sinks in ((37, 5), (100, 0), (300, 70)):
        c = Case([700], [cnt], window, sinks, D=D, page=16)
        clean = c.run(handle)
        c.check(clean)
        sees = ref.window_visible(700, cnt, None, 0, window, sinks, None)
        bad = torch.nonzero(~sees.any(0))[:, 0]
        bad = bad[bad < 700]
        for cache, value in ((c.k_cache, float("nan")), (c.v_cache, float("inf"))):
            cache[c.table[0].long()[bad // 16], :, bad % 16] = value
        c.v_cache[c.table[0].long()[bad[::2] // 16], :, bad[::2] % 16] = float("nan")
        got = c.run(handle)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


def test_a_value_that_only_some_rows_see(handle):
    # an infinity that leaves the window while the chunk goes on
    c = Case([200], [100], 50, 0)
    at = 190
    c.v_cache[int(c.table[0, at // 16]), :, at % 16, 3] = float("inf")
    out, _ = c.run(handle)
    sees = ref.window_visible(200, 100, None, 0, 50, 0, None)[:, at]
    assert sees.any() and not sees.all()
    assert (out[sees][:, :, 3] == float("inf")).all() and out[~sees].isfinite().all()


@pytest.mark.parametrize("cnt", [1, 40])
def test_dropped_pages_may_hold_anything(handle, cnt):
    page, window, sinks = 16, 100, 4
    c = Case([5000], [cnt], window, sinks, page=page)
    clean = c.run(handle)
    first = 5000 - window + 1
    for entry in (-1, 2 ** 31 - 1, -2 ** 31, 10 ** 6):
        c.table[0, 1:first // page] = entry
        got = c.run(handle)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


def test_a_million_positions_in_few_pages(handle):
    # a rolling cache: the table names the same pages over and over
    page, n, window = 64, 40, 900
    c = Case([n * page - 1], [1], window, 3, page=page)
    pages = c.table[0].clone()
    ctx = 1_000_000
    c.table = pages.repeat(ctx // page // n + 2)[None].contiguous()
    c.table[0, 0] = pages[0]
    c.context = torch.tensor([ctx], dtype=torch.int32)
    c.max_context = ctx
    c.check(c.run(handle))


def test_window_of_one_gives_the_own_value(handle):
    for cnt in (1, 100):
        c = Case([300], [cnt], 1, 0)
        out, lse = c.run(handle)
        pos = 300 + torch.arange(cnt)
        v = c.v_cache[c.table[0].long()[pos // 16], :, pos % 16]
        assert torch.equal(out, v.repeat_interleave(2, 1))


def test_rows_that_see_nothing(handle):
    # a node that names nobody, its window in the context's last position only
    c = Case([50], [3], 1, 0, tree=True)
    c.mask[1] = 0
    out, lse = c.run(handle)
    assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()
    c.check((out, lse))


def test_positions_are_clamped(handle):
    c = Case([500], [20], 60, 2, tree=True)
    c.positions[3], c.positions[7], c.positions[9] = -2 ** 31, 2 ** 31 - 1, 0
    c.check(c.run(handle))


def test_mask_without_positions(handle):
    c = Case([500, 20], [20, 70], 60, 2, tree=True)
    c.positions = None
    c.check(c.run(handle))


def test_bounds_that_do_not_hold(handle):
    for cnt in ([1, 1], [30, 4], [100, 2]):
        c = Case([3000, 200], cnt, 1000, 5)
        c.check(c.run(handle, max_context=10, max_nodes=1))
        c.check(c.run(handle, max_context=1 << 40, max_nodes=1 << 20))


def test_positions_past_the_table_are_cut_off(handle):
    for cnt in (2, 60):
        c = Case([500], [cnt], 100, 3, page=16)
        c.table = c.table[:, :20].contiguous()  # 320 positions
        c.check(c.run(handle), reach=320)


def test_far_scores(handle):
    # scores beyond 2^22: such rows are computed apart
    for cnt in (1, 70):
        c = Case([300], [cnt], 90, 3)
        c.q = (c.q.float() * 2.0 ** 20).to(BF16)
        out, lse = c.run(handle)
        want, _, wl, _ = ref.window_attention(c.q, c.k_cache, c.v_cache, c.table, c.context, c.offsets, 90, 3)
        # one position holds all the weight but where two are nearly as large; its weight
        # (2^x with |x| < 1: the maximum is rounded too) is rounded for the product and
        # not in the sum, half a step, and the result is another one
        near = (out.double() - want).abs() <= 2 * ref.rounding(want, BF16)
        assert near.float().mean() > 0.99
        assert ((lse.double() - wl).abs() <= 2.0 ** -15 * wl.abs()).all()


def test_other_scale_and_strided_queries(handle):
    c = Case([300, 40], [9, 2], 70, 4)
    d = c.on_gpu()
    wide = torch.full((11, 10, 128), float("nan"), dtype=BF16, device="cuda")
    wide[:, 3:7] = d["q"]
    d["q"] = wide[:, 3:7]
    out, lse = torch.empty(11, 4, 128, dtype=BF16, device="cuda"), torch.empty(11, 4, device="cuda")
    c.call(handle, d, out, lse, scale=-0.03)
    c.check((out.cpu(), lse.cpu()), scale=-0.03)


def test_rows_behind_the_last_sequence_stay(handle):
    for cnt in ([2, 1], [40, 30]):
        c = Case([300, 40], cnt, 70, 4)
        T = sum(cnt)
        c.q = torch.cat([c.q, c.q[:1]])
        out, lse = c.run(handle)
        assert (out[T:] == 7).all() and (lse[T:] == 7).all()


def test_the_widest_window_is_tree_attention(handle):
    for cnt, tree in (([1, 1], False), ([60, 7], False), ([20, 11], True)):
        c = Case([700, 90], cnt, 1 << 40, 0, tree=tree)
        out, lse = c.run(handle)
        d = c.on_gpu()
        want, wl = torch.empty_like(d["q"]), torch.empty(d["q"].shape[:2], device="cuda")
        handle.tree_attention(d["q"], d["k_cache"], d["v_cache"], want, d["table"], d["context"], d["offsets"],
                              c.max_context, c.max_nodes, mask=d["mask"], lse=wl)
        # (not the same bits: the two may split a context in different places)
        c.check((out, lse))
        c.check((want.cpu(), wl.cpu()))


@pytest.mark.parametrize("cnt", [1, 50])
def test_captured_and_replayed_while_the_context_grows(handle, cnt):
    c = Case([2000, 1500], [cnt, cnt], 256, 4, page=32)
    d = c.on_gpu()
    out, lse = torch.empty_like(d["q"]), torch.empty(d["q"].shape[:2], device="cuda")
    c.call(handle, d, out, lse)  # grows the workspace
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(handle, d, out, lse)
    for ctx in ([2000, 1500], [3, 700], [1999, 0], [256, 1024]):
        c.context = torch.tensor(ctx, dtype=torch.int32)
        d["context"].copy_(c.context)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.check((out.cpu(), lse.cpu()))
