"""lora_add against the formula in 64 bits."""
import random

import pytest
import torch

import layer_ref as ref

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


class Case:
    def __init__(self, T, K, N, R, n, dtype=BF16, widths=None, ids=None, seed=0, base=True, factors=True):
        g = torch.Generator().manual_seed(seed + T + 7 * K + 11 * N + 13 * R)
        randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.widths = widths or (N,)
        S = len(self.widths)
        self.x, self.base = randn(T, K).to(dtype), randn(T, N).to(dtype) if base else None
        self.a, self.b = (randn(n, S * R, K) * K ** -0.5).to(dtype), (randn(n, N, R) * 0.2).to(dtype)
        self.factors = torch.rand(n, generator=g) * 2 - 0.5 if factors else None
        if ids is None:
            rng = random.Random(seed)
            ids = [rng.randint(-1, n - 1) for _ in range(T)]
        self.ids = torch.tensor(ids, dtype=torch.int32)

    def on_gpu(self):
        return {k: None if t is None else t.cuda() for k, t in
                (("x", self.x), ("a", self.a), ("b", self.b), ("ids", self.ids), ("base", self.base),
                 ("factors", self.factors))}

    def run(self, h, in_place=False):
        d = self.on_gpu()
        out = d["base"] if in_place else torch.full((self.x.shape[0], self.b.shape[1]), 7.0,
                                                    dtype=self.x.dtype, device="cuda")
        got = h.lora_add(d["x"], d["a"], d["b"], d["ids"], out, base=d["base"], factors=d["factors"],
                         slices=self.widths if len(self.widths) > 1 else None)
        assert got is out
        torch.cuda.synchronize()
        return out.cpu()

    def check(self, got):
        ids = torch.where(self.ids < self.b.shape[0], self.ids, -1)
        want, err = ref.lora(self.x, self.a, self.b, ids, self.base, self.factors, self.widths)
        assert ((got.double() - want).abs() <= ref.rounding(want, self.x.dtype) + err).all()
        none = ids < 0
        assert torch.equal(got[none], self.base[none] if self.base is not None else torch.zeros_like(got[none]))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,K,N,R,n", [
    (1, 8, 1, 8, 1), (1, 4096, 4096, 16, 8), (2, 16, 7, 8, 3), (5, 40, 16, 16, 2), (17, 72, 65, 24, 40),
    (33, 512, 130, 32, 1), (63, 1000, 64, 40, 63), (64, 520, 200, 64, 5), (65, 256, 129, 104, 3),
    (130, 2048, 96, 128, 9), (300, 584, 1001, 16, 5), (700, 64, 72, 8, 100)])
def test_rows_in_any_order(handle, dtype, T, K, N, R, n):
    c = Case(T, K, N, R, n, dtype)
    if (c.ids < 0).all():
        c.ids[0] = n - 1
    c.check(c.run(handle))


@pytest.mark.parametrize("R", [8, 16, 24, 32, 48, 64, 72, 96, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_every_form_of_the_rank(handle, R, dtype):
    for rows in (1, 20, 50):  # rows of one adapter: one, two and four groups of 16
        c = Case(rows, 192, 100, R, 2, dtype, ids=[1] * rows)
        c.check(c.run(handle))


@pytest.mark.parametrize("R", [8, 16, 24, 32])
@pytest.mark.parametrize("N", [328, 331])
def test_many_rows_of_one_adapter_among_many_adapters(handle, R, N):
    # one launch, several groups of 16 rows of one adapter in it
    for ids in ([3] * 64, [3] * 40 + [9, -1] * 12, list(range(10)) * 6 + [0]):
        c = Case(len(ids), 328, N, R, 10, ids=ids)
        c.check(c.run(handle))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("R,N", [(16, 2112), (24, 2101), (32, 2101), (32, 2104), (64, 2101)])
def test_waves_that_take_several_blocks_of_many_rows(handle, dtype, R, N):
    # the last block of columns is partial: some lanes of a wave have none, and go on with the others
    c = Case(4100, 72, N, R, 2, dtype, ids=[1] * 4000 + [0] * 99 + [-1])
    c.check(c.run(handle))


@pytest.mark.parametrize("widths", [(512, 128, 128), (64, 64), (1, 1, 1, 1), (100, 28, 3), (40, 200, 8, 16)])
@pytest.mark.parametrize("R", [8, 16, 64])
def test_slices_have_their_own_adapters(handle, widths, R):
    c = Case(70, 320, sum(widths), R, 4, widths=widths)
    c.check(c.run(handle))
    c.check(c.run(handle, in_place=True))


def test_many_slices_of_high_rank(handle):
    widths = (256, 64, 64, 32)
    c = Case(40, 640, sum(widths), 128, 3, widths=widths)
    c.check(c.run(handle))


@pytest.mark.parametrize("base,factors,in_place", [(False, True, False), (True, False, False), (True, True, True),
                                                   (False, False, False)])
def test_optional_operands(handle, base, factors, in_place):
    c = Case(90, 256, 328, 16, 6, base=base, factors=factors)
    c.check(c.run(handle, in_place))


def test_ids_outside_name_no_adapter(handle):
    c = Case(70, 128, 72, 16, 3, ids=[3, -5, 2 ** 31 - 1, -2 ** 31, 2, 0, 1] * 10)
    c.check(c.run(handle))
    c = Case(70, 128, 72, 16, 3, ids=[-1] * 70)
    assert torch.equal(c.run(handle), c.base)
    c.base = None
    assert (c.run(handle) == 0).all()


def test_no_adapters_and_no_rows(handle):
    x, base = torch.randn(5, 64).to(BF16).cuda(), torch.randn(5, 24).to(BF16).cuda()
    a, b = torch.empty(0, 8, 64, dtype=BF16, device="cuda"), torch.empty(0, 24, 8, dtype=BF16, device="cuda")
    out = torch.empty_like(base)
    handle.lora_add(x, a, b, torch.zeros(5, dtype=torch.int32, device="cuda"), out, base=base)
    assert torch.equal(out, base)
    handle.lora_add(x[:0], a, b, torch.zeros(0, dtype=torch.int32, device="cuda"), out[:0], base=base[:0])


@pytest.mark.parametrize("T", [1, 50, 200])
def test_strided_rows_leave_what_lies_between(handle, T):
    for N, gap in ((72, 8), (72, 3), (33, 6)):
        c = Case(T, 128, N, 16, 4)
        d = c.on_gpu()
        x = torch.full((T, 128 + 16), float("nan"), dtype=BF16, device="cuda")
        x[:, 8:136] = d["x"]
        wide = [torch.full((T, N + gap), 3.0, dtype=BF16, device="cuda") for _ in range(2)]
        wide[0][:, :N] = d["base"]
        handle.lora_add(x[:, 8:136], d["a"], d["b"], d["ids"], wide[1][:, gap:], base=wide[0][:, :N],
                        factors=d["factors"])
        c.check(wide[1][:, gap:].cpu())
        assert (wide[1][:, :gap] == 3).all()


def test_rows_with_nan_keep_to_themselves(handle):
    c = Case(64, 256, 80, 16, 3, ids=[0, 1, 2, 1] * 16)
    clean = c.run(handle)
    c.x[5, 9], c.base[9, 3] = float("nan"), float("inf")
    got = c.run(handle)
    assert got[5].isnan().all() and got[9, 3] == float("inf")
    keep = [i for i in range(64) if i not in (5, 9)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.equal(got[9, 4:], clean[9, 4:])


@pytest.mark.parametrize("dtype,size", [(FP16, 2.0 ** 14), (FP16, 2.0 ** -12), (BF16, 2.0 ** 40), (BF16, 2.0 ** -40)])
def test_intermediate_values_beyond_the_type(handle, dtype, size):
    # x a^T leaves fp16's range (or is small in it); the factor brings the sum back
    c = Case(30, 512, 64, 32, 2, dtype, base=False)
    c.x = (c.x.float() * size).to(dtype)
    c.a = (c.a.float() * (8 if size > 1 else 1 / 8)).to(dtype)
    c.factors = c.factors / size
    c.check(c.run(handle))


def test_more_rows_than_the_workspace_takes_at_once(handle):
    # four slices of rank 128 leave room for 65536 rows of the intermediate values
    c = Case(65536 + 100, 8, 8, 128, 3, widths=(2, 2, 2, 2))
    c.check(c.run(handle))


def test_same_bits_every_time_and_from_every_place(handle):
    # a row's result depends on neither its neighbours nor its place
    c = Case(48, 1024, 256, 16, 6)
    first = c.run(handle)
    assert torch.equal(first, c.run(handle))


def test_captured_and_replayed_with_other_ids(handle):
    c = Case(48, 1024, 384, 16, 6, widths=(256, 64, 64))
    d = c.on_gpu()
    out = torch.empty_like(d["base"])
    call = lambda: handle.lora_add(d["x"], d["a"], d["b"], d["ids"], out, base=d["base"],  # noqa: E731
                                   factors=d["factors"], slices=c.widths)
    call()  # grows the workspace
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(4):
        rng = random.Random(seed)
        c.ids = torch.tensor([rng.randint(-1, 5) for _ in range(48)], dtype=torch.int32)
        d["ids"].copy_(c.ids)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.check(out.cpu())


def test_base_from_the_shared_projection(handle):
    # the sum of run() and the adapters, in place of its output
    c = Case(40, 512, 192, 16, 4)
    d = c.on_gpu()
    g = torch.Generator().manual_seed(5)
    w = (torch.randn(192, 512, generator=g) / 23).to(BF16).cuda()
    y = torch.empty(40, 192, dtype=BF16, device="cuda")
    handle.run(d["x"], w, y)
    c.base = y.cpu()
    handle.lora_add(d["x"], d["a"], d["b"], d["ids"], y, base=y, factors=d["factors"])
    c.check(y.cpu())


def test_on_another_stream(handle):
    c = Case(48, 1024, 256, 16, 6)
    h = lg.Handle()
    s = torch.cuda.Stream()
    d = c.on_gpu()
    out = torch.empty_like(d["base"])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h.lora_add(d["x"], d["a"], d["b"], d["ids"], out, base=d["base"], factors=d["factors"])
    s.synchronize()
    c.check(out.cpu())
    h.close()
