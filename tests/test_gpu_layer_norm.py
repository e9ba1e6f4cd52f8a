"""add_rms_norm against the formula in 64 bits."""
import pytest
import torch

import layer_ref as ref

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
CODES = {"fp8_token": torch.float8_e4m3fn, "int8_token": torch.int8, "fp8_block": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


def _inputs(T, N, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + 1000 * T + N)
    x = torch.randn(T, N, generator=g) * size
    r = torch.randn(T, N, generator=g) * torch.exp(torch.randn(N, generator=g)) * size
    w = 0.8 + 0.3 * torch.randn(N, generator=g)
    return x.to(dtype), r.to(dtype), w.to(dtype)


def _run(h, x, r, w, kind="", out=True, eps=1e-6, in_place=False):
    T, N = x.shape
    xg, rg, wg = x.cuda(), None if r is None else r.cuda(), w.cuda()
    ro = (rg if in_place else torch.full_like(rg, 7.0)) if r is not None else None
    o = torch.full_like(xg, 7.0) if out else None
    c = s = None
    if kind:
        c = torch.zeros(T, N, dtype=torch.int8, device="cuda").view(CODES[kind])
        s = torch.full((T, N // 128) if kind == "fp8_block" else (T,), 7.0, device="cuda")
    got = h.add_rms_norm(xg, wg, residual=rg, residual_out=ro, out=o, codes=c, scales=s,
                         kind=kind or "fp8_token", eps=eps)
    assert got == (ro, o, c, s)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in got]


def _check(got, x, r, w, kind, eps=1e-6):
    s, y, rel = ref.norm(x, r, w, eps)
    ro, out, codes, scales = got
    if ro is not None:
        assert ((ro.double() - s).abs() <= ref.rounding(s, x.dtype) + ref.U32 * s.abs()).all()
    if out is not None:
        assert ((out.double() - y).abs() <= ref.rounding(y, x.dtype) + rel * y.abs()).all()
    if codes is not None:
        ref.check_codes(codes, scales, y, rel, kind)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [1, 3, 600])
@pytest.mark.parametrize("N,kind", [
    (8, ""), (16, "fp8_token"), (504, ""), (520, ""), (1024, "int8_token"), (2064, "fp8_token"),
    (128, "fp8_block"), (640, "fp8_block"), (4096, "fp8_token"), (4096, "fp8_block"),
    (5120, "int8_token"), (7168, "fp8_block"), (8208, ""), (16384, "fp8_token")])
def test_norm(handle, dtype, T, N, kind):
    x, r, w = _inputs(T, N, dtype)
    _check(_run(handle, x, r, w, kind), x, r, w, kind)


@pytest.mark.parametrize("N,kind", [(32768, "fp8_block"), (32768, "int8_token"), (24592, "fp8_token"), (32760, "")])
def test_widest_rows(handle, N, kind):
    x, r, w = _inputs(5, N, BF16)
    _check(_run(handle, x, r, w, kind), x, r, w, kind)


@pytest.mark.parametrize("kind", ["", "fp8_token", "fp8_block", "int8_token"])
def test_without_residual_and_without_the_16_bit_output(handle, kind):
    x, _, w = _inputs(9, 1280, BF16)
    _check(_run(handle, x, None, w, kind), x, None, w, kind)
    if kind:
        _check(_run(handle, x, None, w, kind, out=False), x, None, w, kind)
        x, r, w = _inputs(9, 1280, FP16)
        _check(_run(handle, x, r, w, kind, out=False, in_place=True), x, r, w, kind)


def test_the_sum_alone(handle):
    x, r, w = _inputs(4, 264, BF16)
    xg, rg = x.cuda(), r.cuda()
    handle.add_rms_norm(xg, w.cuda(), residual=rg, residual_out=rg)
    assert torch.equal(rg.cpu(), (x.float() + r.float()).to(BF16))


@pytest.mark.parametrize("target", ["x", "residual"])
def test_outputs_in_place_of_inputs(handle, target):
    for T in (2, 700):
        x, r, w = _inputs(T, 4104, FP16)
        xg, rg, wg = x.cuda(), r.cuda(), w.cuda()
        if target == "x":
            handle.add_rms_norm(xg, wg, residual=rg, residual_out=rg, out=xg)
            got = [rg, xg]
        else:
            ro = torch.empty_like(xg)
            handle.add_rms_norm(xg, wg, residual=rg, residual_out=ro, out=rg)
            got = [ro, rg]
        _check([t.cpu() for t in got] + [None, None], x, r, w, "")


def test_strided_rows_leave_what_lies_between(handle):
    T, N = 37, 520
    x, r, w = _inputs(T, N, BF16)
    wide = [torch.full((T, N + 24), 3.0, dtype=BF16, device="cuda") for _ in range(4)]
    wide[0][:, 8:8 + N], wide[1][:, 16:16 + N] = x.cuda(), r.cuda()
    xg, rg, ro, o = (t[:, a:a + N] for t, a in zip(wide, (8, 16, 0, 24)))
    handle.add_rms_norm(xg, w.cuda(), residual=rg, residual_out=ro, out=o)
    _check([ro.cpu(), o.cpu(), None, None], x, r, w, "")
    assert (wide[2][:, N:] == 3).all() and (wide[3][:, :24] == 3).all()


@pytest.mark.parametrize("kind", ["fp8_token", "int8_token", "fp8_block"])
@pytest.mark.parametrize("size", [2.0 ** -70, 2.0 ** -50, 2.0 ** 66, 2.0 ** 100])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_any_size(handle, kind, size, eps):
    x, r, w = _inputs(3, 1152, BF16, size=size)
    got = _run(handle, x, r, w, kind, eps=eps)
    _check(got, x, r, w, kind, eps)


def test_weights_of_any_size(handle):
    for size in (2.0 ** -110, 2.0 ** 90):
        x, r, w = _inputs(3, 1152, BF16)
        w = (w.float() * size).to(BF16)
        _check(_run(handle, x, r, w, "fp8_token"), x, r, w, "fp8_token")


def test_rows_of_zeros(handle):
    for kind in CODES:
        x = torch.zeros(3, 256, dtype=BF16)
        w = torch.ones(256, dtype=BF16)
        ro, out, codes, scales = _run(handle, x, x.clone(), w, kind)
        assert (out == 0).all() and (codes.float() == 0).all() and (scales == 1).all()


def test_rows_with_infinities_keep_to_themselves(handle):
    for T in (3, 600):
        x, r, w = _inputs(T, 1024, BF16)
        x[1, 5], x[2, 7] = float("inf"), float("nan")
        ro, out, codes, scales = _run(handle, x, r, w, "fp8_token")
        assert out[1, 5].isnan() and (out[1, :5] == 0).all() and out[2].isnan().all()
        keep = [i for i in range(T) if i not in (1, 2)]
        _check([ro[keep], out[keep], codes[keep], scales[keep]], x[keep], r[keep], w, "fp8_token")


def test_codes_feed_the_layer(handle):
    # the layer's result from the codes is the formula's up to their rounding
    T, N, M = 33, 1024, 256
    x, r, w = _inputs(T, N, BF16)
    g = torch.Generator().manual_seed(3)
    b = torch.randn(M, N, generator=g) / 32
    sb = b.abs().amax(1) / 448
    bq = (b / sb[:, None]).to(torch.float8_e4m3fn)
    xg, rg = x.cuda(), r.cuda()
    codes = torch.empty(T, N, dtype=torch.float8_e4m3fn, device="cuda")
    sa, c = torch.empty(T, device="cuda"), torch.empty(T, M, dtype=BF16, device="cuda")
    handle.add_rms_norm(xg, w.cuda(), residual=rg, residual_out=rg, codes=codes, scales=sa)
    handle.run(codes, bq.cuda(), c, quant="fp8_dynamic", sa=sa, sb=sb.cuda())
    have = codes.cpu().float().double() * sa.cpu().double()[:, None]
    weight = bq.float().double() * sb.double()[:, None]
    want, size = have @ weight.t(), have.abs() @ weight.abs().t()
    tol = ref.rounding(want, BF16) + 2 * (N / 32 + 64) * ref.U32 * size
    assert ((c.cpu().double() - want).abs() <= tol).all()


def test_no_rows(handle):
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    handle.add_rms_norm(e, torch.ones(64, dtype=BF16, device="cuda"), out=torch.empty_like(e))


def test_captured_and_replayed(handle):
    T, N = 24, 4096
    x, r, w = _inputs(T, N, BF16)
    xg, rg, wg = x.cuda(), r.cuda(), w.cuda()
    ro, o = torch.empty_like(xg), torch.empty_like(xg)
    c, s = torch.empty(T, N, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        handle.add_rms_norm(xg, wg, residual=rg, residual_out=ro, out=o, codes=c, scales=s, kind="int8_token")
    for seed in range(4):
        x, r, _ = _inputs(T, N, BF16, seed=seed)
        xg.copy_(x)
        rg.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        _check([t.cpu() for t in (ro, o, c, s)], x, r, w, "int8_token")
