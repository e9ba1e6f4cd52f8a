"""Per-head norms, rotation and the paged append on the GPU against their
64-bit form, within bounds made of the output's half step and the 32-bit
arithmetic before it."""
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


def make(T, Hq, Hk, D, dtype, seed, pad=0):
    """Views of one QKV product with `pad` unused values a row."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, (Hq + 2 * Hk) * D + pad, generator=g).to(dtype).cuda()
    q = x[:, :Hq * D].view(T, Hq, D)
    k = x[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    v = x[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].view(T, Hk, D)
    qw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype)
    kw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype)
    pos = torch.randint(0, 4096, (T,), generator=g, dtype=torch.int32)
    return q, k, v, qw, kw, pos


def inside(got, want, bound, what):
    got = got.cpu().double()
    off = (got - want).abs()
    assert got.shape == want.shape and (off <= bound).all(), \
        f"{what}: {int((~(off <= bound)).sum())} of {off.numel()} values, worst " \
        f"{float((off / bound).nan_to_num(1e9).max()):.3g} of the bound"


@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, False), (128, 128, True),
                                               (64, 32, True), (256, 256, False), (16, 16, False),
                                               (48, 16, False), (80, 80, True), (112, 96, False)])
@pytest.mark.parametrize("T,Hq,Hk,dtype,norm", [(1, 32, 8, BF16, True), (37, 3, 1, FP16, True),
                                                (130, 4, 4, BF16, False), (5, 1, 0, FP16, True)])
def test_norm_and_rotation(handle, T, Hq, Hk, D, rot, interleaved, dtype, norm):
    print(f"[heads] T={T} {Hq}/{Hk}x{D} rot={rot} {interleaved} {dtype} {norm}", flush=True)
    q, k, _, qw, kw, pos = make(T, Hq, Hk, D, dtype, seed=T + D, pad=8)
    table = lg.rope_table(4096, rot)
    qo = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    ko = torch.full_like(k, 7.0, memory_format=torch.contiguous_format)
    handle.qk_norm_rope(q, k, qo, ko, cos_sin=table, positions=pos.cuda(),
                        q_weight=qw.cuda() if norm else None, k_weight=kw.cuda() if norm else None,
                        eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    for x, w, got, name in ((q, qw, qo, "q"), (k, kw, ko, "k")):
        y, size = ref.heads(x.cpu(), w if norm else None, 1e-5, table.cpu(), pos, rot, interleaved)
        inside(got, y, ref.heads_bound(y, size, D, dtype), name)


def test_norm_alone_and_copy(handle):
    q, k, _, qw, _, _ = make(9, 4, 2, 128, BF16, seed=3)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    handle.qk_norm_rope(q, k, qo, ko, q_weight=qw.cuda())
    torch.cuda.synchronize()
    y, size = ref.heads(q.cpu(), qw, 1e-6, None, None, 0, False)
    inside(qo, y, ref.heads_bound(y, size, 128, BF16), "q")
    assert torch.equal(ko, k)  # no norm, no rotation: the bits


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(handle, interleaved):
    q, k, _, qw, kw, pos = make(33, 8, 2, 64, FP16, seed=4)
    table = lg.rope_table(4096, 64)
    want = []
    for x, w in ((q, qw), (k, kw)):
        y, size = ref.heads(x.cpu(), w, 1e-6, table.cpu(), pos, 64, interleaved)
        want.append((y, ref.heads_bound(y, size, 64, FP16)))
    handle.qk_norm_rope(q, k, q, k, cos_sin=table, positions=pos.cuda(), q_weight=qw.cuda(),
                        k_weight=kw.cuda(), interleaved=interleaved)
    torch.cuda.synchronize()
    inside(q, *want[0], "q")
    inside(k, *want[1], "k")


def test_positions_outside_the_table_are_clamped(handle):
    q, k, _, _, _, _ = make(4, 2, 1, 64, BF16, seed=5)
    table = lg.rope_table(100, 64)
    pos = torch.tensor([-5, 99, 100, 2 ** 31 - 1], dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    handle.qk_norm_rope(q, k, qo, ko, cos_sin=table, positions=pos.cuda())
    torch.cuda.synchronize()
    y, size = ref.heads(q.cpu(), None, 0, table.cpu(), pos, 64, False)
    inside(qo, y, ref.heads_bound(y, size, 64, BF16), "q")


def test_extreme_values(handle):
    # a zero head stays zero, an infinite or NaN one spoils itself alone
    q, k, _, qw, kw, pos = make(6, 2, 2, 128, BF16, seed=6)
    q[1, 0] = 0
    q[2, 1, 5] = float("inf")
    q[3, 0, 7] = float("nan")
    q[4, 1] = 1e-30
    table = lg.rope_table(4096, 128)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    handle.qk_norm_rope(q, k, qo, ko, cos_sin=table, positions=pos.cuda(), q_weight=qw.cuda(),
                        k_weight=kw.cuda())
    torch.cuda.synchronize()
    got = qo.float().cpu()
    assert (got[1, 0] == 0).all()
    assert got[2, 1].isnan().any() and got[3, 0].isnan().any()
    keep = torch.ones(6, 2, dtype=torch.bool)
    keep[2, 1] = keep[3, 0] = False
    y, size = ref.heads(q.cpu(), qw, 1e-6, table.cpu(), pos, 128, False)
    inside(qo.cpu()[keep], y[keep], ref.heads_bound(y, size, 128, BF16)[keep], "other heads")


def cache_of(pages, Hk, page, D, dtype, order, seed):
    g = torch.Generator().manual_seed(seed)
    full = torch.randn(pages, Hk, page, D, generator=g).to(dtype).cuda()
    if order == "heads":
        return full
    if order == "tokens":  # [pages, page, heads, dim] in memory
        return full.view(torch.uint8 if dtype == E4M3 else dtype).transpose(1, 2).contiguous() \
            .transpose(1, 2).view(dtype)
    both = torch.empty(pages, 2, Hk, page, D, dtype=dtype, device="cuda")  # keys beside values
    raw = both.view(torch.uint8) if dtype == E4M3 else both
    raw.zero_()
    raw[:, seed % 2].copy_(full.view(raw.dtype))
    return both[:, seed % 2]


def as_double(c):
    return c.cpu().float().double()


@pytest.mark.parametrize("order", ["heads", "tokens", "both"])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hk,D,page,dtype", [(1, 8, 2, 128, 16, BF16), (29, 6, 3, 64, 1, FP16),
                                                  (70, 0, 2, 256, 32, BF16), (40, 5, 5, 48, 8, FP16)])
def test_append(handle, T, Hq, Hk, D, page, dtype, cache, order):
    print(f"[append] T={T} {Hq}/{Hk}x{D} page={page} {dtype} {cache} {order}", flush=True)
    q, k, v, qw, kw, pos = make(T, max(Hq, 1), Hk, D, dtype, seed=T)
    cdt = E4M3 if cache == "e4m3" else dtype
    pages = 2 * T // page + 3
    kc, vc = cache_of(pages, Hk, page, D, cdt, order, 0), cache_of(pages, Hk, page, D, cdt, order, 1)
    old_k, old_v = as_double(kc), as_double(vc)
    g = torch.Generator().manual_seed(9)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 4:  # padding, and slots past the cache
        slots[1], slots[3] = -1, pages * page
    rot = 16 if D == 48 else D
    table = lg.rope_table(4096, rot)
    ks = (torch.rand(Hk, generator=g) * 0.05 + 0.02) if cache == "e4m3" else None
    vs = (torch.rand(Hk, generator=g) * 0.05 + 0.02) if cache == "e4m3" else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    extra = {}
    if Hq:
        extra = dict(q=q, q_out=torch.empty_like(q), q_weight=qw.cuda())
    handle.kv_append(k, v, kc, vc, slots.cuda(), cos_sin=table, positions=pos.cuda(),
                     k_weight=kw.cuda(), k_scale=dev(ks), v_scale=dev(vs), **extra)
    torch.cuda.synchronize()
    y, size = ref.heads(k.cpu(), kw, 1e-6, table.cpu(), pos, rot, False)
    one = torch.ones(1, 1, 1, dtype=torch.float64)
    sk = one if ks is None else ks.double().view(1, -1, 1)
    sv = one if vs is None else vs.double().view(1, -1, 1)
    for c, old, val, siz, s, what in ((kc, old_k, y, size, sk, "keys"),
                                      (vc, old_v, v.cpu().double(), v.cpu().double().abs(), sv, "values")):
        got, want = as_double(c), old.clone()
        bound = torch.zeros_like(want)
        for t in range(T):
            s0 = int(slots[t])
            if not 0 <= s0 < pages * page:
                continue
            at = (s0 // page, slice(None), s0 % page)
            if cache == "e4m3":
                want[at] = (val[t] / s[0]).clamp(-448, 448)
                bound[at] = ref.code_bound(val[t] / s[0], siz[t] / s[0], D, 1.0)
            else:
                want[at] = val[t]
                bound[at] = 0 if what == "values" else ref.heads_bound(val[t], siz[t], D, dtype)
        inside(got, want, bound, what)
    if Hq:
        y, size = ref.heads(q.cpu(), qw, 1e-6, table.cpu(), pos, rot, False)
        inside(extra["q_out"], y, ref.heads_bound(y, size, D, dtype), "q")


def test_codes_saturate_and_keep_nan(handle):
    k = torch.tensor([1e4, -1e4, float("inf"), float("-inf"), float("nan"), 448.0, 465.0, 0.0] * 2,
                     dtype=BF16).view(1, 1, 16).cuda()
    kc = torch.zeros(1, 1, 4, 16).to(E4M3).cuda()
    vc = kc.clone()
    handle.kv_append(k, k, kc, vc, torch.tensor([2], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for c in (kc, vc):
        got = c.cpu().float()[0, 0, 2, :8]
        assert got[:4].tolist() == [448.0, -448.0, 448.0, -448.0]
        assert got[4].isnan() and got[5:].tolist() == [448.0, 448.0, 0.0]
        assert (c.cpu().float()[0, 0, [0, 1, 3]] == 0).all()


def test_no_tokens(handle):
    e = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    kc = torch.zeros(2, 4, 16, 64, dtype=BF16, device="cuda")
    handle.qk_norm_rope(e, e, torch.empty_like(e), torch.empty_like(e))
    handle.kv_append(e, e, kc, kc.clone(), i)
    torch.cuda.synchronize()
    assert (kc == 0).all()


def test_a_cache_past_32_bit_offsets(handle):
    # 2^31 + values: the last page lies beyond what 32-bit element offsets reach
    Hk, page, D = 8, 64, 256
    pages = 2 ** 31 // (Hk * page * D) + 3
    kc = torch.zeros(pages, Hk, page, D, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    _, k, v, _, _, _ = make(2, 1, Hk, D, BF16, seed=1)
    slots = torch.tensor([pages * page - 1, 0], dtype=torch.int32)
    handle.kv_append(k, v, kc, vc, slots.cuda())
    torch.cuda.synchronize()
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(vc[-1, :, -1], v[0])
    assert torch.equal(kc[0, :, 0], k[1]) and int((kc != 0).sum()) == int((k != 0).sum())
