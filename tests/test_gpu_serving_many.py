"""The serving operators' forms for many rows, against 64 bits: several batches
and slices of a row of logits, three jobs a wave in the head kernel, and
row tiles beyond what the call's bound foresaw."""
import math

import pytest
import torch

import serving_ref as ref
from test_gpu_serving_attention import BF16, E4M3, FP16, Case, compare
from test_gpu_serving_heads import make

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu

FP32 = torch.float32


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


# ---------------------------------------------------------------- logits

def logits_of(kind, T, V, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + V)
    x = 3 * torch.randn(T, V, generator=g, device="cuda")
    if kind == "sorted":      # the largest in the last batch, or in the first
        x = x.sort(-1).values
        x[1::2] = x[1::2].flip(-1)
    elif kind == "tied":      # far more places with the k-th value than are kept at a time
        x = torch.randint(-2, 3, (T, V), generator=g, device="cuda").float()
        x[::3] = 1.5
    elif kind == "masked":    # a few tokens allowed, far apart
        keep = torch.randint(0, V, (T, 40), generator=g, device="cuda")
        y = torch.full_like(x, -math.inf)
        x = y.scatter(1, keep, x.gather(1, keep))
    return x.to(dtype)


# 300 and 600 rows: a row per workgroup, 10 or 18 batches a wave.  1100: the same
# by the rule for more than 1024 rows; 2100 and 2600: that rule cuts rows in two.
@pytest.mark.parametrize("T,V", [(300, 70001), (600, 40009), (1100, 40009), (2100, 40009), (2600, 36867)])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("kind", ["random", "sorted", "tied", "masked"])
def test_scores_of_many_rows(handle, T, V, dtype, kind):
    x = logits_of(kind, T, V, dtype)
    g = torch.Generator().manual_seed(T)
    tok = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    if kind == "masked":
        tok = x.argmax(-1).to(torch.int32)
    for top in (1, 8, 20, 32):
        print(f"[score many] {dtype} {kind} T={T} V={V} top={top}", flush=True)
        lp, en = torch.full((T,), 77.0, device="cuda"), torch.full((T,), 77.0, device="cuda")
        ids = torch.full((T, top), -7, dtype=torch.int32, device="cuda")
        tl = torch.full((T, top), 77.0, device="cuda")
        handle.token_logprobs(x, tok, lp, entropy=en, top_ids=ids, top_logprobs=tl, temperature=0.8)
        rows = torch.arange(0, T, 1 if top == 20 else 7, device="cuda")  # (64 bits take their time)
        wlp, wen, wids, wtl, bound = ref_rows(x[rows], tok[rows], top)
        lp, en, ids, tl = lp[rows].double(), en[rows].double(), ids[rows].long(), tl[rows].double()
        assert ((lp - wlp).abs() <= bound * (1 + wlp.abs())).all(), float((lp - wlp).abs().max())
        assert ((en - wen).abs() <= 4 * bound * (1 + math.log(V))).all(), float((en - wen).abs().max())
        assert torch.equal(ids, wids)
        same = tl == wtl
        assert (same | ((tl - wtl).abs() <= bound * (1 + wtl.nan_to_num(0.0, neginf=0.0).abs()))).all()


def ref_rows(x, tok, top):
    """serving_ref.score, on the device that holds x."""
    z = x.double()
    logp = torch.log_softmax(z / 0.8, -1)
    lp = logp.gather(1, tok.long()[:, None])[:, 0]
    plogp = torch.where(logp == -math.inf, torch.zeros_like(logp), logp.exp() * logp)
    order = torch.sort(x.float() + 0.0, dim=-1, descending=True, stable=True).indices[:, :top]
    finite = torch.where(z.abs() < 1e30, z, torch.zeros_like(z)).abs().max() / 0.8
    bound = (x.shape[1] / 64 + 64) * ref.U32 + 8 * ref.U32 * float(finite)
    return lp, -plogp.sum(-1), order, logp.gather(1, order), bound


# ----------------------------------------------------------------- heads

def inside(got, want, bound, what, dtype):
    # The bounds of results are relative; an fp16 result below 2^-14 has steps of
    # 2^-24 whatever its size, and is right if it is the rounded one.
    got, exact = got.cpu().double(), want.to(dtype).double()
    off = (got - want).abs()
    ok = (off <= bound) | (got == exact)
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.numel()} values, worst " \
                     f"{float((off / bound).nan_to_num(1e9)[~ok].max()):.3g} of the bound"


# Jobs of a token (groups of heads of one kind in a wave): 9 and 16 at dim 128, 11
# at 64, 10 at 256: none a multiple of the twelve that a workgroup takes.
@pytest.mark.parametrize("T,Hq,Hk,D", [(1100, 20, 5, 128), (1100, 40, 10, 128), (700, 60, 9, 64), (900, 13, 3, 256)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_of_many_tokens_in_place(handle, T, Hq, Hk, D, dtype, interleaved):
    print(f"[heads many] T={T} {Hq}/{Hk}x{D} {dtype} {interleaved}", flush=True)
    q, k, _, qw, kw, pos = make(T, Hq, Hk, D, dtype, seed=T + D)
    table = lg.rope_table(4096, D // 2)
    want = []
    for x, w in ((q, qw), (k, kw)):
        y, size = ref.heads(x.cpu(), w, 1e-6, table.cpu(), pos, D // 2, interleaved)
        want.append((y, ref.heads_bound(y, size, D, dtype)))
    handle.qk_norm_rope(q, k, q, k, cos_sin=table, positions=pos.cuda(), q_weight=qw.cuda(),
                        k_weight=kw.cuda(), interleaved=interleaved)
    torch.cuda.synchronize()
    inside(q, *want[0], "q", dtype)
    inside(k, *want[1], "k", dtype)


@pytest.mark.parametrize("T,Hq,Hk,D,page", [(1100, 20, 5, 128, 16), (1100, 0, 20, 128, 64), (900, 13, 3, 256, 32)])
@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (FP16, FP16), (BF16, E4M3)])
def test_appends_of_many_tokens(handle, T, Hq, Hk, D, page, dtype, cache):
    print(f"[append many] T={T} {Hq}/{Hk}x{D} page={page} {dtype} {cache}", flush=True)
    q, k, v, qw, kw, pos = make(T, max(Hq, 1), Hk, D, dtype, seed=T)
    pages = T // page + 9
    g = torch.Generator().manual_seed(5)
    kc = torch.randn(pages, Hk, page, D, generator=g).to(cache).cuda()
    vc = torch.randn(pages, Hk, page, D, generator=g).to(cache).cuda()
    old_k, old_v = kc.float().double().cpu(), vc.float().double().cpu()
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    slots[5::50] = -1
    table = lg.rope_table(4096, D)
    ks = torch.rand(Hk, generator=g) * 0.05 + 0.02 if cache is E4M3 else None
    vs = torch.rand(Hk, generator=g) * 0.05 + 0.02 if cache is E4M3 else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    extra = dict(q=q, q_out=torch.empty_like(q), q_weight=qw.cuda()) if Hq else {}
    handle.kv_append(k, v, kc, vc, slots.cuda(), cos_sin=table, positions=pos.cuda(),
                     k_weight=kw.cuda(), k_scale=dev(ks), v_scale=dev(vs), **extra)
    torch.cuda.synchronize()
    y, size = ref.heads(k.cpu(), kw, 1e-6, table.cpu(), pos, D, False)
    stored = slots >= 0
    at = slots[stored].long()
    for c, old, val, siz, s, keys in ((kc, old_k, y, size, ks, True),
                                      (vc, old_v, v.cpu().double(), v.cpu().double().abs(), vs, False)):
        want, bound = old.clone(), torch.zeros_like(old)
        if s is not None:
            val, siz = val / s.double()[:, None], siz / s.double()[:, None]
            b = ref.code_bound(val, siz, D, 1.0)
            val = val.clamp(-448, 448)
        else:
            b = ref.heads_bound(val, siz, D, dtype) if keys else torch.zeros_like(val)
        want[at // page, :, at % page] = val[stored]
        bound[at // page, :, at % page] = b[stored]
        inside(c.float(), want, bound, "keys" if keys else "values", cache)
    if Hq:
        y, size = ref.heads(q.cpu(), qw, 1e-6, table.cpu(), pos, D, False)
        inside(extra["q_out"], y, ref.heads_bound(y, size, D, dtype), "q", dtype)


# ------------------------------------------------------------- attention

# The bound of 20 nodes plans one row tile (80 or 320 rows of a key head: of 128 or
# 256 rows), the 300 nodes need several: each workgroup takes more than one.
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("dtype,cache", [(BF16, None), (FP16, None), (BF16, E4M3), (FP16, E4M3)])
@pytest.mark.parametrize("ctx,mask", [(70, "tree"), (1100, "none")])
def test_more_nodes_than_the_bound(handle, D, G, dtype, cache, ctx, mask):
    print(f"[attend many] D={D} G={G} {dtype} {cache} ctx={ctx} {mask}", flush=True)
    c = Case([ctx, 9], [300, 2], 1, G, D, 16, dtype, cache, mask=mask, seed=D + G)
    c.check(handle, max_nodes=20)


@pytest.mark.parametrize("mask", ["tree", "none"])
def test_more_nodes_than_the_bound_in_joined_splits(handle, mask):
    # one row tile of 16 rows planned, 640 workgroups: splits are joined by a
    # second launch, which has to reach the other tiles' rows as well
    c = Case([5000] + [300] * 9, [40, 3] + [1] * 8, 16, 1, 64, 16, BF16, mask=mask, seed=2)
    c.check(handle, max_nodes=1)


@pytest.mark.parametrize("n,G", [(1, 4), (30, 4), (70, 8)])
def test_no_bound_on_the_context(handle, n, G):
    c = Case([3000, 5], [n, 2], 2, G, 128, 16, mask="none", seed=6)
    a = c.run(handle)
    b = c.run(handle, max_context=2 ** 63 - 1)
    want = c.ref()
    compare(a, want)
    compare(b, want)
