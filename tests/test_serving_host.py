"""The serving operators without a GPU: argument errors of the C entry points
and of the binding, the layout of the argument records, and the plans'
helpers.  Nothing here reaches a device."""
import os

import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
from epilogue_scaled_gemm_amd import serving  # noqa: E402

needs_lib = pytest.mark.skipif(not os.path.exists(lg.LIB_PATH), reason="library not built")
OK, INVALID, UNSUPPORTED = 0, -1, -2
FAKE = 0x10000  # never dereferenced: every call below fails validation or does nothing

HEADS = ("dtype tokens dim q_heads q q_ts q_hs q_out qo_ts qo_hs kv_heads k k_ts k_hs k_out ko_ts "
         "ko_hs v v_ts v_hs kc kc_ps kc_hs kc_ts vc vc_ps vc_hs vc_ts cache_type pages page_size "
         "k_scale v_scale slots qw kw eps rope rope_rows rope_dim positions interleaved").split()
ATT = ("dtype tokens q_heads kv_heads dim q q_ts q_hs kc kc_ps kc_hs kc_ts vc vc_ps vc_hs vc_ts "
       "cache_type pages page_size k_scale v_scale sequences table table_stride max_pages context "
       "offsets max_context max_nodes mask mask_words scale out lse").split()
SCORE = ("dtype rows vocab logits row_stride tokens temperature logprobs entropy top top_ids "
         "top_logprobs").split()


@pytest.fixture()
def handle():
    if torch.cuda.is_available():
        pytest.skip("fake-pointer error paths run on the CPU only")
    if not os.path.exists(lg.LIB_PATH):
        pytest.skip("library not built")
    h = lg.Handle()
    yield h
    h.close()


def _call(h, entry, fmt, names, base, kw):
    d = dict(base)
    d.update(kw)
    assert set(d) <= set(names)
    rc = getattr(lg.library(), entry)(h._h, fmt.pack(*[d.get(n, 0) for n in names]), None)
    if rc != OK:
        assert lg.library().lin_gemm_last_error(h._h)
    return rc


HEADS_OK = dict(tokens=0, dim=128, q_heads=4, q=FAKE, q_ts=512, q_hs=128, q_out=FAKE, qo_ts=512,
                qo_hs=128, kv_heads=2, k=FAKE, k_ts=256, k_hs=128, k_out=FAKE, ko_ts=256,
                ko_hs=128, v=FAKE, v_ts=256, v_hs=128, kc=FAKE, kc_ps=4096, kc_hs=2048, kc_ts=128,
                vc=FAKE, vc_ps=4096, vc_hs=2048, vc_ts=128, pages=8, page_size=16, slots=FAKE,
                eps=1e-6, rope=FAKE, rope_rows=64, rope_dim=128, positions=FAKE)

BOTH = [
    (dict(), OK),                                   # no tokens: nothing to do
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(tokens=-1), INVALID), (dict(q_heads=-1), INVALID), (dict(kv_heads=-3), INVALID),
    (dict(dim=0), UNSUPPORTED), (dict(dim=24), UNSUPPORTED), (dict(dim=272), UNSUPPORTED),
    (dict(tokens=1 << 40), UNSUPPORTED), (dict(q_heads=5000), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(rope_dim=8), UNSUPPORTED), (dict(rope_dim=144), UNSUPPORTED),
    (dict(rope_rows=0), INVALID), (dict(tokens=4, positions=0), INVALID),
    (dict(tokens=4, q=0), INVALID), (dict(tokens=4, q_out=0), INVALID), (dict(tokens=4, k=0), INVALID),
    (dict(tokens=4, q=FAKE + 8), UNSUPPORTED), (dict(tokens=4, q_ts=260), UNSUPPORTED),
    (dict(tokens=4, k_hs=4), UNSUPPORTED), (dict(tokens=4, qw=FAKE + 2), UNSUPPORTED),
    (dict(tokens=4, rope=FAKE + 4), UNSUPPORTED), (dict(tokens=4, positions=FAKE + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(tokens=4, k_out=0), INVALID), (dict(tokens=4, ko_ts=2), UNSUPPORTED),
    (dict(tokens=4, q_heads=0, kv_heads=0), OK)])
def test_qk_norm_rope_refusals(handle, kw, status):
    assert _call(handle, "lin_gemm_qk_norm_rope", serving._HEADS, HEADS, HEADS_OK, kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(kv_heads=0), INVALID), (dict(cache_type=3), INVALID), (dict(cache_type=1), UNSUPPORTED),
    (dict(pages=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=24), UNSUPPORTED),
    (dict(pages=1 << 28, page_size=16), UNSUPPORTED), (dict(kc=0), INVALID), (dict(vc=0), INVALID),
    (dict(kc=FAKE + 4), UNSUPPORTED), (dict(kc_ts=4), UNSUPPORTED),
    (dict(cache_type=2, kc_ts=8), UNSUPPORTED), (dict(tokens=4, v=0), INVALID),
    (dict(tokens=4, slots=0), INVALID), (dict(tokens=4, slots=FAKE + 2), UNSUPPORTED),
    (dict(tokens=4, v_ts=4), UNSUPPORTED), (dict(tokens=4, k_scale=FAKE + 1), UNSUPPORTED)])
def test_kv_append_refusals(handle, kw, status):
    assert _call(handle, "lin_gemm_kv_append", serving._HEADS, HEADS, HEADS_OK, kw) == status


ATT_OK = dict(tokens=0, q_heads=4, kv_heads=2, dim=128, q=FAKE, q_ts=512, q_hs=128, kc=FAKE,
              kc_ps=4096, kc_hs=2048, kc_ts=128, vc=FAKE, vc_ps=4096, vc_hs=2048, vc_ts=128,
              pages=8, page_size=16, sequences=2, table=FAKE, table_stride=4, max_pages=4,
              context=FAKE, offsets=FAKE, max_context=32, max_nodes=2, scale=0.1, out=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(tokens=4, sequences=0), OK),
    (dict(dtype=2), INVALID), (dict(tokens=-1), INVALID), (dict(sequences=-1), INVALID),
    (dict(max_context=-1), INVALID), (dict(max_nodes=-1), INVALID), (dict(mask_words=-1), INVALID),
    (dict(dim=96), UNSUPPORTED), (dict(dim=512), UNSUPPORTED), (dict(kv_heads=0), UNSUPPORTED),
    (dict(q_heads=0), UNSUPPORTED), (dict(kv_heads=3), UNSUPPORTED),
    (dict(tokens=1 << 30), UNSUPPORTED), (dict(sequences=1 << 20), UNSUPPORTED),
    (dict(tokens=1 << 22, q_heads=64), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(cache_type=5), INVALID), (dict(cache_type=1), UNSUPPORTED), (dict(page_size=12), UNSUPPORTED),
    (dict(pages=0), INVALID), (dict(vc=0), INVALID), (dict(vc_ps=4), UNSUPPORTED),
    (dict(tokens=4, q=0), INVALID), (dict(tokens=4, out=0), INVALID), (dict(tokens=4, table=0), INVALID),
    (dict(tokens=4, context=0), INVALID), (dict(tokens=4, offsets=0), INVALID),
    (dict(tokens=4, max_pages=0), INVALID), (dict(tokens=4, table_stride=3), INVALID),
    (dict(tokens=4, max_pages=1 << 27, table_stride=1 << 27), INVALID),
    (dict(tokens=4, mask=FAKE, mask_words=1 << 21), UNSUPPORTED),
    (dict(tokens=4, q=FAKE + 8), UNSUPPORTED), (dict(tokens=4, q_hs=4), UNSUPPORTED),
    (dict(tokens=4, out=FAKE + 2), UNSUPPORTED), (dict(tokens=4, mask=FAKE + 4, mask_words=1), UNSUPPORTED),
    (dict(tokens=4, lse=FAKE + 1), UNSUPPORTED)])
def test_tree_attention_refusals(handle, kw, status):
    assert _call(handle, "lin_gemm_tree_attention", serving._ATTENTION, ATT, ATT_OK, kw) == status


@pytest.mark.parametrize("name", ["kc", "vc"])
@pytest.mark.parametrize("stride,value,status", [
    ("_ps", -8, UNSUPPORTED), ("_ps", 1 << 30, UNSUPPORTED), ("_ts", -8, UNSUPPORTED),
    ("_ts", 1 << 26, UNSUPPORTED), ("_ts", 1 << 40, UNSUPPORTED)])
def test_tree_attention_refuses_pages_beyond_32_bit_offsets(handle, name, stride, value, status):
    kw = {"tokens": 4, name + stride: value}
    assert _call(handle, "lin_gemm_tree_attention", serving._ATTENTION, ATT, ATT_OK, kw) == status


SCORE_OK = dict(rows=0, vocab=100, logits=FAKE, row_stride=100, tokens=FAKE, temperature=1.0,
                logprobs=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(vocab=-1), INVALID),
    (dict(top=-1), INVALID), (dict(temperature=0.0), INVALID), (dict(temperature=-1.0), INVALID),
    (dict(temperature=float("nan")), INVALID), (dict(temperature=float("inf")), INVALID),
    (dict(top=33), UNSUPPORTED), (dict(top=20, vocab=10), UNSUPPORTED),
    (dict(rows=4, vocab=0), UNSUPPORTED), (dict(rows=1 << 30), UNSUPPORTED),
    (dict(vocab=1 << 31), UNSUPPORTED), (dict(rows=4, logits=0), INVALID),
    (dict(rows=4, tokens=0), INVALID), (dict(rows=4, logprobs=0), INVALID),
    (dict(rows=4, row_stride=99), INVALID), (dict(rows=4, logits=FAKE + 1), UNSUPPORTED),
    (dict(rows=4, dtype=2, logits=FAKE + 2), UNSUPPORTED), (dict(rows=4, entropy=FAKE + 2), UNSUPPORTED)])
def test_token_logprobs_refusals(handle, kw, status):
    assert _call(handle, "lin_gemm_token_logprobs", serving._SCORE, SCORE, SCORE_OK, kw) == status


@needs_lib
def test_null_handle_and_null_arguments():
    lib = lg.library()
    for f in ("qk_norm_rope", "kv_append", "tree_attention", "token_logprobs"):
        assert getattr(lib, "lin_gemm_" + f)(None, None, None) == INVALID


def test_null_arguments(handle):
    lib = lg.library()
    for f in ("qk_norm_rope", "kv_append", "tree_attention", "token_logprobs"):
        assert getattr(lib, "lin_gemm_" + f)(handle._h, None, None) == INVALID


def test_records_match_the_header():
    # every field of the three records is eight bytes wide
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                             "include", "lin_gemm.h")).read()
    import re
    for name, fmt in (("lin_heads_t", serving._HEADS), ("lin_attention_t", serving._ATTENTION),
                      ("lin_score_t", serving._SCORE)):
        end = text.index("} " + name + ";")
        body = text[text.rindex("typedef struct {", 0, end):end]
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S).split("{", 1)[1]
        fields, kinds = [], ""
        for decl in body.split(";"):
            decl = decl.strip()
            if not decl:
                continue
            kind = "d" if decl.startswith("double") else "q"
            n = len(decl.split(","))
            fields += [decl] * n
            kinds += kind * n
            assert "*" in decl or decl.split()[0] in ("int64_t", "double"), decl
        assert fmt.size == 8 * len(fields)
        got = "".join((c[-1]) * int(c[:-1] or 1) for c in re.findall(r"\d*[qd]", fmt.format))
        assert got == kinds, name


@pytest.fixture()
def addressed(handle, monkeypatch):
    """A handle whose binding takes CPU tensors: only a check of the binding
    itself can raise ValueError (a call that got through would fail in the
    library, there being no device)."""
    monkeypatch.setattr(serving, "_at", lambda name, t: FAKE)
    monkeypatch.setattr(serving, "_stream_of", lambda stream, t: 0)
    return handle


def test_binding_refuses_cpu_tensors(handle):
    with pytest.raises(ValueError, match="GPU"):
        handle.qk_norm_rope(_bf(3, 4, 64), _bf(3, 2, 64), _bf(3, 4, 64), _bf(3, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        handle.token_logprobs(torch.zeros(3, 50), torch.zeros(3, dtype=torch.int32), torch.zeros(3))


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("bad", ["dtype", "k_dtype", "dim", "rows", "out_shape", "inner", "weight",
                                 "table", "positions", "positions_dtype", "grad"])
def test_binding_refuses_wrong_heads(addressed, bad):
    q, k = _bf(3, 4, 64), _bf(3, 2, 64)
    kw = dict(q=q, k=k, q_out=_bf(3, 4, 64), k_out=_bf(3, 2, 64), cos_sin=torch.zeros(9, 64),
              positions=torch.zeros(3, dtype=torch.int32), q_weight=_bf(64))
    error, match = ValueError, None
    if bad == "dtype":
        kw["q"] = q.float()
    elif bad == "k_dtype":
        kw["k"] = k.half()
    elif bad == "dim":
        kw["k"] = _bf(3, 2, 32)
    elif bad == "rows":
        kw["k"] = _bf(1, 2, 64)
    elif bad == "out_shape":
        kw["q_out"] = _bf(3, 1, 64)
    elif bad == "inner":
        kw["q_out"] = _bf(3, 64, 4).transpose(1, 2)
    elif bad == "weight":
        kw["q_weight"] = _bf(1)
    elif bad == "table":
        kw["cos_sin"] = torch.zeros(9, 64, dtype=torch.float64)
    elif bad == "positions":
        kw["positions"] = None
    elif bad == "positions_dtype":
        kw["positions"] = torch.zeros(3, dtype=torch.int64)
    elif bad == "grad":
        kw["q"] = q.requires_grad_()
        error, match = RuntimeError, "forward only"
    with pytest.raises(error, match=match):
        addressed.qk_norm_rope(**kw)


@pytest.mark.parametrize("bad", ["cache_heads", "cache_dtype", "v_cache", "slots", "scale16", "scale",
                                 "q_alone", "qw_alone", "q_rows", "inner"])
def test_binding_refuses_wrong_appends(addressed, bad):
    kw = dict(k=_bf(3, 2, 64), v=_bf(3, 2, 64), k_cache=_bf(5, 2, 16, 64), v_cache=_bf(5, 2, 16, 64),
              slots=torch.zeros(3, dtype=torch.int32))
    if bad == "cache_heads":
        kw["k_cache"] = _bf(5, 1, 16, 64)
    elif bad == "cache_dtype":
        kw["k_cache"] = kw["k_cache"].half()
    elif bad == "v_cache":
        kw["v_cache"] = _bf(4, 2, 16, 64)
    elif bad == "slots":
        kw["slots"] = torch.zeros(2, dtype=torch.int32)
    elif bad == "scale16":
        kw["k_scale"] = torch.ones(2)
    elif bad == "scale":
        kw.update(k_cache=torch.zeros(5, 2, 16, 64).to(torch.float8_e4m3fn),
                  v_cache=torch.zeros(5, 2, 16, 64).to(torch.float8_e4m3fn), k_scale=torch.ones(1))
    elif bad == "q_alone":
        kw["q"] = _bf(3, 4, 64)
    elif bad == "qw_alone":
        kw["q_weight"] = _bf(64)
    elif bad == "q_rows":
        kw.update(q=_bf(2, 4, 64), q_out=_bf(2, 4, 64))
    elif bad == "inner":
        kw["k_cache"] = _bf(5, 2, 64, 16).transpose(2, 3)
    with pytest.raises(ValueError):
        addressed.kv_append(**kw)


@pytest.mark.parametrize("bad", ["dim", "v_cache", "table_dtype", "context", "offsets", "mask_rows",
                                 "mask_words", "mask_dtype", "out", "lse", "grad"])
def test_binding_refuses_wrong_attention(addressed, bad):
    i32 = torch.int32
    kw = dict(q=_bf(3, 4, 64), k_cache=_bf(5, 2, 16, 64), v_cache=_bf(5, 2, 16, 64),
              out=_bf(3, 4, 64), page_table=torch.zeros(2, 2, dtype=i32),
              context=torch.zeros(2, dtype=i32), offsets=torch.zeros(3, dtype=i32), max_context=16,
              max_nodes=2, mask=torch.zeros(3, 1, dtype=torch.int64))
    error, match = ValueError, None
    if bad == "dim":
        kw["k_cache"] = _bf(5, 2, 16, 128)
    elif bad == "v_cache":
        kw["v_cache"] = _bf(5, 2, 8, 64)
    elif bad == "table_dtype":
        kw["page_table"] = kw["page_table"].long()
    elif bad == "context":
        kw["context"] = torch.zeros(1, dtype=i32)
    elif bad == "offsets":
        kw["offsets"] = torch.zeros(2, dtype=i32)
    elif bad == "mask_rows":
        kw["mask"] = torch.zeros(1, 1, dtype=torch.int64)
    elif bad == "mask_words":
        kw["max_nodes"] = 65
    elif bad == "mask_dtype":
        kw["mask"] = torch.zeros(3, 1, dtype=torch.bool)
    elif bad == "out":
        kw["out"] = _bf(3, 4, 64).half()
    elif bad == "lse":
        kw["lse"] = torch.zeros(3)
    elif bad == "grad":
        kw["q"].requires_grad_()
        error, match = RuntimeError, "forward only"
    with pytest.raises(error, match=match):
        addressed.tree_attention(**kw)


@pytest.mark.parametrize("bad", ["dtype", "inner", "tokens", "tokens_dtype", "top_rows", "top_widths",
                                 "ids_dtype", "entropy", "grad"])
def test_binding_refuses_wrong_scores(addressed, bad):
    kw = dict(logits=torch.zeros(3, 50), tokens=torch.zeros(3, dtype=torch.int32),
              logprobs=torch.zeros(3), entropy=torch.zeros(3),
              top_ids=torch.zeros(3, 4, dtype=torch.int32), top_logprobs=torch.zeros(3, 4))
    error, match = ValueError, None
    if bad == "dtype":
        kw["logits"] = torch.zeros(3, 50, dtype=torch.float64)
    elif bad == "inner":
        kw["logits"] = torch.zeros(50, 3).t()
    elif bad == "tokens":
        kw["tokens"] = torch.zeros(1, dtype=torch.int32)
    elif bad == "tokens_dtype":
        kw["tokens"] = torch.zeros(3, dtype=torch.int64)
    elif bad == "top_rows":
        kw["top_ids"] = torch.zeros(2, 4, dtype=torch.int32)
    elif bad == "top_widths":
        kw["top_logprobs"] = torch.zeros(3, 5)
    elif bad == "ids_dtype":
        kw["top_ids"] = torch.zeros(3, 4)
    elif bad == "entropy":
        kw["entropy"] = torch.zeros(3, dtype=torch.float64)
    elif bad == "grad":
        kw["logits"].requires_grad_()
        error, match = RuntimeError, "forward only"
    with pytest.raises(error, match=match):
        addressed.token_logprobs(**kw)


def test_tree_mask_and_depth():
    mask, depth = lg.tree_mask([[-1, 0, 0, 1, -1], [-1]], device="cpu")
    assert mask.shape == (6, 1) and mask.dtype == torch.int64
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b1]
    assert depth.tolist() == [0, 1, 1, 2, 0, 0]
    chain, depth = lg.tree_mask([list(range(-1, 129))], device="cpu")
    assert chain.shape == (130, 3)
    assert chain[63].tolist() == [-1, 0, 0] and chain[129].tolist() == [-1, -1, 3]
    assert depth.tolist() == list(range(130))
    with pytest.raises(ValueError):
        lg.tree_mask([[-1, 1]], device="cpu")
    with pytest.raises(ValueError):
        lg.tree_mask([[-2]], device="cpu")


def test_node_slots():
    table = torch.tensor([[7, 2, 0], [5, 1, 3]], dtype=torch.int32)
    ctx = torch.tensor([3, 5], dtype=torch.int32)
    off = torch.tensor([0, 3, 4], dtype=torch.int32)
    got = lg.node_slots(table, ctx, off, 4)
    # positions 3, 4, 5 of the first sequence, 5 of the second
    assert got.tolist() == [7 * 4 + 3, 2 * 4, 2 * 4 + 1, 1 * 4 + 1] and got.dtype == torch.int32
    # an empty sequence in between
    off = torch.tensor([0, 0, 2], dtype=torch.int32)
    assert lg.node_slots(table, ctx, off, 4).tolist() == [1 * 4 + 1, 1 * 4 + 2]


def test_rope_table_keeps_far_phases():
    t = lg.rope_table(200001, 32, device="cpu")
    assert t.shape == (200001, 32) and t.dtype == torch.float32
    i, pos = 3, 200000
    angle = pos * 10000.0 ** (-2 * i / 32)
    import math
    # correctly rounded to fp32 from 64 bits: half a step of 1
    assert abs(float(t[pos, i]) - math.cos(angle)) < 2.0 ** -24
    assert abs(float(t[pos, 16 + i]) - math.sin(angle)) < 2.0 ** -24
