"""The norm with codes and the adapters without a GPU: argument errors of the C
entry points and of the binding, and the layout of the argument records."""
import os
import re

import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
from epilogue_scaled_gemm_amd import serving  # noqa: E402

OK, INVALID, UNSUPPORTED = 0, -1, -2
FAKE = 0x10000  # never dereferenced: every call below fails validation or does nothing
BF16 = torch.bfloat16

NORM = ("dtype rows width x x_s residual residual_s residual_out residual_out_s weight eps out out_s "
        "kind codes scales").split()
LORA = ("dtype rows inner width rank x x_s adapters a b ids factors base base_s out out_s slices w0 w1 "
        "w2 w3").split()


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


NORM_OK = dict(rows=0, width=256, x=FAKE, x_s=256, residual=FAKE, residual_s=256, residual_out=FAKE,
               residual_out_s=256, weight=FAKE, eps=1e-6, out=FAKE, out_s=256, codes=FAKE, scales=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(width=-8), INVALID), (dict(width=0), UNSUPPORTED), (dict(width=12, codes=0), UNSUPPORTED),
    (dict(width=24), UNSUPPORTED), (dict(width=24, codes=0), OK), (dict(width=272), OK),
    (dict(width=272, kind=2), UNSUPPORTED), (dict(width=32776, codes=0), UNSUPPORTED),
    (dict(kind=3), INVALID), (dict(kind=-1), INVALID), (dict(kind=9, codes=0), OK),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=1e39), INVALID),
    (dict(rows=1 << 32), UNSUPPORTED), (dict(rows=4, residual_out=0, out=0, codes=0), INVALID),
    (dict(rows=4, x=0), INVALID), (dict(rows=4, weight=0), INVALID), (dict(rows=4, scales=0), INVALID),
    (dict(rows=4, x_s=248), INVALID), (dict(rows=4, out_s=0), INVALID), (dict(rows=4, residual_s=-256), INVALID),
    (dict(rows=4, x_s=260), UNSUPPORTED), (dict(rows=4, residual_out_s=258), UNSUPPORTED),
    (dict(rows=4, x=FAKE + 8), UNSUPPORTED), (dict(rows=4, residual=FAKE + 2), UNSUPPORTED),
    (dict(rows=4, out=FAKE + 4), UNSUPPORTED), (dict(rows=4, weight=FAKE + 8), UNSUPPORTED),
    (dict(rows=4, codes=FAKE + 8), UNSUPPORTED), (dict(rows=4, scales=FAKE + 2), UNSUPPORTED)])
def test_add_rms_norm_refusals(handle, kw, status):
    assert _call(handle, "lin_gemm_add_rms_norm", serving._NORM, NORM, NORM_OK, kw) == status


LORA_OK = dict(rows=0, inner=64, width=48, rank=16, x=FAKE, x_s=64, adapters=3, a=FAKE, b=FAKE, ids=FAKE,
               factors=FAKE, base=FAKE, base_s=48, out=FAKE, out_s=48, slices=1, w0=48)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(dtype=2), INVALID), (dict(rows=-1), INVALID), (dict(adapters=-1), INVALID),
    (dict(inner=-8), INVALID), (dict(rank=0), UNSUPPORTED), (dict(rank=12), UNSUPPORTED),
    (dict(rank=136), UNSUPPORTED), (dict(inner=0), UNSUPPORTED), (dict(inner=20), UNSUPPORTED),
    (dict(inner=(1 << 20) + 8), UNSUPPORTED), (dict(width=0, w0=0), UNSUPPORTED),
    (dict(width=(1 << 20) + 1), UNSUPPORTED), (dict(rows=1 << 24), UNSUPPORTED),
    (dict(adapters=1 << 31), UNSUPPORTED), (dict(slices=0), UNSUPPORTED), (dict(slices=5), UNSUPPORTED),
    (dict(w0=47), INVALID), (dict(slices=2, w1=0), INVALID), (dict(slices=2, w0=64, w1=-16), INVALID),
    (dict(slices=3, w0=16, w1=16, w2=16), OK), (dict(w0=1 << 62), INVALID),
    (dict(rows=4, x=0), INVALID), (dict(rows=4, a=0), INVALID), (dict(rows=4, b=0), INVALID),
    (dict(rows=4, ids=0), INVALID), (dict(rows=4, out=0), INVALID), (dict(rows=4, x_s=56), INVALID),
    (dict(rows=4, base_s=40), INVALID), (dict(rows=4, out_s=-48), INVALID), (dict(rows=4, x_s=68), UNSUPPORTED),
    (dict(rows=4, x=FAKE + 8), UNSUPPORTED), (dict(rows=4, a=FAKE + 2), UNSUPPORTED),
    (dict(rows=4, b=FAKE + 8), UNSUPPORTED), (dict(rows=4, ids=FAKE + 2), UNSUPPORTED),
    (dict(rows=4, factors=FAKE + 1), UNSUPPORTED), (dict(rows=4, out=FAKE + 1), UNSUPPORTED),
    (dict(rows=4, base=FAKE + 1), UNSUPPORTED)])
def test_lora_add_refusals(handle, kw, status):
    assert _call(handle, "lin_gemm_lora_add", serving._LORA, LORA, LORA_OK, kw) == status


WINDOW = ("dtype tokens q_heads kv_heads dim q q_ts q_hs kc kc_ps kc_hs kc_ts vc vc_ps vc_hs vc_ts "
          "cache_type pages page_size k_scale v_scale sequences table table_stride max_pages context "
          "offsets max_context max_nodes mask mask_words scale out lse window sinks positions").split()
WINDOW_OK = dict(tokens=0, q_heads=4, kv_heads=2, dim=128, q=FAKE, q_ts=512, q_hs=128, kc=FAKE,
                 kc_ps=4096, kc_hs=2048, kc_ts=128, vc=FAKE, vc_ps=4096, vc_hs=2048, vc_ts=128,
                 pages=8, page_size=16, sequences=2, table=FAKE, table_stride=4, max_pages=4,
                 context=FAKE, offsets=FAKE, max_context=32, max_nodes=2, scale=0.1, out=FAKE, window=16)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(window=0), INVALID), (dict(window=-5), INVALID), (dict(sinks=-1), INVALID),
    (dict(window=1 << 62, sinks=1 << 62), OK), (dict(positions=FAKE), INVALID),
    (dict(positions=FAKE, mask=FAKE, mask_words=1), OK),
    (dict(tokens=4, positions=FAKE + 2, mask=FAKE, mask_words=1), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(dim=96), UNSUPPORTED), (dict(tokens=4, q=0), INVALID),
    (dict(tokens=4, mask=FAKE + 4, mask_words=1), UNSUPPORTED), (dict(tokens=4, out=FAKE + 2), UNSUPPORTED)])
def test_window_attention_refusals(handle, kw, status):
    assert _call(handle, "lin_gemm_window_attention", serving._WINDOW, WINDOW, WINDOW_OK, kw) == status


def test_null_handle_and_null_arguments(handle):
    for f in ("add_rms_norm", "lora_add", "window_attention"):
        entry = getattr(lg.library(), "lin_gemm_" + f)
        assert entry(None, None, None) == INVALID and entry(handle._h, None, None) == INVALID


def test_records_match_the_header():
    # every field of a record is eight bytes wide
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                             "include", "lin_gemm.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, fmt, names in (("lin_norm_t", serving._NORM, NORM), ("lin_lora_t", serving._LORA, LORA)):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1)
        count = 0
        for line in filter(None, (x.strip() for x in body.split(";"))):
            for part in line.split(","):
                size = re.search(r"\[(\d+)\]", part)
                count += int(size.group(1)) if size else 1
        assert count == len(names) and fmt.size == 8 * count
    # the windowed record is the other attention's and three fields more
    body = re.search(r"typedef struct \{([^}]*)\} lin_window_t;", text).group(1)
    assert [x.split()[-1].lstrip("*") for x in body.replace(",", ";").split(";") if x.strip()] == [
        "attention", "window", "sinks", "positions"]
    assert serving._WINDOW.size == serving._ATTENTION.size + 24 == 8 * len(WINDOW)


@pytest.fixture()
def addressed(handle, monkeypatch):
    # CPU tensors stand for GPU ones up to the call itself
    monkeypatch.setattr(serving, "_at", lambda name, t: t.data_ptr())
    monkeypatch.setattr(serving, "_stream_of", lambda stream, t: None)
    return handle


def _t(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("bad", ["dtype", "dims", "weight", "weight_dtype", "residual", "residual_dtype", "out",
                                 "inner", "kind", "codes_dtype", "codes", "scales", "scales_alone", "block",
                                 "grad"])
def test_binding_refuses_wrong_norms(addressed, bad):
    kw = dict(x=_t(3, 256), weight=_t(256), residual=_t(3, 256), residual_out=_t(3, 256), out=_t(3, 256),
              codes=_t(3, 256, dtype=torch.float8_e4m3fn), scales=torch.zeros(3))
    error, match = ValueError, None
    if bad == "dtype":
        kw["x"] = torch.zeros(3, 256)
    elif bad == "dims":
        kw["x"] = _t(256)
    elif bad == "weight":
        kw["weight"] = _t(128)
    elif bad == "weight_dtype":
        kw["weight"] = torch.zeros(256)
    elif bad == "residual":
        kw["residual"] = _t(1, 256)
    elif bad == "residual_dtype":
        kw["residual"] = torch.zeros(3, 256)
    elif bad == "out":
        kw["out"] = _t(4, 256)
    elif bad == "inner":
        kw["x"] = _t(256, 3).t()
    elif bad == "kind":
        kw["kind"] = "fp8"
    elif bad == "codes_dtype":
        kw["kind"] = "int8_token"
    elif bad == "codes":
        kw["codes"] = _t(3, 128, dtype=torch.float8_e4m3fn)
    elif bad == "scales":
        kw["scales"] = torch.zeros(6)
    elif bad == "scales_alone":
        kw["codes"] = None
    elif bad == "block":
        kw["kind"] = "fp8_block"
    elif bad == "grad":
        kw["weight"].requires_grad_()
        error, match = RuntimeError, "forward only"
    with pytest.raises(error, match=match):
        addressed.add_rms_norm(**kw)


@pytest.mark.parametrize("bad", ["dtype", "a", "a_slices", "a_dtype", "b_strided", "ids", "ids_dtype", "out",
                                 "out_dtype", "base", "factors", "slices", "many_slices", "inner", "grad"])
def test_binding_refuses_wrong_adapters(addressed, bad):
    kw = dict(x=_t(3, 64), a=_t(2, 16, 64), b=_t(2, 48, 16), ids=_t(3, dtype=torch.int32), out=_t(3, 48),
              base=_t(3, 48), factors=torch.zeros(2))
    error, match = ValueError, None
    if bad == "dtype":
        kw["x"] = torch.zeros(3, 64)
    elif bad == "a":
        kw["a"] = _t(3, 16, 64)
    elif bad == "a_slices":
        kw["slices"] = (16, 32)
    elif bad == "a_dtype":
        kw["a"] = kw["a"].half()
    elif bad == "b_strided":
        kw["b"] = _t(2, 16, 48).transpose(1, 2)
    elif bad == "ids":
        kw["ids"] = _t(1, dtype=torch.int32)
    elif bad == "ids_dtype":
        kw["ids"] = _t(3, dtype=torch.int64)
    elif bad == "out":
        kw["out"] = _t(3, 40)
    elif bad == "out_dtype":
        kw["out"] = torch.zeros(3, 48)
    elif bad == "base":
        kw["base"] = _t(1, 48).expand(3, 48)[:1]
    elif bad == "factors":
        kw["factors"] = torch.zeros(3)
    elif bad == "slices":
        kw["slices"] = (24, 16)
    elif bad == "many_slices":
        kw.update(a=_t(2, 80, 64), slices=(8, 8, 8, 8, 16))
    elif bad == "inner":
        kw["x"] = _t(64, 3).t()
    elif bad == "grad":
        kw["a"].requires_grad_()
        error, match = RuntimeError, "forward only"
    with pytest.raises(error, match=match):
        addressed.lora_add(**kw)


@pytest.mark.parametrize("bad", ["positions", "positions_dtype", "without_mask", "mask", "grad"])
def test_binding_refuses_wrong_windows(addressed, bad):
    i32 = dict(dtype=torch.int32)
    kw = dict(q=_t(3, 4, 64), k_cache=_t(6, 2, 16, 64), v_cache=_t(6, 2, 16, 64), out=_t(3, 4, 64),
              page_table=torch.zeros(2, 3, **i32), context=torch.zeros(2, **i32), offsets=torch.zeros(3, **i32),
              max_context=10, max_nodes=2, window=8, mask=torch.zeros(3, 1, dtype=torch.int64),
              positions=torch.zeros(3, **i32))
    error, match = ValueError, None
    if bad == "positions":
        kw["positions"] = torch.zeros(2, **i32)
    elif bad == "positions_dtype":
        kw["positions"] = torch.zeros(3, dtype=torch.int64)
    elif bad == "without_mask":
        kw["mask"] = None
    elif bad == "mask":
        kw["mask"] = torch.zeros(2, 1, dtype=torch.int64)
    elif bad == "grad":
        kw["q"].requires_grad_()
        error, match = RuntimeError, "forward only"
    with pytest.raises(error, match=match):
        addressed.window_attention(**kw)


def test_a_row_that_stands_for_many_is_refused(addressed):
    # stride 0 between rows of an output would be written by all of them
    with pytest.raises(lg.LinGemmError):
        addressed.add_rms_norm(_t(3, 64), _t(64), out=_t(1, 64).expand(3, 64))
