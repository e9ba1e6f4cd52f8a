"""Factors that 64 bits hold and the kernels' 32 do not are refused, on the CPU,
before anything is enqueued."""
import os

import pytest
import torch

from test_serving_host import ATT, ATT_OK, INVALID, OK, SCORE, SCORE_OK

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
from epilogue_scaled_gemm_amd import serving  # noqa: E402


@pytest.fixture()
def handle():
    if not os.path.exists(lg.LIB_PATH):
        pytest.skip("library not built")
    h = lg.Handle()
    yield h
    h.close()


def call(h, entry, fmt, names, base, **kw):
    d = dict(base, **kw)  # no tokens: nothing is launched
    return getattr(lg.library(), entry)(h._h, fmt.pack(*[d.get(n, 0) for n in names]), None)


@pytest.mark.parametrize("temperature,status", [
    (1e-40, INVALID), (3e-39, INVALID), (5e-324, INVALID), (1e-38, OK), (0.7, OK), (1e44, OK),
    (1e46, INVALID), (1e300, INVALID)])
def test_temperatures(handle, temperature, status):
    assert call(handle, "lin_gemm_token_logprobs", serving._SCORE, SCORE, SCORE_OK,
                temperature=temperature) == status


@pytest.mark.parametrize("scale,status", [
    (1e39, INVALID), (-1e39, INVALID), (2.4e38, INVALID), (2.3e38, OK), (-2.3e38, OK), (0.0, OK),
    (1e-300, OK)])
def test_scales(handle, scale, status):
    assert call(handle, "lin_gemm_tree_attention", serving._ATTENTION, ATT, ATT_OK,
                scale=scale) == status
