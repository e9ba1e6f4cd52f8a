"""The draft-verification example at contexts beyond 32768 positions."""
import importlib.util
import os

import pytest
import torch

pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_context_of_40000():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("verify_drafts",
                                                  os.path.join(ROOT, "examples", "verify_drafts.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    with torch.no_grad():
        d = example.Drafts(2, 40000, 5, 64, 1000)
        layer = example.Layer(512, 8, 2, 64, 1000, d.pages, 64, False)
        assert layer.table.shape[0] > int(d.positions.max())
        got = example.verify(layer, d)
        worst = example.check(layer, d, got)
    assert all(v <= 1 for v in worst.values()), worst
