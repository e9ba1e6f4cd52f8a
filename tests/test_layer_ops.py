"""Dispatcher entries of the norm with codes, the adapters and the windowed
attention without a GPU."""
import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
import epilogue_scaled_gemm_amd.torch_ops  # noqa: E402,F401

ops = torch.ops.lingemm
BF16, I32 = torch.bfloat16, torch.int32


def meta(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_fake_shapes():
    x, w = meta(7, 256), meta(256)
    total, out, codes, scales = ops.add_rms_norm(x, w)
    assert total.shape == codes.shape == scales.shape == (0,) and out.shape == x.shape
    for kind, dt, ss in (("fp8_token", torch.float8_e4m3fn, (7,)), ("int8_token", torch.int8, (7,)),
                         ("fp8_block", torch.float8_e4m3fn, (7, 2))):
        total, out, codes, scales = ops.add_rms_norm(x, w, residual=x, kind=kind)
        assert total.shape == out.shape == codes.shape == x.shape and total.dtype == out.dtype == BF16
        assert codes.dtype == dt and scales.shape == ss and scales.dtype == torch.float32
    y = ops.lora_add(x, meta(3, 16, 256), meta(3, 40, 16), meta(7, dtype=I32))
    assert y.shape == (7, 40) and y.dtype == BF16
    q, cache = meta(7, 8, 64), meta(4, 2, 16, 64)
    out, lse = ops.window_attention(q, cache, cache, meta(2, 3, dtype=I32), meta(2, dtype=I32),
                                    meta(3, dtype=I32), 40, 4, 16, 2)
    assert out.shape == q.shape and lse.shape == (7, 8) and lse.dtype == torch.float32


def test_fakes_refuse():
    with pytest.raises(ValueError):
        ops.add_rms_norm(meta(7, 256, dtype=torch.float32), meta(256))
    with pytest.raises(ValueError):
        ops.add_rms_norm(meta(7, 256), meta(256), kind="fp8")
    with pytest.raises(ValueError):
        ops.lora_add(meta(256), meta(3, 16, 256), meta(3, 40, 16), meta(1, dtype=I32))
    with pytest.raises(ValueError):
        ops.window_attention(meta(7, 512), meta(4, 2, 16, 64), meta(4, 2, 16, 64), meta(2, 3, dtype=I32),
                             meta(2, dtype=I32), meta(3, dtype=I32), 40, 4, 16)


def test_cpu_tensors_are_refused():
    with pytest.raises(Exception):
        ops.add_rms_norm(torch.zeros(2, 64, dtype=BF16), torch.ones(64, dtype=BF16))
