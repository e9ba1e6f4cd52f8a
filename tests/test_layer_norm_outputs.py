"""The dispatcher's norm gives the outputs that are asked for and computes no others."""
import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
import epilogue_scaled_gemm_amd.torch_ops  # noqa: E402,F401

ops = torch.ops.lingemm
BF16 = torch.bfloat16


def meta(*shape):
    return torch.empty(*shape, dtype=BF16, device="meta")


def test_fake_shapes_without_the_16_bit_rows():
    x, w = meta(7, 256), meta(256)
    total, out, codes, scales = ops.add_rms_norm(x, w, residual=x, kind="fp8_block", normed=False)
    assert total.shape == codes.shape == x.shape and out.shape == (0,) and out.dtype == BF16
    assert scales.shape == (7, 2)
    total, out, codes, scales = ops.add_rms_norm(x, w, residual=x, normed=False)
    assert total.shape == x.shape and out.shape == codes.shape == scales.shape == (0,)
    assert ops.add_rms_norm(x, w, normed=True)[1].shape == x.shape


def test_no_output_is_refused():
    with pytest.raises(ValueError, match="no output"):
        ops.add_rms_norm(meta(7, 256), meta(256), normed=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, torch.float16])
@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("kind", ["", "fp8_token", "int8_token", "fp8_block"])
def test_the_other_outputs_are_the_same_bits(kind, T, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(T)
    x, r = (torch.randn(T, 1280, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = (1 + 0.1 * torch.randn(1280, generator=g, device="cuda")).to(dtype)
    want = ops.add_rms_norm(x, w, residual=r, kind=kind)
    got = ops.add_rms_norm(x, w, residual=r, kind=kind, normed=False)
    assert got[1].numel() == 0
    for i in (0, 2, 3):
        assert got[i].dtype == want[i].dtype and torch.equal(got[i].view(torch.uint8), want[i].view(torch.uint8))


@pytest.mark.gpu
def test_opcheck_without_the_16_bit_rows():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x, w = torch.randn(5, 256, device="cuda").to(BF16), torch.ones(256, device="cuda").to(BF16)
    for kind in ("", "fp8_token", "int8_token", "fp8_block"):
        torch.library.opcheck(ops.add_rms_norm.default, (x, w), dict(residual=x.clone(), kind=kind, normed=False),
                              test_utils=("test_schema", "test_faketensor"))
