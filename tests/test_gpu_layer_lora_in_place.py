"""lora_add in place of its base, in one launch and in two, with rows that are 16-byte aligned or not."""
import pytest
import torch

from test_gpu_layer_lora import BF16, FP16, Case

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("widths", [(328,), (331,), (256, 64, 72), (257, 64, 9)])
@pytest.mark.parametrize("T,R", [(1, 16), (40, 8), (40, 24), (64, 32), (40, 64), (300, 16), (300, 72), (4200, 16)])
def test_in_place(handle, dtype, widths, T, R):
    c = Case(T, 200, sum(widths), R, 10, dtype, widths=widths)
    c.check(c.run(handle, in_place=True))
    assert torch.equal(c.run(handle, in_place=True), c.run(handle))


@pytest.mark.parametrize("T", [30, 300])
@pytest.mark.parametrize("N,gap", [(328, 8), (331, 2), (328, 5)])
def test_in_place_between_other_columns(handle, T, N, gap):
    c = Case(T, 200, N, 24, 10)
    d = c.on_gpu()
    wide = torch.full((T, N + 2 * gap), 3.0, dtype=BF16, device="cuda")
    rows = wide[:, gap:gap + N]
    rows.copy_(d["base"])
    handle.lora_add(d["x"], d["a"], d["b"], d["ids"], rows, base=rows, factors=d["factors"])
    c.check(rows.cpu())
    assert (wide[:, :gap] == 3).all() and (wide[:, gap + N:] == 3).all()
