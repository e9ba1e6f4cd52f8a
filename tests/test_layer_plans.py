"""How adapter calls are cut, without a GPU: one launch for few rows and up to two rounds of
workgroups on 256 CUs, two launches beyond."""
import os

import pytest
import torch

from test_layer_host import LORA, LORA_OK

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
from epilogue_scaled_gemm_amd import serving  # noqa: E402


@pytest.fixture()
def handle():
    if torch.cuda.is_available():
        pytest.skip("fake-pointer error paths run on the CPU only")
    if not os.path.exists(lg.LIB_PATH):
        pytest.skip("library not built")
    h = lg.Handle()
    yield h
    h.close()


def launches(h, rows, adapters, width, rank=16):
    # without a device two launches fail where they grow the workspace, one where it launches
    d = dict(LORA_OK, rows=rows, adapters=adapters, inner=4096, x_s=4096, width=width, w0=width, base_s=width,
             out_s=width, rank=rank)
    assert lg.library().lin_gemm_lora_add(h._h, serving._LORA.pack(*[d.get(n, 0) for n in LORA]), None) != 0
    return 1 if b"adapter launch" in lg.library().lin_gemm_last_error(h._h) else 2


@pytest.mark.parametrize("rows,adapters,width,count", [
    (1, 8, 6144, 1), (48, 24, 4096, 1), (64, 64, 4096, 1),  # 64 x 8 workgroups
    (42, 64, 6144, 1), (43, 64, 6144, 2), (44, 64, 6144, 2),  # 42, 43 and 44 x 12
    (57, 64, 4099, 2), (56, 64, 4099, 1),                     # 57 and 56 x 9
    (65, 64, 64, 2), (64, 7, 4096, 2), (16, 1, 4096, 1)])
def test_one_launch_or_two(handle, rows, adapters, width, count):
    assert launches(handle, rows, adapters, width) == count


def test_high_ranks_take_two_launches(handle):
    assert launches(handle, 1, 8, 4096, rank=32) == 1 and launches(handle, 1, 8, 4096, rank=40) == 2
