"""window_attention where a row's window ends beyond what the page table holds, or nothing is left of it."""
import pytest
import torch

import layer_ref as ref
from test_gpu_layer_window import BF16, E4M3, FP16, Case

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


# Tables of whole blocks (32 positions of few rows, 64 to 128 of many) that end before the windows of
# all rows, or of the later rows, begin.  Outputs hold something else before the call.
@pytest.mark.parametrize("ctx,cnt,window,reach", [
    (500, 2, 100, 320), (500, 60, 100, 384), (250, 200, 30, 384), (3000, 1, 1000, 1280), (3000, 60, 1000, 1280),
    (3000, 300, 1000, 1280), (1200, 300, 64, 1280), (5000, 9, 1, 4096)])
@pytest.mark.parametrize("D,dtype,cache", [(128, BF16, BF16), (128, FP16, E4M3), (64, BF16, BF16), (256, FP16, FP16)])
@pytest.mark.parametrize("sinks", [0, 3])
def test_windows_that_begin_past_the_table(handle, ctx, cnt, window, reach, D, dtype, cache, sinks):
    c = Case([ctx], [cnt], window, sinks, D=D, dtype=dtype, cache=cache)
    c.table = c.table[:, :reach // c.page].contiguous()
    got = c.run(handle)
    c.check(got, reach=reach)
    if sinks == 0 and ctx - window + 1 >= reach:
        assert (got[0] == 0).all() and (got[1] == -float("inf")).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cnt", [4, 130])
def test_trees_past_the_table_beside_one_within_it(handle, D, cnt):
    c = Case([3000, 600], [cnt, cnt], 500, 0, D=D, tree=True)
    c.table = c.table[:, :1024 // c.page].contiguous()
    got = c.run(handle)
    c.check(got, reach=1024)
    assert (got[0][:cnt] == 0).all() and (got[1][:cnt] == -float("inf")).all()
