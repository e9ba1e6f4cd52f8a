"""window_attention, many rows at once: rows that see nothing beside others, and NaN codes or values in
positions that some or all rows do not see."""
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


@pytest.mark.parametrize("D,dtype,cache", [(64, BF16, BF16), (128, FP16, FP16), (128, BF16, E4M3), (256, BF16, BF16)])
@pytest.mark.parametrize("ctx,cnt,window", [(50, 60, 1), (9000, 70, 1), (9000, 200, 150), (3, 300, 200)])
def test_rows_that_see_nothing_among_many(handle, D, dtype, cache, ctx, cnt, window):
    # nodes that name nobody, so far behind the context that their windows hold nothing of it: single
    # ones, whole waves of 32 rows and whole tiles
    c = Case([ctx], [cnt], window, 0, D=D, dtype=dtype, cache=cache, tree=True)
    empty = [1, 17] + list(range(32, 64)) + list(range(128, 200))
    empty = torch.tensor([i for i in empty if i < cnt])
    c.mask[empty], c.positions[empty] = 0, ctx + cnt - 1
    got = c.run(handle)
    c.check(got)
    assert (got[0][empty] == 0).all() and (got[1][empty] == -float("inf")).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [(BF16, E4M3), (FP16, E4M3), (FP16, FP16)])
@pytest.mark.parametrize("cnt,tree", [(3, False), (130, False), (130, True)])
def test_nan_outside_the_windows(handle, D, dtype, cache, cnt, tree):
    for window, sinks in ((37, 5), (300, 70)):
        c = Case([700], [cnt], window, sinks, D=D, dtype=dtype, cache=cache, tree=tree)
        clean = c.run(handle)
        c.check(clean)
        sees = ref.window_visible(700, cnt, c.mask, 0, window, sinks, c.positions)
        bad = torch.nonzero(~sees.any(0))[:, 0]
        bad = bad[bad < 700]
        for t in (c.k_cache, c.v_cache):
            bits = t.view(torch.uint8 if cache is E4M3 else torch.int16)
            bits[c.table[0].long()[bad // 16], :, bad % 16] = 0x7F if cache is E4M3 else 0x7E01
        got = c.run(handle)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_nan_code_that_only_some_rows_see(handle, D, dtype):
    at, window, cnt = 190, 50, 100
    c = Case([200], [cnt], window, 0, D=D, dtype=dtype, cache=E4M3)
    clean = c.run(handle)
    c.v_cache.view(torch.uint8)[int(c.table[0, at // 16]), :, at % 16, 3] = 0x7F
    out, lse = c.run(handle)
    sees = ref.window_visible(200, cnt, None, 0, window, 0, None)[:, at]
    assert sees.any() and not sees.all()
    assert out[sees][:, :, 3].isnan().all() and torch.equal(lse, clean[1])
    out[:, :, 3] = torch.where(sees[:, None], clean[0][:, :, 3], out[:, :, 3])
    # two sums of the same values in other orders may round to neighbours: two half steps
    assert ((out.double() - clean[0].double()).abs() <= 2 * ref.rounding(clean[0].double(), dtype)).all()


@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16), (256, BF16)])
@pytest.mark.parametrize("cnt", [4, 90])
def test_an_infinity_that_every_row_sees(handle, D, dtype, cnt):
    # among positions that no row has masked
    at = 280
    c = Case([300], [cnt], 200, 0, D=D, dtype=dtype)
    clean = c.run(handle)
    c.check(clean)
    c.v_cache[int(c.table[0, at // 16]), :, at % 16, 3] = float("inf")
    out, lse = c.run(handle)
    assert (out[:, :, 3] == float("inf")).all() and torch.equal(lse, clean[1])
    out[:, :, 3] = clean[0][:, :, 3]
    # two sums of the same values in other orders may round to neighbours: two half steps
    assert ((out.double() - clean[0].double()).abs() <= 2 * ref.rounding(clean[0].double(), dtype)).all()
