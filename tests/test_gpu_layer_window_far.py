"""window_attention of sequences whose context has passed 2^30 positions: what the page table
holds of them is seen or not by the same comparison as nearer ones."""
import pytest
import torch

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


FURTHEST = 2 ** 31 - 2 ** 23 - 1000


@pytest.mark.parametrize("far", [2 ** 30 - 3, 2 ** 30, 2 ** 30 + 1000, FURTHEST])
@pytest.mark.parametrize("low", [-700, 0, 1, 101, 330])  # where the window of the first node begins
@pytest.mark.parametrize("cnt", [3, 90])
@pytest.mark.parametrize("D,dtype,cache,tree", [(128, BF16, BF16, False), (64, FP16, E4M3, False),
                                                (128, FP16, FP16, True), (256, BF16, BF16, True)])
def test_far_contexts(handle, far, low, cnt, D, dtype, cache, tree):
    # the same visible positions of a table of 320: of a context of 1000 and of one further on
    near = 1000
    c = Case([near], [cnt], near - low + 1, 2, D=D, dtype=dtype, cache=cache, tree=tree)
    c.table = c.table[:, :320 // c.page].contiguous()
    want, window = c.run(handle), c.window
    c.check(want, reach=320)
    on = c.on_gpu()
    c.window = window + far - near
    c.context = torch.tensor([far], dtype=torch.int32)
    if tree:
        c.positions = c.positions + (far - near)
    c.on_gpu = lambda: {**on, **{n: None if getattr(c, n) is None else getattr(c, n).cuda()
                                 for n in ("context", "positions")}}
    c.max_context = far
    got = c.run(handle)
    # (another cut of the positions adds in another order)
    c.window, c.context = window, torch.tensor([near], dtype=torch.int32)
    if tree:
        c.positions = c.positions - (far - near)
    c.check(got, reach=320)


@pytest.mark.parametrize("cnt", [1, 70])
def test_windows_wider_than_every_context(handle, cnt):
    c = Case([1000], [cnt], 2000, 0)
    c.table = c.table[:, :320 // c.page].contiguous()
    want = c.run(handle)
    c.context = torch.tensor([FURTHEST], dtype=torch.int32)
    for window in (2 ** 31 - 2 ** 23, 2 ** 31 - 1, 2 ** 31, 2 ** 62):
        c.window = window
        got = c.run(handle)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
