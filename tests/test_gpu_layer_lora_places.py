"""A row of lora_add gives the same bits wherever it stands in a call of the same size, and whoever
shares its adapter or its window of 64 rows."""
import random

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


SIZES = [  # rows, inner, width, rank, adapters: one launch, then two; rows aligned and not
    (16, 520, 256, 16, 4), (48, 1024, 256, 16, 6), (64, 584, 331, 24, 10), (64, 1024, 256, 32, 64),
    (64, 1000, 256, 64, 6), (200, 2048, 384, 16, 5), (333, 584, 201, 40, 9), (4200, 256, 128, 128, 12)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,K,N,R,n", SIZES)
def test_rows_in_another_order(handle, dtype, T, K, N, R, n):
    c = Case(T, K, N, R, n, dtype)
    first = c.run(handle)
    c.check(first)
    for seed in range(3):
        order = list(range(T))
        random.Random(seed).shuffle(order)
        order = torch.tensor(order)
        moved = Case(T, K, N, R, n, dtype)
        moved.x, moved.base, moved.ids = c.x[order], c.base[order], c.ids[order]
        assert torch.equal(moved.run(handle), first[order])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,K,N,R,n", SIZES)
def test_a_row_among_few_and_among_many_of_its_adapter(handle, dtype, T, K, N, R, n):
    # the adapter's rows of the window: one, up to 16, up to 32 and all of it
    c = Case(T, K, N, R, n, dtype)
    row, want = T // 2, None
    for among in (0, 10, 25, T):
        c.ids = torch.tensor([(t % (n - 1)) if abs(t - row) > among else n - 1 for t in range(T)], dtype=torch.int32)
        got = c.run(handle)
        c.check(got)
        assert want is None or torch.equal(got[row], want)
        want = got[row]
