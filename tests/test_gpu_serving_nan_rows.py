"""Token log probabilities of rows that hold NaN: no probability is a number,
and every index of `top_ids` can still be used as one."""
import math

import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    yield h
    h.close()


def run(h, x, top):
    T = x.shape[0]
    lp, en = torch.full((T,), 77.0, device="cuda"), torch.full((T,), 77.0, device="cuda")
    ids = torch.full((T, top), -7, dtype=torch.int32, device="cuda")
    tl = torch.full((T, top), 77.0, device="cuda")
    h.token_logprobs(x.cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"), lp, entropy=en,
                     top_ids=ids, top_logprobs=tl)
    torch.cuda.synchronize()
    return lp.cpu(), en.cpu(), ids.cpu(), tl.cpu()


# One slice of one batch, of several batches (enough rows for the device), and
# several slices; a vocabulary of less than a vector.
@pytest.mark.parametrize("T,V", [(4, 7), (4, 40), (300, 3005), (300, 40009), (4, 40009), (1, 131072)])
@pytest.mark.parametrize("kind", ["all", "few left", "half", "whole batches", "ends"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_indices_stay_in_range(handle, dtype, kind, T, V):
    top = min(V, 20)
    print(f"[score NaN] {dtype} {kind} T={T} V={V} top={top}", flush=True)
    g = torch.Generator().manual_seed(V + T)
    x = torch.randn(T, V, generator=g)
    clean = x.to(dtype)
    bad = torch.zeros(V, dtype=torch.bool)
    if kind == "all":
        bad[:] = True
    elif kind == "few left":               # fewer numbers than places
        bad[:] = True
        bad[torch.randperm(V, generator=g)[:min(3, V - 1)]] = False
    elif kind == "half":
        bad[torch.randperm(V, generator=g)[:(V + 1) // 2]] = True
    elif kind == "whole batches":
        bad[: max(1, V // 3)] = True
    else:
        bad[:3] = True
        bad[V - 3:] = True
    rows = range(0, T, 2) if T > 1 else [0]
    for t in rows:
        x[t, bad] = math.nan
    lp, en, ids, tl = run(handle, x.to(dtype), top)
    assert ((ids >= 0) & (ids < V)).all(), (int(ids.min()), int(ids.max()))
    assert lp[::2].isnan().all() and en[::2].isnan().all() and tl[::2].isnan().all()
    if T > 1:                               # the rows between them are what they were
        want = run(handle, clean, top)
        for got, w in zip((lp, en, ids, tl), want):
            assert torch.equal(got[1::2], w[1::2])
