"""Log probabilities, entropy and top tokens on the GPU against 64 bits."""
import math

import pytest
import torch

import serving_ref as ref

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


def run(h, logits, tokens, top, temperature=1.0):
    T = logits.shape[0]
    lp = torch.full((T,), 77.0, device="cuda")
    en = torch.full((T,), 77.0, device="cuda")
    ids = torch.full((T, top), -7, dtype=torch.int32, device="cuda") if top else None
    tl = torch.full((T, top), 77.0, device="cuda") if top else None
    h.token_logprobs(logits, tokens.cuda(), lp, entropy=en, top_ids=ids, top_logprobs=tl,
                     temperature=temperature)
    torch.cuda.synchronize()
    return lp.cpu().double(), en.cpu().double(), None if ids is None else ids.cpu().long(), \
        None if tl is None else tl.cpu().double()


def check(h, logits, tokens, top, temperature=1.0):
    lp, en, ids, tl = run(h, logits, tokens, top, temperature)
    wlp, wen, wids, wtl, bound = ref.score(logits.cpu(), tokens, top, temperature)
    size = 1 + wlp.nan_to_num(0.0, neginf=0.0).abs()
    same = (lp == wlp) | (lp.isnan() & wlp.isnan())
    assert (same | ((lp - wlp).abs() <= bound * size)).all(), (lp - wlp).abs().max()
    assert ((en - wen).abs() <= 4 * bound * (1 + math.log(logits.shape[1]))).all(), (en - wen).abs().max()
    if top:
        assert torch.equal(ids, wids), (ids, wids)
        same = tl == wtl
        assert (same | ((tl - wtl).abs() <= bound * (1 + wtl.nan_to_num(0.0, neginf=0.0).abs()))).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,top", [(1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 7, 5), (5, 33, 32), (1, 64, 8),
                                     (4, 1000, 20), (7, 4095, 32), (1, 32003, 5), (3, 50257, 20),
                                     (48, 9001, 20), (600, 3001, 3), (520, 40, 32), (2, 131072, 0)])
def test_scores(handle, dtype, T, V, top):
    print(f"[score] {dtype} T={T} V={V} top={top}", flush=True)
    g = torch.Generator().manual_seed(T * 7 + V)
    x = (3 * torch.randn(T, V, generator=g)).to(dtype).cuda()
    tok = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    check(handle, x, tok, top, 0.7 if V % 2 else 1.3)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_lower_index(handle, dtype):
    for V in (40, 3001, 70001):
        g = torch.Generator().manual_seed(V)
        x = torch.randint(-2, 3, (3, V), generator=g).to(dtype)
        x[1] = 1.5                      # all equal
        x[2, ::2] = 0.0
        x[2, 1::2] = -0.0               # one value
        check(handle, x.cuda(), torch.zeros(3, dtype=torch.int32), 32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_orders_that_fill_the_list(handle, dtype):
    V = 20011
    x = torch.linspace(-30, 30, V).repeat(2, 1)
    x[1] = x[1].flip(0)
    check(handle, x.to(dtype).cuda(), torch.tensor([0, V - 1], dtype=torch.int32), 32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_vocabularies(handle, dtype):
    V = 5003
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, V, generator=g)
    low = torch.finfo(dtype).min
    x[0, 100:] = -math.inf
    x[1, torch.randperm(V, generator=g)[:V - 3]] = -math.inf
    x[2, 10:] = low
    x[3] = low                           # all of the lowest value: uniform
    x = x.to(dtype)
    tok = torch.tensor([3, int(x[1].argmax()), 12, 4], dtype=torch.int32)
    check(handle, x.cuda(), tok, 20)
    tok = torch.tensor([200, int(x[1].argmin()), 2, V - 1], dtype=torch.int32)
    check(handle, x.cuda(), tok, 20)     # a masked token: -inf


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 600])
def test_rows_without_a_distribution(handle, dtype, T):
    V = 3005
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, V, generator=g).to(dtype)
    ok = x.clone()
    kinds = [-math.inf, math.inf, math.nan]
    for i, k in enumerate(kinds[:T] if T < 3 else kinds):
        x[i, :] = k if k == -math.inf else x[i]
        x[i, V // 2] = k
    tok = torch.zeros(T, dtype=torch.int32)
    lp, en, ids, tl = run(handle, x.cuda(), tok, 4)
    n = min(T, 3)
    assert lp[:n].isnan().all() and en[:n].isnan().all() and tl[:n].isnan().all()
    assert ((ids >= 0) & (ids < V)).all()
    if T > 3:                            # the rows beside them
        check(handle, ok.cuda(), tok, 4)
        assert torch.equal(lp[3:], run(handle, ok.cuda(), tok, 4)[0][3:])


def test_tokens_outside_the_vocabulary(handle):
    x = torch.randn(4, 100).cuda()
    lp = run(handle, x, torch.tensor([-1, 100, 5, 2 ** 31 - 1], dtype=torch.int32), 1)[0]
    assert lp.isnan().tolist() == [True, True, False, True]


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_apart_and_unaligned(handle, dtype):
    g = torch.Generator().manual_seed(11)
    wide = torch.randn(9, 2111, generator=g).to(dtype).cuda()
    tok = torch.randint(0, 700, (9,), generator=g, dtype=torch.int32)
    for at in (0, 1, 3, 5, 7):
        check(handle, wide[:, at:at + 703], tok, 7)
    flat = wide.reshape(-1)
    for V in (5, 8, 13):                 # less than one whole vector
        check(handle, flat[1:1 + 4 * V].view(4, V), tok[:4] % V, min(V, 5))


def test_large_magnitudes(handle):
    x = torch.tensor([[3e38, -3e38, 0.0, 3e38], [1e4, 1e4 + 0.5, -1e4, 1e4 - 1]]).cuda()
    lp, en, ids, _ = run(handle, x, torch.tensor([0, 1], dtype=torch.int32), 2)
    assert abs(float(lp[0]) + math.log(2)) < 1e-6 and abs(float(en[0]) - math.log(2)) < 1e-6
    assert ids.tolist() == [[0, 3], [1, 0]]
    want = torch.log_softmax(x[1].cpu().double(), 0)[1]
    assert abs(float(lp[1] - want)) < 1e-5


def test_repeats_are_equal(handle):
    x = torch.randn(5, 60001).bfloat16().cuda()
    tok = torch.arange(5, dtype=torch.int32)
    a, b = run(handle, x, tok, 20), run(handle, x, tok, 20)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
