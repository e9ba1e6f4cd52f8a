"""The memory that attention calls keep for joining splits is bounded."""
import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,ctx,Hq", [(2100, 5000, 32), (4100, 8200, 64)])
def test_workspace_of_prompt_parts(n, ctx, Hq):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Hk, D, page = 8, 128, 64
    pages = (ctx + n + page - 1) // page
    g = torch.Generator(device="cuda").manual_seed(n)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    k, v, q = randn(pages, Hk, page, D), randn(pages, Hk, page, D), randn(n, Hq, D)
    out, lse = torch.empty_like(q), torch.empty(n, Hq, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    context = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    h = lg.Handle()
    run = lambda q, out, lse, offsets: h.tree_attention(  # noqa: E731
        q, k, v, out, table, context, offsets, max_context=ctx, max_nodes=q.shape[0], lse=lse)
    run(q[:1], out[:1], lse[:1], torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    run(q, out, lse, offsets)
    torch.cuda.synchronize()
    grown = free - torch.cuda.mem_get_info()[0]
    assert grown <= (1 << 27) + (1 << 22), f"{grown >> 20} MB"  # (and a page of the allocator's)
    # a few rows, in 64 bits
    for t in (0, 1, n // 2, n - 1):
        for head in (0, Hq - 1):
            kk = k[:, head * Hk // Hq].reshape(-1, D)[:ctx + t + 1].double()
            vv = v[:, head * Hk // Hq].reshape(-1, D)[:ctx + t + 1].double()
            z = kk @ q[t, head].double() / D ** 0.5
            p = torch.softmax(z, 0)
            want, size = p @ vv, p @ vv.abs()
            # weights and results are rounded to bfloat16
            assert ((out[t, head].double() - want).abs() <= 2.0 ** -8 * (want.abs() + 1.01 * size)).all()
            assert abs(float(lse[t, head] - torch.logsumexp(z, 0))) < 1e-4
    h.close()
