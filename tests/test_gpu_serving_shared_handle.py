"""One handle for the layers and the serving operators in any order: every
call writes its outputs anew, with the results of a handle of its own."""
import itertools

import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")

pytestmark = pytest.mark.gpu


def test_any_order_and_every_time():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    # attention: split and joined by the last workgroup (one node); by a second
    # launch (20 nodes x 4 heads)
    page, D, ctx = 16, 64, 5000
    pages = (ctx + 20 + page - 1) // page
    kc, vc = randn(pages, 2, page, D).bfloat16(), randn(pages, 2, page, D).bfloat16()
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    one, many = randn(1, 8, D).bfloat16(), randn(20, 8, D).bfloat16()
    logits, tok = randn(2, 60001), i32(7, 60000)
    A, B = randn(4, 2048).bfloat16(), randn(512, 2048).bfloat16()
    outs = dict(one=torch.empty_like(one), one_lse=torch.empty(1, 8, device="cuda"),
                many=torch.empty_like(many), many_lse=torch.empty(20, 8, device="cuda"),
                C=torch.empty(4, 512, dtype=torch.bfloat16, device="cuda"),
                lp=torch.empty(2, device="cuda"), en=torch.empty(2, device="cuda"),
                ids=torch.empty(2, 4, dtype=torch.int32, device="cuda"),
                best=torch.empty(2, 4, device="cuda"))

    def attend(h, q, out, lse):
        h.tree_attention(q, kc, vc, out, table, i32(ctx), i32(0, q.shape[0]), max_context=ctx,
                         max_nodes=q.shape[0], lse=lse)

    steps = dict(
        one=lambda h: attend(h, one, outs["one"], outs["one_lse"]),
        many=lambda h: attend(h, many, outs["many"], outs["many_lse"]),
        layer=lambda h: h.run(A, B, outs["C"]),
        score=lambda h: h.token_logprobs(logits, tok, outs["lp"], entropy=outs["en"],
                                         top_ids=outs["ids"], top_logprobs=outs["best"]))

    def clear():
        for t in outs.values():
            t.fill_(-77)

    def handle():
        h = lg.Handle()
        h.set_force("decode swap=1 split=4 reduce=lastwg waves=8 unroll=2 rows=16")
        return h

    want = {}
    for name, step in steps.items():
        clear()
        with handle() as h:
            step(h)
            torch.cuda.synchronize()
        want.update({k: t.clone() for k, t in outs.items() if not (t == -77).all()})
    assert set(want) == set(outs)
    # a plain reference for what a mistake made alike every time would pass
    z = torch.log_softmax(logits.cpu().double(), -1)
    assert (want["lp"].cpu().double() - z[torch.arange(2), tok.cpu().long()]).abs().max() < 1e-4
    pos = torch.arange(ctx + 1)
    flat = lambda c: c.float().cpu().double()[table[0].cpu().long()][pos // page, :, pos % page]  # noqa: E731
    p = torch.softmax(one.float().cpu().double().view(2, 4, D) @ flat(kc).permute(1, 2, 0).contiguous() / 8, -1)
    o = (p @ flat(vc).transpose(0, 1).contiguous()).view(1, 8, D)
    assert (want["one"].float().cpu().double() - o).abs().max() < 2.0 ** -8 * 3
    # the same handle, in every order of the steps
    with handle() as h:
        for order in itertools.permutations(steps):
            clear()
            for name in order:
                steps[name](h)
            torch.cuda.synchronize()
            for k, t in outs.items():
                assert torch.equal(t, want[k]), (order, k)
