"""The serving operators as they are used: through the dispatcher, on streams,
in graphs, and together in the draft-verification example."""
import importlib.util
import os

import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
import epilogue_scaled_gemm_amd.torch_ops  # noqa: E402,F401

pytestmark = pytest.mark.gpu

ops = torch.ops.lingemm
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("verify_drafts",
                                              os.path.join(ROOT, "examples", "verify_drafts.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(sequences=3, context=200, nodes=9, hidden=512, heads=8, kv_heads=2, dim=64, vocab=1000,
         page=16, cache8=False, seed=0):
    d = example.Drafts(sequences, context, nodes, page, vocab, seed)
    return example.Layer(hidden, heads, kv_heads, dim, vocab, d.pages, page, cache8, seed), d


@pytest.mark.parametrize("kw", [dict(), dict(cache8=True, dim=128), dict(sequences=1, nodes=1),
                                dict(context=3000, nodes=40, seed=3), dict(vocab=999, page=64)])
def test_the_example_step_by_step(kw):
    print(f"[example] {kw}", flush=True)
    layer, d = make(**kw)
    with torch.no_grad():
        got = example.verify(layer, d)
        worst = example.check(layer, d, got)
    assert all(v <= 1 for v in worst.values()), worst
    paths = example.accept(d, got)
    assert [p[0] for p in paths] == [0] * len(d.parents)


def test_opcheck():
    layer, d = make()
    T = d.tokens.shape[0]
    q = torch.randn(T, 8, 64, device="cuda").bfloat16()
    k = torch.randn(T, 2, 64, device="cuda").bfloat16()
    utils = ("test_schema", "test_faketensor")
    torch.library.opcheck(ops.qk_norm_rope.default, (q, k),
                          dict(cos_sin=layer.table, positions=d.positions,
                               q_weight=layer.q_weight), test_utils=utils)
    torch.library.opcheck(ops.kv_append.default,
                          (k, k.clone(), layer.k_cache, layer.v_cache, d.slots),
                          dict(cos_sin=layer.table, positions=d.positions, q=q), test_utils=utils)
    torch.library.opcheck(ops.tree_attention.default,
                          (q, layer.k_cache, layer.v_cache, d.table, d.context, d.offsets,
                           d.max_context, d.max_nodes), dict(mask=d.mask), test_utils=utils)
    torch.library.opcheck(ops.token_logprobs.default,
                          (torch.randn(T, 1000, device="cuda"), d.tokens), dict(top=3),
                          test_utils=utils)


def test_no_gradient():
    q = torch.randn(2, 2, 64, device="cuda").bfloat16().requires_grad_()
    k = torch.randn(2, 1, 64, device="cuda").bfloat16()
    a, _ = ops.qk_norm_rope(q, k)
    with pytest.raises(RuntimeError):
        a.float().sum().backward()
    with pytest.raises(RuntimeError, match="forward only"):
        lg.Handle().qk_norm_rope(q, k, torch.empty_like(q), torch.empty_like(k))


@pytest.mark.parametrize("kw", [dict(), dict(context=5000, nodes=3, sequences=1, vocab=30001)])
def test_graph_replays_match_eager(kw):
    # The second shape splits its context and its rows over workgroups: run
    # once eagerly on the capture stream, so that the workspace is there.
    layer, d = make(**kw)
    with torch.no_grad():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            example.verify(layer, d)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                captured = example.verify(layer, d)
        gen = torch.Generator(device="cuda").manual_seed(1)
        for rep in range(5):
            d.tokens.copy_(torch.randint(0, 900, d.tokens.shape, generator=gen, device="cuda",
                                         dtype=torch.int32))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            eager = example.verify(layer, d)
            torch.cuda.synchronize()
            for name in ("q_rot", "attended", "lse", "logprobs", "entropy", "top_ids", "top_logprobs"):
                assert torch.equal(captured[name], eager[name]), f"replay {rep}: {name}"


def test_two_streams_at_once():
    # each stream has its handle, so splits in flight share no workspace
    cases = [make(context=4000, nodes=2, sequences=1, seed=s) for s in (1, 2)]
    with torch.no_grad():
        want = [example.verify(*c) for c in cases]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in cases]
        for _ in range(5):
            got = []
            for c, s in zip(cases, streams):
                with torch.cuda.stream(s):
                    got.append(example.verify(*c))
            torch.cuda.synchronize()
            for w, g in zip(want, got):
                for name in ("attended", "lse", "logprobs", "top_ids"):
                    assert torch.equal(w[name], g[name]), name


def test_workspaces_shared_with_the_layers():
    # one handle: split attention, split scoring and a split-K layer in turn
    # use the same workspace and counters, and keep each other's results
    h = lg.Handle()
    layer, d = make(context=5000, nodes=2, sequences=1)
    T = d.tokens.shape[0]
    q = torch.randn(T, 8, 64, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(T, 8, device="cuda")
    logits = torch.randn(2, 60001, device="cuda")
    lp, ids = torch.empty(2, device="cuda"), torch.empty(2, 4, dtype=torch.int32, device="cuda")
    A = torch.randn(4, 2048, device="cuda").bfloat16()
    B = torch.randn(512, 2048, device="cuda").bfloat16()
    C = torch.empty(4, 512, dtype=torch.bfloat16, device="cuda")
    h.set_force("decode swap=1 split=4 reduce=lastwg waves=8 unroll=2 rows=16")
    seen = []
    for _ in range(4):
        h.tree_attention(q, layer.k_cache, layer.v_cache, out, d.table, d.context, d.offsets,
                         max_context=d.max_context, max_nodes=d.max_nodes, mask=d.mask, lse=lse)
        h.run(A, B, C)
        h.token_logprobs(logits, d.tokens[:2], lp, top_ids=ids)
        torch.cuda.synchronize()
        seen.append([t.clone() for t in (out, lse, C, lp, ids)])
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))
    h.close()
