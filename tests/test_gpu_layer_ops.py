"""The norm with codes, the adapters and the windowed attention as they are
used: together in a layer's decode steps, through the dispatcher, on
streams and in graphs."""
import importlib.util
import os

import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
import epilogue_scaled_gemm_amd.torch_ops  # noqa: E402,F401

pytestmark = pytest.mark.gpu

ops = torch.ops.lingemm
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("serve_adapters", os.path.join(ROOT, "examples", "serve_adapters.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("args", [
    [], ["--requests", "1", "--context", "0", "--steps", "4"],
    ["--requests", "40", "--context", "3000", "--window", "1000", "--sinks", "0", "--rank", "8", "--adapters", "9"],
    ["--requests", "70", "--context", "100", "--dim", "64", "--heads", "12", "--kv-heads", "2", "--rank", "64",
     "--page", "64", "--window", "1"]])
def test_the_example_step_by_step(args):
    print(f"[example] {args}", flush=True)
    assert example.main(args + ["--check"]) == 0


def make(requests=5, seed=0):
    layer = example.Layer(512, 8, 2, 64, 256, 3, 16, 400, seed)
    return layer, example.Requests(requests, 300, 8, layer, 3, 16, 512, seed)


def test_opcheck():
    L, r = make()
    utils = ("test_schema", "test_faketensor")
    x = r.stream
    for kind in ("", "fp8_token", "int8_token", "fp8_block"):
        torch.library.opcheck(ops.add_rms_norm.default, (x, L.norms[0]), dict(residual=x.clone(), kind=kind),
                              test_utils=utils)
    base = torch.randn(5, sum(L.slices), device="cuda").bfloat16()
    torch.library.opcheck(ops.lora_add.default, (x, L.qkv_a, L.qkv_b, r.ids),
                          dict(base=base, factors=L.factors, slices=L.slices), test_utils=utils)
    q = torch.randn(5, 8, 64, device="cuda").bfloat16()
    torch.library.opcheck(ops.window_attention.default,
                          (q, r.k_cache, r.v_cache, r.table, r.context, r.offsets, r.max_context, 1, 60, 4),
                          test_utils=utils)


def test_a_step_on_another_stream():
    L, r = make()
    with torch.no_grad():
        want = example.step(L, r, 100, 4)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = example.step(L, r, 100, 4)
        s.synchronize()
    for name in want:
        assert torch.equal(got[name].view(torch.uint8), want[name].view(torch.uint8)), name


def test_a_captured_step():
    # the layer's new operators in one graph, replayed between eager steps
    L, r = make()
    T, nq = r.stream.shape[0], L.slices[0]
    s = torch.cuda.Stream()

    def run():
        _, x, codes, scales = ops.add_rms_norm(r.stream, L.norms[0], kind="fp8_token")
        y = ops.lora_add(x, L.qkv_a, L.qkv_b, r.ids, factors=L.factors, slices=L.slices)
        q = y[:, :nq].view(T, L.heads, L.dim)
        seen, lse = ops.window_attention(q, r.k_cache, r.v_cache, r.table, r.context, r.offsets, r.max_context,
                                         1, 100, 4)
        return x, codes, scales, y, seen, lse

    with torch.no_grad():
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()  # grows the workspace of this stream's handle
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = run()
        for seed in range(4):
            g = torch.Generator(device="cuda").manual_seed(seed)
            r.stream.normal_(generator=g)
            r.context.random_(0, 300, generator=g)
            r.ids.random_(-1, 3, generator=g)
            want = run()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
