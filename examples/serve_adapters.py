"""One decoder layer with a sliding window, serving requests that each bring a
low-rank adapter of their own: a few decode steps in a row.

    stream + norm -> FP8 codes and 16-bit rows       add_rms_norm
    QKV product of the codes                         scaled_linear (fp8_dynamic)
    adapters of q, k and v, in one call              lora_add
    norms, rotation, paged append                    kv_append
    attention within the window                      window_attention
    output product, its adapters                     scaled_linear, lora_add
    sum with the stream, norm -> block FP8 codes     add_rms_norm
    feed-forward products, sum with the stream       scaled_linear (block_fp8, bf16)

Weights are random; --check compares every step with a plain computation.

    python examples/serve_adapters.py [--requests 6] [--context 900] [--window 256] [--steps 3] [--check]
"""
import argparse
import math
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import epilogue_scaled_gemm_amd as lg  # noqa: E402
import epilogue_scaled_gemm_amd.torch_ops  # noqa: E402,F401

ops = torch.ops.lingemm
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class Layer:
    def __init__(self, hidden, heads, kv_heads, dim, inner, adapters, rank, positions, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.slices = (heads * dim, kv_heads * dim, kv_heads * dim)
        w = randn(sum(self.slices), hidden) / math.sqrt(hidden)
        self.qkv_scale = w.abs().amax(1) / 448.0
        self.qkv = (w / self.qkv_scale[:, None]).to(E4M3)
        self.out = (randn(hidden, heads * dim) / math.sqrt(heads * dim)).to(BF16)
        w = randn(inner, hidden) / math.sqrt(hidden)
        blocks = w.view(inner // 128, 128, hidden // 128, 128)
        self.up_scale = blocks.abs().amax((1, 3)) / 448.0
        self.up = (blocks / self.up_scale[:, None, :, None]).view(inner, hidden).to(E4M3)
        self.up_scale = self.up_scale.contiguous()
        self.down = (randn(hidden, inner) / math.sqrt(inner)).to(BF16)
        self.norms = [(1 + 0.1 * randn(hidden)).to(BF16) for _ in range(2)]
        self.k_weight, self.q_weight = [(1 + 0.1 * randn(dim)).to(BF16) for _ in range(2)]
        self.table = lg.rope_table(positions, dim)
        self.qkv_a = (randn(adapters, 3 * rank, hidden) / math.sqrt(hidden)).to(BF16)
        self.qkv_b = (0.1 * randn(adapters, sum(self.slices), rank)).to(BF16)
        self.out_a = (randn(adapters, rank, heads * dim) / math.sqrt(heads * dim)).to(BF16)
        self.out_b = (0.1 * randn(adapters, hidden, rank)).to(BF16)
        self.factors = 0.5 + torch.rand(adapters, generator=g, device="cuda")


class Requests:
    """Lengths, pages and adapters of the running requests; the cache."""

    def __init__(self, count, context, steps, layer, adapters, page, hidden, seed=0):
        rng = random.Random(seed)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        lengths = [max(0, context - 41 * b) for b in range(count)]
        pages = [(n + steps + page - 1) // page for n in lengths]
        order = list(range(sum(pages)))
        rng.shuffle(order)
        table = torch.zeros(count, max(pages), dtype=torch.int32)
        for b, n in enumerate(pages):
            table[b, :n] = torch.tensor(order[sum(pages[:b]):sum(pages[:b + 1])])
        i32 = dict(dtype=torch.int32, device="cuda")
        self.page, self.table, self.max_context = page, table.cuda(), max(lengths) + steps
        self.context = torch.tensor(lengths, **i32)
        self.offsets = torch.arange(count + 1, **i32)
        # every fourth request has no adapter; others share them
        self.ids = torch.tensor([-1 if b % 4 == 3 else rng.randrange(adapters) for b in range(count)], **i32)
        shape = (sum(pages), layer.kv_heads, page, layer.dim)
        self.k_cache, self.v_cache = (torch.randn(shape, generator=g, device="cuda").to(BF16) for _ in range(2))
        self.stream = torch.randn(count, hidden, generator=g, device="cuda").to(BF16)


def step(L, r, window, sinks):
    """One token of every request; what each operator got and gave, by name."""
    T, D = r.stream.shape[0], L.dim
    nq, nk, _ = L.slices
    _, x, codes, scales = ops.add_rms_norm(r.stream, L.norms[0], kind="fp8_token")
    plain = ops.scaled_linear(codes, L.qkv, scale_a=scales, scale_b=L.qkv_scale, quant="fp8_dynamic")
    qkv = ops.lora_add(x, L.qkv_a, L.qkv_b, r.ids, base=plain, factors=L.factors, slices=L.slices)
    q = qkv[:, :nq].view(T, L.heads, D)
    k = qkv[:, nq:nq + nk].view(T, L.kv_heads, D)
    v = qkv[:, nq + nk:].view(T, L.kv_heads, D)
    slots = lg.node_slots(r.table, r.context, r.offsets, r.page)
    turned = ops.kv_append(k, v, r.k_cache, r.v_cache, slots, cos_sin=L.table, positions=r.context,
                           k_weight=L.k_weight, q=q, q_weight=L.q_weight)
    seen, lse = ops.window_attention(turned, r.k_cache, r.v_cache, r.table, r.context, r.offsets,
                                     r.max_context, 1, window, sinks)
    shared = ops.scaled_linear(seen.view(T, nq), L.out)
    y = ops.lora_add(seen.view(T, nq), L.out_a, L.out_b, r.ids, base=shared, factors=L.factors)
    total, _, codes2, scales2 = ops.add_rms_norm(y, L.norms[1], residual=r.stream, kind="fp8_block", normed=False)
    up = ops.scaled_linear(codes2, L.up, scale_a=scales2, scale_b=L.up_scale, quant="block_fp8", act="silu")
    out = ops.scaled_linear(up, L.down, residual=total)
    return dict(stream=r.stream, x=x, codes=codes, scales=scales, plain=plain, qkv=qkv, turned=turned, seen=seen,
                lse=lse, shared=shared, y=y, total=total, codes2=codes2, scales2=scales2, out=out)


def check(L, r, got, window, sinks):
    """The new operators' results against plain computations of their own inputs, in 64
    bits; the largest error over its allowed size of each."""
    bf, worst = 2.0 ** -8, {}  # half a step of bfloat16

    def near(name, have, want, tol):
        worst[name] = float(((have.double() - want).abs() / tol).max())

    def normed(s, w):
        s = s.double()
        return s / (s.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()

    want = normed(got["stream"], L.norms[0])
    near("x", got["x"], want, bf * want.abs() * 1.02 + 1e-6)
    have = got["codes"].float() * got["scales"][:, None]  # e4m3: half a step of 3 bits
    near("codes", have, want, 2.0 ** -4 * want.abs() * 1.02 + 2.0 ** -9 * got["scales"][:, None].double())
    s = got["y"].double() + got["stream"].double()
    near("total", got["total"], s, bf * s.abs() * 1.02 + 1e-6)
    want = normed(s, L.norms[1])
    wide = got["scales2"].repeat_interleave(128, 1)
    near("codes2", got["codes2"].float() * wide, want,
         2.0 ** -4 * want.abs() * 1.02 + 2.0 ** -9 * wide.double())

    def adapted(x, a, b, base, widths):
        want, size = base.double(), base.double().abs()
        R = b.shape[2]
        for t, i in enumerate(r.ids.tolist()):
            if i < 0:
                continue
            h, at = a[i].double() @ x[t].double(), 0
            for j, w in enumerate(widths):
                p, m = h[j * R:(j + 1) * R], b[i, at:at + w].double()
                want[t, at:at + w] += L.factors[i].double() * (m @ p)
                size[t, at:at + w] += L.factors[i].double() * (m.abs() @ p.abs())
                at += w
        return want, bf * want.abs() * 1.02 + 2.0 ** -14 * size

    near("qkv", got["qkv"], *adapted(got["x"], L.qkv_a, L.qkv_b, got["plain"], L.slices))
    T, D = got["seen"].shape[0], L.dim
    near("y", got["y"], *adapted(got["seen"].view(T, -1), L.out_a, L.out_b, got["shared"], (got["y"].shape[1],)))
    want = torch.zeros_like(got["seen"], dtype=torch.float64)
    tol = torch.zeros_like(want)
    G = L.heads // L.kv_heads
    for t, n in enumerate(r.context.tolist()):
        at = torch.tensor([c for c in range(n + 1) if c < sinks or c > n - window], device="cuda")
        page = r.table[t].long()[at // r.page]
        for h in range(L.kv_heads):
            k, v = r.k_cache[page, h, at % r.page].double(), r.v_cache[page, h, at % r.page].double()
            w = torch.softmax(got["turned"][t, h * G:(h + 1) * G].double() @ k.t().contiguous() / math.sqrt(D), 1)
            want[t, h * G:(h + 1) * G] = w @ v
            tol[t, h * G:(h + 1) * G] = bf * (w @ v).abs() * 1.02 + (bf + 1e-4) * (w @ v.abs())
    near("seen", got["seen"], want, tol)
    return worst


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--context", type=int, default=900)
    ap.add_argument("--window", type=int, default=256)
    ap.add_argument("--sinks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--adapters", type=int, default=3)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=4)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--page", type=int, default=16)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    worst = {}
    with torch.no_grad():
        layer = Layer(a.hidden, a.heads, a.kv_heads, a.dim, a.inner, a.adapters, a.rank, a.context + a.steps + 1)
        r = Requests(a.requests, a.context, a.steps, layer, a.adapters, a.page, a.hidden)
        for i in range(a.steps):
            got = step(layer, r, a.window, a.sinks)
            torch.cuda.synchronize()
            print(f"step {i}: contexts {r.context.tolist()}, rms of the stream "
                  f"{float(got['out'].float().square().mean().sqrt()):.4f}")
            if a.check:
                for k, v in check(layer, r, got, a.window, a.sinks).items():
                    worst[k] = max(worst.get(k, 0.0), v)
            r.stream, r.context = got["out"], r.context + 1
    if a.check:
        print("error over its allowed size:", {k: round(v, 3) for k, v in worst.items()})
        return 0 if all(v <= 1 for v in worst.values()) else 1
    return 0


if __name__ == "__main__":
    sys.exit(main())
