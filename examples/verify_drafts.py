"""Verifying drafted tokens with one decoder layer, the way a server runs it.

Each sequence has a cached context and a tree of drafted tokens (node 0 the
last accepted one).  One pass scores every draft:

    QKV product (FP8, quantized on the fly)    scaled_linear_dynamic
    norms, rotation, paged append              kv_append
    attention of all trees                     tree_attention
    output product + residual                  scaled_linear
    head product                               scaled_linear
    log probabilities, entropy, top tokens     token_logprobs

and the longest path whose every token is the most likely one after its
parent is accepted.  Weights are random; --check compares every step with a
plain computation.

    python examples/verify_drafts.py [--sequences 4] [--context 1000] [--nodes 16] [--check]
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
    """Weights of the layer and the head, the rotation table, the cache."""

    def __init__(self, hidden, heads, kv_heads, dim, vocab, pages, page, cache8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        n = (heads + 2 * kv_heads) * dim
        w = randn(n, hidden) / math.sqrt(hidden)
        self.qkv_scale = w.abs().amax(1) / 448.0
        self.qkv = (w / self.qkv_scale[:, None]).to(E4M3)
        self.out = (randn(hidden, heads * dim) / math.sqrt(heads * dim)).to(BF16)
        self.head = (randn(vocab, hidden) / math.sqrt(hidden)).to(BF16)
        self.embedding = randn(vocab, hidden).to(BF16)
        self.q_weight = (1 + 0.1 * randn(dim)).to(BF16)
        self.k_weight = (1 + 0.1 * randn(dim)).to(BF16)
        self.table = lg.rope_table(pages * page, dim)  # no position is beyond the cache
        shape = (pages, kv_heads, page, dim)
        dt = E4M3 if cache8 else BF16
        self.k_cache, self.v_cache = randn(*shape).to(dt), randn(*shape).to(dt)
        self.k_scale = torch.full((kv_heads,), 0.05, device="cuda") if cache8 else None
        self.v_scale = torch.full((kv_heads,), 0.05, device="cuda") if cache8 else None


class Drafts:
    """A plan: trees, page tables and lengths of the sequences."""

    def __init__(self, sequences, context, nodes, page, vocab, seed=0):
        rng = random.Random(seed)
        self.context_list = [max(1, context - 37 * b) for b in range(sequences)]
        self.parents = [[rng.randint(max(0, i - 3), i - 1) if i else -1
                         for i in range(max(1, nodes - b % 3))] for b in range(sequences)]
        self.mask, depth = lg.tree_mask(self.parents)
        counts = [len(p) for p in self.parents]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.context = torch.tensor(self.context_list, **i32)
        self.offsets = torch.tensor([sum(counts[:b]) for b in range(sequences + 1)], **i32)
        need = [(c + n + page - 1) // page for c, n in zip(self.context_list, counts)]
        order = list(range(sum(need)))
        rng.shuffle(order)
        table = torch.zeros(sequences, max(need), dtype=torch.int32)
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[sum(need[:b]):sum(need[:b + 1])])
        self.pages, self.table = sum(need), table.cuda()
        self.max_context, self.max_nodes = max(self.context_list), max(counts)
        self.slots = lg.node_slots(self.table, self.context, self.offsets, page)
        owner = torch.repeat_interleave(torch.arange(sequences, device="cuda"),
                                        torch.tensor(counts, device="cuda"))
        self.positions = (self.context[owner] + depth).to(torch.int32)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens = torch.randint(0, vocab, (sum(counts),), generator=g, device="cuda",
                                    dtype=torch.int32)
        # the row whose distribution a node's token is drawn from: its parent's
        # (a root's token is accepted already: it looks at itself)
        flat, at = [], 0
        for p in self.parents:
            flat += [at + max(u, 0) for u in p]
            at += len(p)
        self.parent_rows = torch.tensor(flat, device="cuda")


def verify(layer, d, top=4):
    """One pass over all drafts.  Returns what each step gave, by name."""
    L = layer
    T, D = d.tokens.shape[0], L.dim
    nq, nk = L.heads * D, L.kv_heads * D
    x = L.embedding[d.tokens.long()]
    qkv = ops.scaled_linear_dynamic(x, L.qkv, L.qkv_scale)
    q = qkv[:, :nq].view(T, L.heads, D)
    k = qkv[:, nq:nq + nk].view(T, L.kv_heads, D)
    v = qkv[:, nq + nk:].view(T, L.kv_heads, D)
    q_rot = ops.kv_append(k, v, L.k_cache, L.v_cache, d.slots, cos_sin=L.table,
                          positions=d.positions, k_weight=L.k_weight, k_scale=L.k_scale,
                          v_scale=L.v_scale, q=q, q_weight=L.q_weight)
    attended, lse = ops.tree_attention(q_rot, L.k_cache, L.v_cache, d.table, d.context, d.offsets,
                                       d.max_context, d.max_nodes, mask=d.mask, k_scale=L.k_scale,
                                       v_scale=L.v_scale)
    y = ops.scaled_linear(attended.view(T, nq), L.out, residual=x)
    logits = ops.scaled_linear(y, L.head)
    # row i of `following` scores node i's token under its parent's distribution
    following = logits[d.parent_rows]
    logprobs, entropy, top_ids, top_logprobs = ops.token_logprobs(following, d.tokens, top=top)
    return dict(x=x, q=q, k=k, v=v, q_rot=q_rot, attended=attended, lse=lse, y=y, logits=logits,
                following=following, logprobs=logprobs, entropy=entropy, top_ids=top_ids,
                top_logprobs=top_logprobs)


def accept(d, got):
    """Per sequence, the longest path from the root whose tokens are all the
    most likely ones after their parents."""
    best = (got["top_ids"][:, 0] == d.tokens).tolist()
    paths, at = [], 0
    for p in d.parents:
        path = {0: [0]}
        for i in range(1, len(p)):
            if best[at + i] and p[i] in path:
                path[i] = path[p[i]] + [i]
        paths.append(max(path.values(), key=len))
        at += len(p)
    return paths


def check(layer, d, got):
    """Every operator's result against a plain computation of its own inputs,
    in 64 bits; returns the largest error over its allowed size."""
    L, D = layer, layer.dim
    worst = {}
    bf = 2.0 ** -8  # half a step of bfloat16

    def turned(x, w):
        y = x.double()
        y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
        row = L.table.double()[d.positions.long()][:, None, :]
        c, s = row[..., :D // 2], row[..., D // 2:]
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    want = turned(got["q"], L.q_weight)
    worst["q_rot"] = ((got["q_rot"].double() - want).abs() / (bf * want.abs() + 1e-5)).max()
    G = L.heads // L.kv_heads
    want, size = torch.zeros_like(got["attended"], dtype=torch.float64), None
    size = torch.zeros_like(want)
    for b, p in enumerate(d.parents):
        t0, n, c = int(d.offsets[b]), len(p), d.context_list[b]
        pages = d.table[b, :(c + n + L.page - 1) // L.page].long()
        for h in range(L.kv_heads):
            def rows(cache, scale):
                x = cache.float()[pages, h].double().reshape(-1, D)[:c + n]
                return x if scale is None else x * scale[h].double()
            k, v = rows(L.k_cache, L.k_scale), rows(L.v_cache, L.v_scale)
            sees = torch.ones(n, c + n, dtype=torch.bool, device="cuda")
            for j in range(n):
                sees[:, c + j] = (d.mask[t0:t0 + n, j // 64] >> (j % 64)) & 1 == 1
            for g in range(G):
                q = got["q_rot"][t0:t0 + n, h * G + g].double()
                z = (q @ k.t().contiguous() / math.sqrt(D)).masked_fill(~sees, -math.inf)
                w = torch.softmax(z, 1)
                want[t0:t0 + n, h * G + g] = w @ v
                size[t0:t0 + n, h * G + g] = w @ v.abs()
    worst["attended"] = ((got["attended"].double() - want).abs() / (bf * want.abs() + (bf + 1e-4) * size)).max()
    logp = torch.log_softmax(got["following"].double(), -1)
    mine = logp.gather(1, d.tokens.long()[:, None])[:, 0]
    worst["logprobs"] = ((got["logprobs"].double() - mine).abs() / 2e-4).max()
    worst["entropy"] = ((got["entropy"].double() + (logp.exp() * logp).sum(-1)).abs() / 2e-3).max()
    top = torch.sort(got["following"].float(), dim=-1, descending=True, stable=True).indices
    worst["top_ids"] = (got["top_ids"].long() != top[:, :got["top_ids"].shape[1]]).any().double() * 2
    return {k: float(v) for k, v in worst.items()}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--context", type=int, default=1000)
    ap.add_argument("--nodes", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--page", type=int, default=16)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    with torch.no_grad():
        d = Drafts(a.sequences, a.context, a.nodes, a.page, a.vocab)
        layer = Layer(a.hidden, a.heads, a.kv_heads, a.dim, a.vocab, d.pages, a.page, a.cache == "e4m3")
        got = verify(layer, d)
        torch.cuda.synchronize()
        for b, path in enumerate(accept(d, got)):
            t0 = int(d.offsets[b])
            print(f"sequence {b}: context {d.context_list[b]}, {len(d.parents[b])} nodes, accepted "
                  f"{path}, mean log probability of the drafts "
                  f"{float(got['logprobs'][t0:t0 + len(d.parents[b])].mean()):.3f}")
        if a.check:
            worst = check(layer, d, got)
            print("error over its allowed size:", {k: round(v, 3) for k, v in worst.items()})
            return 0 if all(v <= 1 for v in worst.values()) else 1
    return 0


if __name__ == "__main__":
    sys.exit(main())
