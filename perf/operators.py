"""Workloads of the operators that stand between the scaled linear layers of a
decoder when tokens are served, one token or a tree of drafted tokens at a
time: per-head norms with the position rotation, appending keys and values
to a paged cache, attention of drafted tokens over that cache, and the log
probabilities of given tokens.

``run`` computes a workload in elementary torch operations, or, where ``own``
is true, with the library's kernels (``epilogue_scaled_gemm_amd.Handle``).
``exact`` gives the same from the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
      "e4m3": torch.float8_e4m3fn}
MAX_POS = 131072  # rows of the rotation table
EPS = 1e-6


# ------------------------------------------------------------------- cases

def _rope(name, **kw):
    c = dict(op="norm_rope", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, pairs="half",
             norm=True, dtype="bf16", far=False)
    return {"name": name, **c, **kw} if name else {**c, **kw}


def _append(name, **kw):
    c = dict(op="append", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, pairs="half",
             norm=False, dtype="bf16", cache="bf16", page=16, spare=64, far=False)
    return {"name": name, **c, **kw} if name else {**c, **kw}


def _attend(name, **kw):
    c = dict(op="attend", batch=1, context=1024, nodes=1, ragged=False, tree=True, heads=32,
             kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=16)
    return {"name": name, **c, **kw} if name else {**c, **kw}


def _score(name, **kw):
    c = dict(op="score", tokens=1, vocab=32000, top=5, dtype="bf16", temperature=1.0)
    return {"name": name, **c, **kw} if name else {**c, **kw}


def listed():
    return [
        # One decoded token of a 32/8-head layer (the 6144-wide QKV product): latency.
        _rope("norm_rope_step"),
        # A long prompt through the same layer: bandwidth.
        _rope("norm_rope_prompt", tokens=8191),
        # A decode step of 24 sequences into an 8-bit cache, queries in the same call.
        _append("append_step_8bit", tokens=24, norm=True, cache="e4m3"),
        # A prompt's keys and values into 64-token pages, positions far out.
        _append("append_prompt", tokens=4099, page=64, far=True),
        # One token over a short context: latency.
        _attend("attend_one_token", context=1023),
        # A decode step of 48 sequences of uneven length over an 8-bit cache: bandwidth.
        _attend("attend_step_8bit", batch=48, context=8191, ragged=True, cache="e4m3"),
        # Small trees of uneven size, narrow heads.
        _attend("attend_small_trees", batch=7, context=1500, nodes=23, ragged=True, heads=16,
                kv_heads=4, dim=64, dtype="fp16", cache="fp16", page=32),
        # 64 drafted tokens each over long contexts: bandwidth and matrix rate together.
        _attend("attend_trees_long", batch=4, context=32000, nodes=64, page=64),
        # A part of a prompt over what is cached of it: matrix rate.
        _attend("attend_prompt_part", batch=2, context=5001, nodes=1500, tree=False, page=64),
        # Scoring one sampled token: latency.
        _score("score_step", vocab=32003),
        # Scoring drafted tokens, 32-bit logits, an odd vocabulary, many alternatives.
        _score("score_drafts", tokens=48, vocab=128259, top=20, dtype="fp32", temperature=0.7),
        # Scoring a prompt: bandwidth.
        _score("score_prompt", tokens=2048, vocab=131072, top=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "attend", "attend", "score"))
    dtype = rng.choice(("bf16", "fp16"))
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 6, 8))
    dim = rng.choice((64, 128, 128, 256))
    if op in ("norm_rope", "append"):
        most = max(16, 8191 * 40 * 128 // ((heads + 2 * kv_heads) * dim))
        kw = dict(tokens=_log_int(rng, 1, min(8191, most)), heads=heads, kv_heads=kv_heads, dim=dim,
                  rot=rng.choice((dim, dim // 2, 32)), pairs=rng.choice(("half", "interleaved")),
                  norm=rng.random() < 0.6, dtype=dtype, far=rng.random() < 0.5)
        if op == "norm_rope":
            return _rope(None, **kw)
        return _append(None, **kw, cache=rng.choice((dtype, "e4m3")),
                       page=rng.choice((8, 16, 32, 64)), spare=rng.randint(1, 100))
    if op == "attend":
        nodes = rng.choice((1, _log_int(rng, 2, 64), _log_int(rng, 2, 1000)))
        context = _log_int(rng, 1, 32000)
        # no more work than the largest listed cases
        most = min(64, max(1, int(2 ** 30 / (kv_heads * dim * (context + nodes) * 4))),
                   max(1, int(4e9 / (heads * dim * nodes * (context + nodes)))))
        if nodes * (context + nodes) * heads * dim > 30e9:
            nodes = max(1, int(30e9 / (heads * dim * (context + 1000))))
        return _attend(None, batch=_log_int(rng, 1, most), context=context, nodes=nodes,
                       ragged=rng.random() < 0.7, tree=nodes <= 128 and rng.random() < 0.7,
                       heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                       cache=rng.choice((dtype, dtype, "e4m3")), page=rng.choice((8, 16, 32, 64, 128)))
    vocab = _log_int(rng, 1000, 200000)
    dtype = rng.choice(("bf16", "fp16", "fp32"))
    most = 2048 * 131072 * 2 // (vocab * (4 if dtype == "fp32" else 2))
    return _score(None, tokens=_log_int(rng, 1, min(4000, most)), vocab=vocab, dtype=dtype,
                  top=rng.choice((0, 1, 5, 20, 32)), temperature=rng.choice((1.0, 0.7, 1.3)))


def _lengths(c):
    """(contexts, node counts) of a case's sequences."""
    B, L, n = c["batch"], c["context"], c["nodes"]
    if not c["ragged"]:
        return [L] * B, [n] * B
    return ([L - (b * 7919) % (L // 2 + 1) for b in range(B)],
            [n - (b * 31) % (n // 2 + 1) for b in range(B)])


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, scale, generator=g)


_tables = {}


def _table(rot):
    """Cosines, then sines, of every position: a model's constant, made once."""
    if rot not in _tables:
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        a = torch.arange(MAX_POS, dtype=torch.float64)[:, None] * inv[None, :]
        _tables[rot] = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    return _tables[rot]


def _positions(c, g):
    first = torch.randint(0, MAX_POS - 8192, (1,), generator=g, device="cuda") if c["far"] else 0
    return (torch.arange(c["tokens"], device="cuda") + first).to(torch.int32)


def _trees(rng, counts):
    """Random trees: node 0 is the root, each later node hangs on an earlier
    one.  Bit j of word j // 64 of a node's mask: it sees node j."""
    words = (max(counts) + 63) // 64
    rows = []
    for n in counts:
        seen = []
        for i in range(n):
            up = seen[rng.randint(max(0, i - 6), i - 1)] if i else 0
            seen.append(up | 1 << i)
        rows += seen
    out = np.zeros((len(rows), words), dtype=np.uint64)
    for w in range(words):
        out[:, w] = [(r >> (64 * w)) & (2 ** 64 - 1) for r in rows]
    return torch.from_numpy(out.view(np.int64)).cuda()


def prepare(case, seed):
    c = case
    g = _generator(seed)
    s = {"case": c}
    if c["op"] in ("norm_rope", "append"):
        T, H, K, D, dt = c["tokens"], c["heads"], c["kv_heads"], c["dim"], DT[c["dtype"]]
        # the QKV layer's output; queries, keys and values are views of it
        s["qkv"] = qkv = _randn(g, T, (H + 2 * K) * D, dtype=dt)
        s["q"] = qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + K) * D].view(T, K, D)
        s["v"] = qkv[:, (H + K) * D:].view(T, K, D)
        s["table"] = _table(c["rot"])
        s["positions"] = _positions(c, g)
        s["qw"] = (_randn(g, D, scale=0.2) + 1.0).to(dt) if c["norm"] else None
        s["kw"] = (_randn(g, D, scale=0.2) + 1.0).to(dt) if c["norm"] else None
        s["q_out"] = torch.empty(T, H, D, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(T, K, D, dtype=dt, device="cuda")
        if c["op"] == "append":
            page = c["page"]
            pages = (T + page - 1) // page + c["spare"]
            shape = (pages, K, page, D)
            s["k_cache"] = _randn(g, *shape, dtype=torch.bfloat16).to(DT[c["cache"]])
            s["v_cache"] = _randn(g, *shape, dtype=torch.bfloat16).to(DT[c["cache"]])
            if T <= 64:  # a decode step: each token in a page of its own sequence
                at = torch.randperm(pages * page, generator=g, device="cuda")[:T]
            else:        # a prompt: whole pages, in the order that the allocator gave
                order = torch.randperm(pages, generator=g, device="cuda")
                t = torch.arange(T, device="cuda")
                at = order[t // page] * page + t % page
            s["slots"] = at.to(torch.int32)
            s["k_scale"] = s["v_scale"] = None
            if c["cache"] == "e4m3":
                s["k_scale"] = torch.rand(K, generator=g, device="cuda") * 0.05 + 0.02
                s["v_scale"] = torch.rand(K, generator=g, device="cuda") * 0.05 + 0.02
        return s
    if c["op"] == "attend":
        H, K, D, page, dt = c["heads"], c["kv_heads"], c["dim"], c["page"], DT[c["dtype"]]
        ctx, cnt = _lengths(c)
        B, T = c["batch"], sum(cnt)
        need = [(x + n + page - 1) // page for x, n in zip(ctx, cnt)]
        order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
        s["table"] = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            s["table"][b, :n] = order[at:at + n]
            at += n
        shape = (sum(need), K, page, D)
        s["k_cache"] = _randn(g, *shape, dtype=torch.bfloat16).to(DT[c["cache"]])
        s["v_cache"] = _randn(g, *shape, dtype=torch.bfloat16).to(DT[c["cache"]])
        s["k_scale"] = s["v_scale"] = None
        if c["cache"] == "e4m3":
            s["k_scale"] = torch.rand(K, generator=g, device="cuda") + 0.5
            s["v_scale"] = torch.rand(K, generator=g, device="cuda") + 0.5
        s["q"] = _randn(g, T, (H + 2 * K) * D, dtype=dt, scale=1.5)[:, :H * D].view(T, H, D)
        s["context"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.tensor(np.cumsum([0] + cnt), dtype=torch.int32, device="cuda")
        s["mask"] = _trees(random.Random(seed), cnt) if c["tree"] else None
        s["max_context"], s["max_nodes"] = max(ctx), max(cnt)
        s["out"] = torch.empty(T, H, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(T, H, device="cuda")
        return s
    T, V = c["tokens"], c["vocab"]
    s["logits"] = _randn(g, T, V, dtype=DT[c["dtype"]], scale=3.0)
    s["tokens"] = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    s["logprobs"] = torch.empty(T, device="cuda")
    s["entropy"] = torch.empty(T, device="cuda")
    s["top_ids"] = s["top_logprobs"] = None
    if c["top"]:
        s["top_ids"] = torch.empty(T, c["top"], dtype=torch.int32, device="cuda")
        s["top_logprobs"] = torch.empty(T, c["top"], device="cuda")
    return s


# ------------------------------------------------------------- plain forms

def _plain_heads(x, weight, c, table, positions):
    """One round of per-head norm (where asked for) and rotation, in 32 bits."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rot = c["rot"]
    row = table[positions.long()][:, None, :]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    if c["pairs"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], -1)
    a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_store(cache, slots, x, scale):
    page = cache.shape[2]
    at = slots.long()
    if scale is not None:
        x = (x / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        cache = cache.view(torch.uint8)
    cache[at // page, :, at % page] = x.to(cache.dtype)


def _plain_norm_rope(s):
    c = s["case"]
    q = _plain_heads(s["q"], s["qw"], c, s["table"], s["positions"]).to(s["q"].dtype)
    k = _plain_heads(s["k"], s["kw"], c, s["table"], s["positions"]).to(s["k"].dtype)
    return {"q": q, "k": k}


def _plain_append(s):
    c = s["case"]
    q = _plain_heads(s["q"], s["qw"], c, s["table"], s["positions"]).to(s["q"].dtype)
    k = _plain_heads(s["k"], s["kw"], c, s["table"], s["positions"])
    _plain_store(s["k_cache"], s["slots"], k, s["k_scale"])
    _plain_store(s["v_cache"], s["slots"], s["v"].float(), s["v_scale"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    q, kc, vc = s["q"], s["k_cache"], s["v_cache"]
    T, H, D = q.shape
    B, K, page = s["table"].shape[0], kc.shape[1], kc.shape[2]
    G, n, L = H // K, s["max_nodes"], s["table"].shape[1] * page
    node = torch.arange(n, device=q.device)
    first, count = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    row = (first[:, None] + node).clamp(max=T - 1)                       # [B, n]
    qf = q[row].float().view(B, n, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, n * G, D)
    at = s["table"].long()
    if kc.dtype == torch.float8_e4m3fn:
        k = kc.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["k_scale"][:, None, None]
        v = vc.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["v_scale"][:, None, None]
    else:
        k, v = kc[at].float(), vc[at].float()
    k = k.permute(0, 2, 4, 1, 3).reshape(B, K, D, L)                     # [B, K, D, L]
    v = v.transpose(1, 2).reshape(B, K, L, D)
    ctx = s["context"].long()[:, None]
    pos = torch.arange(L, device=q.device)[None, :] - ctx                # drafted node at a position
    if s["mask"] is None:
        sees = pos[:, None, :] <= node[None, :, None]
    else:
        p = pos.clamp(0, s["mask"].shape[1] * 64 - 1)[:, None, :].expand(B, n, L)
        sees = (torch.gather(s["mask"][row], 2, p >> 6) >> (p & 63)) & 1 > 0
        sees = (pos[:, None, :] < 0) | sees
    sees = sees & (pos < count[:, None])[:, None, :]                     # [B, n, L]
    scores = torch.matmul(qf, k).mul_(1.0 / math.sqrt(D)).view(B, K, n, G, L)
    scores.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    e = scores.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, K, n * G, L), v).view(B, K, n, G, D) / total
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * n, H, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B * n, H)
    # back from the padded rows: node t of the call is node t - first of its sequence
    t = torch.arange(T, device=q.device)
    b = (t[:, None] >= s["offsets"][None, 1:].long()).sum(1)
    back = b * n + t - first[b]
    return {"out": o[back].to(q.dtype), "lse": lse[back]}


def _plain_score(s):
    c = s["case"]
    x = s["logits"].float()
    z = x / c["temperature"]
    top = z.amax(-1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(-1, keepdim=True)
    lse = top + total.log()
    got = z.gather(1, s["tokens"].long()[:, None])
    entropy = total.log() - (e * (z - top)).sum(-1, keepdim=True) / total
    out = {"logprobs": (got - lse)[:, 0], "entropy": entropy[:, 0]}
    if c["top"]:
        # one order of values and places: larger values first, then lower places
        bits = (x + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 32)
        key = key + (0x7FFFFFFF - torch.arange(x.shape[1], device=x.device))
        ids = 0x7FFFFFFF - (torch.topk(key, c["top"], dim=1).values & 0x7FFFFFFF)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = z.gather(1, ids) - lse
    return out


# ------------------------------------------------------- the library's own

_kept = []


def _handle():
    if not _kept:
        import epilogue_scaled_gemm_amd
        _kept.append(epilogue_scaled_gemm_amd.Handle())
    return _kept[0]


def _own_norm_rope(s):
    q, k = _handle().qk_norm_rope(
        s["q"], s["k"], s["q_out"], s["k_out"], cos_sin=s["table"], positions=s["positions"],
        q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=s["case"]["pairs"] != "half")
    return {"q": q, "k": k}


def _own_append(s):
    _handle().kv_append(
        s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], cos_sin=s["table"],
        positions=s["positions"], k_weight=s["kw"], eps=EPS,
        interleaved=s["case"]["pairs"] != "half", k_scale=s["k_scale"], v_scale=s["v_scale"],
        q=s["q"], q_out=s["q_out"], q_weight=s["qw"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    _handle().tree_attention(
        s["q"], s["k_cache"], s["v_cache"], s["out"], s["table"], s["context"], s["offsets"],
        max_context=s["max_context"], max_nodes=s["max_nodes"], mask=s["mask"],
        k_scale=s["k_scale"], v_scale=s["v_scale"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_score(s):
    _handle().token_logprobs(
        s["logits"], s["tokens"], s["logprobs"], entropy=s["entropy"], top_ids=s["top_ids"],
        top_logprobs=s["top_logprobs"], temperature=s["case"]["temperature"])
    out = {"logprobs": s["logprobs"], "entropy": s["entropy"]}
    if s["case"]["top"]:
        out.update(top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "append": _own_append, "attend": _own_attend,
                "score": _own_score}[op](state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "attend": _plain_attend,
            "score": _plain_score}[op](state)


# -------------------------------------------------------------------- work

_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def work(case):
    c = case
    if c["op"] in ("norm_rope", "append"):
        T, D, e = c["tokens"], c["dim"], _SIZE[c["dtype"]]
        rows = T * c["rot"] * 4 + T * 4
        if c["op"] == "norm_rope":
            n = T * (c["heads"] + c["kv_heads"]) * D
            return {"bytes": 2 * n * e + rows, "flops": 10 * n}
        n = T * (c["heads"] + 2 * c["kv_heads"]) * D
        put = T * c["heads"] * D * e + T * 2 * c["kv_heads"] * D * _SIZE[c["cache"]]
        return {"bytes": n * e + put + rows + 4 * T, "flops": 10 * n}
    if c["op"] == "attend":
        ctx, cnt = _lengths(c)
        H, K, D = c["heads"], c["kv_heads"], c["dim"]
        kept = sum(x + n for x, n in zip(ctx, cnt))
        # what a node sees: the context and itself at least, all before it without a tree
        pairs = sum(n * x + (n if c["tree"] else n * (n + 1) // 2) for x, n in zip(ctx, cnt))
        size = kept * K * D * 2 * _SIZE[c["cache"]] + sum(cnt) * H * (D * 2 * 2 + 4)
        return {"bytes": size, "flops": 4 * H * D * pairs}
    n = c["tokens"] * c["vocab"]
    return {"bytes": n * _SIZE[c["dtype"]] + c["tokens"] * (12 + 8 * c["top"]), "flops": 5 * n}


# ------------------------------------------- the definitions, in 64 bits

def _exact_heads(x, weight, c, table, positions):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    half = c["rot"] // 2
    turn = table.double()[positions.long()]
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None, :]
    head, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["pairs"] == "half":
        z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn
        return torch.cat((z.real, z.imag, rest), dim=-1)
    z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous()) * turn
    return torch.cat((torch.view_as_real(z).reshape(head.shape), rest), dim=-1)


def _exact_cache(cache, slots, x, scale):
    out = cache.double()
    if scale is not None:
        x = torch.clamp(x / scale.double().view(1, -1, 1), -448, 448)
    page = cache.shape[2]
    flat = out.permute(0, 2, 1, 3).reshape(-1, out.shape[1], out.shape[3])
    flat = flat.index_copy(0, slots.long(), x)
    return flat.view(-1, page, out.shape[1], out.shape[3]).permute(0, 2, 1, 3).contiguous()


def _exact_attend(s):
    q = s["q"]
    T, H, D = q.shape
    K, page = s["k_cache"].shape[1:3]
    G = H // K
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    offsets, ctx = s["offsets"].tolist(), s["context"].tolist()
    for b in range(len(ctx)):
        t0, t1 = offsets[b], offsets[b + 1]
        n, L = t1 - t0, ctx[b] + t1 - t0
        sees = torch.ones(n, L, dtype=torch.bool, device=q.device)
        for j in range(n):
            if s["mask"] is None:
                sees[:, ctx[b] + j] = torch.arange(n, device=q.device) >= j
            else:
                sees[:, ctx[b] + j] = (s["mask"][t0:t1, j // 64] >> (j % 64)) & 1 == 1
        pages = s["table"][b, :(L + page - 1) // page].long()
        for h in range(K):
            k = s["k_cache"].view(-1, K, page, D)[:, h]
            v = s["v_cache"].view(-1, K, page, D)[:, h]
            if k.dtype == torch.float8_e4m3fn:
                k = k.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * s["k_scale"][h].double()
                v = v.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * s["v_scale"][h].double()
            else:
                k, v = k[pages].double(), v[pages].double()
            k, v = k.reshape(-1, D)[:L], v.reshape(-1, D)[:L]
            x = q[t0:t1, h * G:(h + 1) * G].double().reshape(n * G, D) @ k.t().contiguous() / math.sqrt(D)
            x = x.masked_fill(~sees.repeat_interleave(G, 0), -math.inf)
            lse[t0:t1, h * G:(h + 1) * G] = torch.logsumexp(x, 1).view(n, G)
            out[t0:t1, h * G:(h + 1) * G] = (torch.softmax(x, 1) @ v).view(n, G, D)
    return {"out": out, "lse": lse}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("norm_rope", "append"):
        q = _exact_heads(s["q"], s["qw"], c, s["table"], s["positions"])
        k = _exact_heads(s["k"], s["kw"], c, s["table"], s["positions"])
        if c["op"] == "norm_rope":
            return {"q": q, "k": k}
        return {"q": q, "k_cache": _exact_cache(s["k_cache"], s["slots"], k, s["k_scale"]),
                "v_cache": _exact_cache(s["v_cache"], s["slots"], s["v"].double(), s["v_scale"])}
    if c["op"] == "attend":
        return _exact_attend(s)
    z = s["logits"].double() / c["temperature"]
    logp = torch.log_softmax(z, -1)
    out = {"logprobs": logp[torch.arange(c["tokens"]), s["tokens"].long()],
           "entropy": -(logp.exp() * logp).sum(-1)}
    if c["top"]:
        ids = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = logp.gather(1, ids)
    return out
