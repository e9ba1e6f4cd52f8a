"""Workloads of what a served decoder layer does around its scaled linear
layers besides heads, cache and trees: the root-mean-square norm with the
residual's addition, which also gives the 8-bit codes and scales that the next
layer reads; low-rank adapters of many requests beside a shared projection;
and attention with a sliding window and a few first tokens that stay visible,
over the paged cache.

``run`` computes a workload in elementary torch operations, or, where ``own``
is true, with the library's kernels (``epilogue_scaled_gemm_amd.Handle``).
``exact`` gives the same from the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
CODES = {"fp8_token": torch.float8_e4m3fn, "int8_token": torch.int8, "fp8_block": torch.float8_e4m3fn}
QMAX = {"fp8_token": 448.0, "int8_token": 127.0, "fp8_block": 448.0}
EPS = 1e-6


# ------------------------------------------------------------------- cases

def _norm(name, **kw):
    """kind: of the 8-bit output ("" for none); out: whether the 16-bit one is wanted too."""
    c = dict(op="norm", tokens=1, width=4096, residual=True, kind="fp8_token", out=False, dtype="bf16")
    return {"name": name, **c, **kw} if name else {**c, **kw}


def _lora(name, **kw):
    """slices: 1, or 3 for a QKV product whose parts have adapters of their own.  runs: rows of
    one request follow each other (prompts), or every row has an adapter of its own choice."""
    c = dict(op="lora", tokens=1, inner=4096, width=4096, rank=16, slices=1, adapters=8, runs=False,
             dtype="bf16")
    return {"name": name, **c, **kw} if name else {**c, **kw}


def _window(name, **kw):
    c = dict(op="window", batch=1, context=1024, nodes=1, window=1024, sinks=4, ragged=False,
             tree=False, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=16)
    return {"name": name, **c, **kw} if name else {**c, **kw}


def listed():
    return [
        # One decoded token before an FP8 layer: latency.
        _norm("norm_step"),
        # A decode step of 24 sequences before a block FP8 layer with adapters (which read 16 bits).
        _norm("norm_step_blocks", tokens=24, width=8192, kind="fp8_block", out=True),
        # Part of a prompt before an INT8 layer, fp16 stream.
        _norm("norm_prompt_int8", tokens=1000, width=5120, kind="int8_token", dtype="fp16"),
        # A long prompt, both outputs: bandwidth.
        _norm("norm_prompt", tokens=8191, out=True),
        # One token through a QKV product (4096 + 1024 + 1024) with an adapter: latency.
        _lora("lora_step_qkv", width=6144, slices=3),
        # A decode step of 48 requests with 24 adapters among them: their weights' bytes.
        _lora("lora_step_many", tokens=48, adapters=24),
        # Short prompts of several requests, a higher rank, an odd output width.
        _lora("lora_prompts_odd", tokens=300, inner=2048, width=4099, rank=64, adapters=5, runs=True,
              dtype="fp16"),
        # A long batch of prompts through a QKV product: bandwidth.
        _lora("lora_prompt_qkv", tokens=8191, width=6144, rank=32, slices=3, adapters=4, runs=True),
        # One token, far past its window: latency.
        _window("window_one_token", context=8191),
        # A decode step of 48 sequences of uneven length, 8-bit cache: bandwidth.
        _window("window_step_8bit", batch=48, context=8191, window=4096, ragged=True, cache="e4m3"),
        # Small drafted trees, narrow heads, a short window.
        _window("window_small_trees", batch=7, context=1500, nodes=23, window=500, sinks=3, ragged=True,
                tree=True, heads=16, kv_heads=4, dim=64, dtype="fp16", cache="fp16", page=32),
        # A part of a prompt over what is cached of it: matrix rate.
        _window("window_prompt_part", batch=2, context=5001, nodes=1500, page=64, sinks=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "lora", "window"))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "norm":
        kind = rng.choice(("", "fp8_token", "int8_token", "fp8_block"))
        step = {"": 8, "fp8_block": 128}.get(kind, 16)
        width = step * _log_int(rng, 256 // step, 16384 // step)
        return _norm(None, tokens=_log_int(rng, 1, min(8191, 8191 * 4096 // width)), width=width,
                     residual=rng.random() < 0.8, kind=kind, out=not kind or rng.random() < 0.5,
                     dtype=dtype)
    if op == "lora":
        inner, width = 8 * _log_int(rng, 32, 1024), _log_int(rng, 64, 14336)
        rank, slices = rng.choice((8, 16, 24, 32, 64, 128)), rng.choice((1, 1, 2, 3))
        adapters = _log_int(rng, 1, max(1, min(64, 2 ** 26 // (rank * (slices * inner + width)))))
        most = 8191 * 4096 // max(inner, width)
        most = min(most, int(2e10 / (adapters * rank * (slices * inner + width))))
        return _lora(None, tokens=_log_int(rng, 1, max(1, min(8191, most))), inner=inner, width=width,
                     rank=rank, slices=slices, adapters=adapters, runs=rng.random() < 0.5, dtype=dtype)
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 6, 8))
    dim = rng.choice((64, 128, 128, 256))
    nodes = rng.choice((1, _log_int(rng, 2, 64), _log_int(rng, 2, 1000)))
    context, window, sinks = _log_int(rng, 1, 32000), _log_int(rng, 16, 8192), rng.choice((0, 1, 4, 64))
    seen = sinks + min(window, context) + nodes
    # no more work than the largest listed cases; a cache of at most 2 GB
    if nodes * seen * heads * dim > 3e10:
        nodes = max(1, int(3e10 / (heads * dim * (seen + 1000))))
    most = min(64, int(2 ** 30 / (kv_heads * dim * (context + nodes) * 2)),
               int(2 ** 29 / (kv_heads * dim * seen * 2)), int(3e10 / (heads * dim * nodes * seen)))
    return _window(None, batch=_log_int(rng, 1, max(1, most)), context=context, nodes=nodes, window=window,
                   sinks=sinks, ragged=rng.random() < 0.7, tree=nodes <= 128 and rng.random() < 0.5,
                   heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                   cache=rng.choice((dtype, dtype, "e4m3")), page=rng.choice((8, 16, 32, 64, 128)))


def _lengths(c):
    """(contexts, node counts) of a window case's sequences."""
    B, L, n = c["batch"], c["context"], c["nodes"]
    if not c["ragged"]:
        return [L] * B, [n] * B
    return ([L - (b * 7919) % (L // 2 + 1) for b in range(B)],
            [n - (b * 31) % (n // 2 + 1) for b in range(B)])


def _widths(c):
    """Output columns of each slice: of three, two thirds belong to the first (queries)."""
    N, S = c["width"], c["slices"]
    rest = [N // (2 * S)] * (S - 1)
    return [N - sum(rest)] + rest


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, scale, generator=g)


def _trees(rng, counts):
    """Random trees: node 0 is the root, each later node hangs on an earlier one.  Bit j % 64 of
    word j // 64 of a node's mask: it sees node j.  And each node's distance from the root."""
    words = (max(counts) + 63) // 64
    rows, depth = [], []
    for n in counts:
        seen, at = [], []
        for i in range(n):
            up = rng.randint(max(0, i - 6), i - 1) if i else -1
            seen.append((seen[up] if i else 0) | 1 << i)
            at.append(at[up] + 1 if i else 0)
        rows += seen
        depth += at
    out = np.zeros((len(rows), words), dtype=np.uint64)
    for w in range(words):
        out[:, w] = [(r >> (64 * w)) & (2 ** 64 - 1) for r in rows]
    return torch.from_numpy(out.view(np.int64)).cuda(), torch.tensor(depth, device="cuda")


def _prepare_norm(c, g, s):
    T, N, dt = c["tokens"], c["width"], DT[c["dtype"]]
    # the stream of a trained model: some channels are far larger than others
    loud = torch.exp(0.7 * _randn(g, N))
    s["x"] = _randn(g, T, N, dtype=dt, scale=0.5)
    s["residual"] = (_randn(g, T, N) * loud).to(dt) if c["residual"] else None
    s["weight"] = (0.6 + 0.2 * _randn(g, N)).to(dt)
    s["residual_out"] = torch.empty(T, N, dtype=dt, device="cuda") if c["residual"] else None
    s["out"] = torch.empty(T, N, dtype=dt, device="cuda") if c["out"] else None
    s["codes"] = s["scales"] = None
    if c["kind"]:
        s["codes"] = torch.empty(T, N, dtype=CODES[c["kind"]], device="cuda")
        s["scales"] = torch.empty((T, N // 128) if c["kind"] == "fp8_block" else (T,), device="cuda")


def _prepare_lora(c, g, s, seed):
    T, K, N, dt = c["tokens"], c["inner"], c["width"], DT[c["dtype"]]
    n, R, S = c["adapters"], c["rank"], c["slices"]
    s["x"] = _randn(g, T, K, dtype=dt)
    s["base"] = _randn(g, T, N, dtype=dt)  # what the shared projection gave
    s["a"] = _randn(g, n, S * R, K, dtype=dt, scale=K ** -0.5)
    s["b"] = _randn(g, n, N, R, dtype=dt, scale=0.1)
    s["factors"] = torch.rand(n, generator=g, device="cuda") + 0.5
    rng = random.Random(seed)
    if c["runs"]:
        ids = []
        while len(ids) < T:
            ids += [rng.randint(-1, n - 1)] * min(T - len(ids), rng.randint(1, max(1, T // 4)))
    else:
        ids = [rng.randint(0, n - 1) if rng.random() < 0.95 else -1 for _ in range(T)]
    if max(ids) < 0:
        ids[0] = rng.randint(0, n - 1)
    s["ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    s["widths"] = _widths(c)
    s["out"] = torch.empty(T, N, dtype=dt, device="cuda")


def _prepare_window(c, g, s, seed):
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
    # queries are a view of the QKV product's output
    s["q"] = _randn(g, T, (H + 2 * K) * D, dtype=dt, scale=1.5)[:, :H * D].view(T, H, D)
    s["context"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["offsets"] = torch.tensor(np.cumsum([0] + cnt), dtype=torch.int32, device="cuda")
    s["mask"] = s["positions"] = None
    if c["tree"]:
        s["mask"], depth = _trees(random.Random(seed), cnt)
        first = torch.repeat_interleave(s["context"].long(), torch.tensor(cnt, device="cuda"))
        s["positions"] = (first + depth).to(torch.int32)
    s["max_context"], s["max_nodes"] = max(ctx), max(cnt)
    s["out"] = torch.empty(T, H, D, dtype=dt, device="cuda")
    s["lse"] = torch.empty(T, H, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "norm":
        _prepare_norm(case, g, s)
    elif case["op"] == "lora":
        _prepare_lora(case, g, s, seed)
    else:
        _prepare_window(case, g, s, seed)
    return s


# ------------------------------------------------------------- plain forms

def _as_values(codes):
    """Codes as a floating type that holds each of them exactly."""
    return codes.to(torch.bfloat16) if codes.dtype == torch.int8 else codes


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    got = {}
    if s["residual"] is not None:
        x = x + s["residual"].float()
        got["residual_out"] = x.to(s["x"].dtype)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if c["out"]:
        got["out"] = y.to(s["x"].dtype)
    if c["kind"]:
        qmax = QMAX[c["kind"]]
        y = y.view(*s["scales"].shape, -1)  # a group's values last
        most = y.abs().amax(-1)
        scales = torch.where(most > 0, most / qmax, torch.ones_like(most))
        q = y / scales[..., None]
        q = q.round() if c["kind"] == "int8_token" else q
        codes = q.clamp(-qmax, qmax).to(CODES[c["kind"]])
        got["codes"], got["scales"] = _as_values(codes.view(s["x"].shape)), scales
    return got


def _plain_lora(s):
    c = s["case"]
    T, n, R, S = c["tokens"], c["adapters"], c["rank"], c["slices"]
    x, ids = s["x"].float(), s["ids"].long()
    at = ids.clamp(min=0)
    f = torch.where(ids >= 0, s["factors"][at], 0.0)[:, None]
    if T < n:  # the weights of each row's adapter
        h = torch.matmul(s["a"][at].float(), x[:, :, None])                      # [T, S R, 1]
        h = h.view(T, S, R)
        b = s["b"][at].float()                                                   # [T, N, R]
        parts = [torch.matmul(p, h[:, i, :, None])[:, :, 0]
                 for i, p in enumerate(torch.split(b, s["widths"], 1))]
    else:      # all adapters at once, of which each row keeps its own
        mine = (ids[:, None] == torch.arange(n, device=ids.device))[:, :, None, None]
        h = torch.matmul(x, s["a"].float().view(n * S * R, -1).t()).view(T, n, S, R)
        h = torch.where(mine, h, 0.0)
        b = s["b"].float().permute(0, 2, 1)                                      # [n, R, N]
        parts = [torch.matmul(h[:, :, i].reshape(T, n * R), p.reshape(n * R, -1))
                 for i, p in enumerate(torch.split(b, s["widths"], 2))]
    return {"out": (s["base"].float() + f * torch.cat(parts, 1)).to(s["base"].dtype)}


def _plain_window(s):
    c = s["case"]
    q, kc, vc = s["q"], s["k_cache"], s["v_cache"]
    T, H, D = q.shape
    B, K, page = s["table"].shape[0], kc.shape[1], kc.shape[2]
    G, n, W, S = H // K, s["max_nodes"], c["window"], c["sinks"]
    node = torch.arange(n, device=q.device)
    first, count = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    row = (first[:, None] + node).clamp(max=T - 1)                       # [B, n]
    qf = q[row].float().view(B, n, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, n * G, D)
    # the positions that any row sees: the first ones, and from the window of node 0 on
    ctx = s["context"].long()[:, None]
    start = (ctx - W + 1).clamp(min=S)
    span = min(W - 1, s["max_context"]) + n
    pos = torch.cat([torch.arange(S, device=q.device).expand(B, S),
                     start + torch.arange(span, device=q.device)], 1)    # [B, L]
    there = pos < ctx + count[:, None]
    pos = torch.where(there, pos, 0)
    L = pos.shape[1]
    at = torch.gather(s["table"].long(), 1, pos // page)

    def rows(cache, scale):
        if scale is None:
            x = cache[at, :, pos % page].float()
        else:
            x = cache.view(torch.uint8)[at, :, pos % page].view(torch.float8_e4m3fn).float()
            x = x * scale[:, None]
        return x                                                         # [B, L, K, D]

    k = rows(kc, s["k_scale"]).permute(0, 2, 3, 1).contiguous()
    v = rows(vc, s["v_scale"]).permute(0, 2, 1, 3).contiguous()
    own_pos = ctx + node if s["positions"] is None else s["positions"].long()[row]   # [B, n]
    near = (pos[:, None, :] > own_pos[:, :, None] - W) | (pos < S)[:, None, :]       # [B, n, L]
    drafted = (pos - ctx)[:, None, :]
    if s["mask"] is None:
        sees = near & (pos[:, None, :] <= own_pos[:, :, None])
    else:
        p = drafted.clamp(0, s["mask"].shape[1] * 64 - 1).expand(B, n, L)
        named = (torch.gather(s["mask"][row], 2, p >> 6) >> (p & 63)) & 1 > 0
        sees = torch.where(drafted < 0, near, named)
    sees = sees & there[:, None, :]
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


# ------------------------------------------------------- the library's own

_kept = []


def _handle():
    if not _kept:
        import epilogue_scaled_gemm_amd
        _kept.append(epilogue_scaled_gemm_amd.Handle())
    return _kept[0]


def _own_norm(s):
    c = s["case"]
    _handle().add_rms_norm(s["x"], s["weight"], residual=s["residual"], residual_out=s["residual_out"],
                           out=s["out"], codes=s["codes"], scales=s["scales"],
                           kind=c["kind"] or "fp8_token", eps=EPS)
    got = {}
    if s["residual"] is not None:
        got["residual_out"] = s["residual_out"]
    if c["out"]:
        got["out"] = s["out"]
    if c["kind"]:
        got["codes"], got["scales"] = _as_values(s["codes"]), s["scales"]
    return got


def _own_lora(s):
    _handle().lora_add(s["x"], s["a"], s["b"], s["ids"], s["out"], base=s["base"], factors=s["factors"],
                       slices=s["widths"])
    return {"out": s["out"]}


def _own_window(s):
    c = s["case"]
    _handle().window_attention(
        s["q"], s["k_cache"], s["v_cache"], s["out"], s["table"], s["context"], s["offsets"],
        max_context=s["max_context"], max_nodes=s["max_nodes"], window=c["window"], sinks=c["sinks"],
        mask=s["mask"], positions=s["positions"], k_scale=s["k_scale"], v_scale=s["v_scale"],
        lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "lora": _own_lora, "window": _own_window}[op](state)
    return {"norm": _plain_norm, "lora": _plain_lora, "window": _plain_window}[op](state)


# -------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "norm":
        T, N = c["tokens"], c["width"]
        per = 2 + 4 * c["residual"] + 2 * c["out"] + (1 if c["kind"] else 0)
        groups = {"": 0, "fp8_block": N // 128}.get(c["kind"], 1)
        return {"bytes": T * N * per + 2 * N + 4 * T * groups, "flops": 8 * T * N}
    if c["op"] == "lora":
        T, K, N, R, S = c["tokens"], c["inner"], c["width"], c["rank"], c["slices"]
        used = min(T, c["adapters"])
        return {"bytes": 2 * T * (K + 2 * N) + 4 * T + 2 * used * R * (S * K + N),
                "flops": 2 * T * R * (S * K + N) + 2 * T * N}
    ctx, cnt = _lengths(c)
    H, K, D, W, S = c["heads"], c["kv_heads"], c["dim"], c["window"], c["sinks"]
    kept = pairs = 0
    for x, n in zip(ctx, cnt):
        first = max(0, x - W + 1)
        kept += x + n - first + min(S, first)
        for j in range(n):
            if c["tree"]:  # the context in the window of the deepest place, and itself at least
                low = max(0, min(x, x + j - W + 1))
                pairs += x - low + min(S, low) + 1
            else:
                low = max(0, x + j - W + 1)
                pairs += x + j + 1 - low + min(S, low)
    size = kept * K * D * 2 * (1 if c["cache"] == "e4m3" else 2) + sum(cnt) * H * (D * 2 * 2 + 4)
    return {"bytes": size, "flops": 4 * H * D * pairs}


# ------------------------------------------- the definitions, in 64 bits

def _exact_norm(c, s):
    total = s["x"].double()
    found = {}
    if s["residual"] is not None:
        total = total + s["residual"].double()
        found["residual_out"] = total
    y = total * s["weight"].double() / torch.sqrt((total * total).sum(1, keepdim=True) / c["width"] + EPS)
    if c["out"]:
        found["out"] = y
    if c["kind"]:
        wide = 128 if c["kind"] == "fp8_block" else c["width"]
        groups = y.unfold(1, wide, wide)
        scales = groups.abs().max(-1).values / QMAX[c["kind"]]
        codes = groups / scales[..., None]
        if c["kind"] == "int8_token":  # whole numbers; e4m3 ones stay as they are before their rounding
            codes = codes.round()
        found["codes"] = codes.reshape(y.shape)
        found["scales"] = scales if c["kind"] == "fp8_block" else scales[:, 0]
    return found


def _exact_lora(c, s):
    out = s["base"].double()
    R = c["rank"]
    for i in range(c["adapters"]):
        rows = torch.nonzero(s["ids"] == i)[:, 0]
        if not rows.numel():
            continue
        h = s["x"][rows].double() @ s["a"][i].double().t()
        col = 0
        for j, w in enumerate(s["widths"]):
            add = h[:, j * R:(j + 1) * R] @ s["b"][i, col:col + w].double().t()
            out[rows, col:col + w] += s["factors"][i].double() * add
            col += w
    return {"out": out}


def _exact_window(c, s):
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
        place = torch.arange(L, device=q.device).expand(n, L)
        at = torch.arange(n, device=q.device)[:, None] + ctx[b]
        if s["positions"] is not None:
            at = s["positions"][t0:t1, None].long()
        sees = (place < c["sinks"]) | (at - place < c["window"])
        if s["mask"] is None:
            sees = sees & (place <= at)
        else:
            for j in range(n):
                sees[:, ctx[b] + j] = (s["mask"][t0:t1, j // 64] >> (j % 64)) & 1 == 1
        # what no row sees is left out of the products
        some = torch.nonzero(sees.any(0))[:, 0]
        sees = sees[:, some]
        pages, inside = s["table"][b].long()[some // page], some % page
        for h in range(K):
            k, v = s["k_cache"], s["v_cache"]
            if k.dtype == torch.float8_e4m3fn:
                k = k.view(torch.uint8)[pages, h, inside].view(torch.float8_e4m3fn).double() * s["k_scale"][h].double()
                v = v.view(torch.uint8)[pages, h, inside].view(torch.float8_e4m3fn).double() * s["v_scale"][h].double()
            else:
                k, v = k[pages, h, inside].double(), v[pages, h, inside].double()
            x = q[t0:t1, h * G:(h + 1) * G].double().reshape(n * G, D) @ k.t().contiguous() / math.sqrt(D)
            x = x.masked_fill(~sees.repeat_interleave(G, 0), -math.inf)
            lse[t0:t1, h * G:(h + 1) * G] = torch.logsumexp(x, 1).view(n, G)
            out[t0:t1, h * G:(h + 1) * G] = (torch.softmax(x, 1) @ v).view(n, G, D)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "lora": _exact_lora, "window": _exact_window}[case["op"]](case, s)
