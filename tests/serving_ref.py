"""Plain 64-bit forms of the serving operators on the CPU, with the error
bounds that their tests hold the kernels to.

Bounds.  A result rounded to a type is off by at most eps / 2 of its value;
binary32 arithmetic of n steps on values of size a by n 2^-24 a.  Each
function returns (result, bound) with the bound made of these two parts.
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def heads(x, weight, eps, table, positions, rot, interleaved):
    """(y, a): the normalised and rotated heads in 64 bits, and the size of
    the values that went into each."""
    y = x.double()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    size = y.abs()
    if table is not None:
        row = table.double()[positions.long().clamp(0, table.shape[0] - 1)][:, None, :]
        c, s = row[..., :rot // 2], row[..., rot // 2:]
        lo, hi = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved else
                  (slice(0, rot // 2), slice(rot // 2, rot)))
        a, b = y[..., lo].clone(), y[..., hi].clone()
        y, size = y.clone(), size.clone()
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        size[..., lo] = size[..., hi] = a.abs() + b.abs()
    return y, size


def heads_bound(y, size, dim, dtype):
    # the norm adds dim squares (half of their relative error), a root, a
    # division and two products; the rotation two products and a sum
    return half_step(dtype) * y.abs() * (1 + 2.0 ** -8) + (dim / 2 + 16) * U32 * size + 1e-30


def code_bound(y, size, dim, scale):
    # e4m3: half a step of 2^-3, half of the smallest step 2^-9
    return 2.0 ** -4 * y.abs() * (1 + 2.0 ** -8) + 2.0 ** -10 * scale + \
        (dim / 2 + 20) * U32 * size


def visible(ctx, n, mask, t0):
    """bool [n, ctx + n]"""
    sees = torch.ones(n, ctx + n, dtype=torch.bool)
    for j in range(n):
        if mask is None:
            sees[:, ctx + j] = torch.arange(n) >= j
        elif j // 64 < mask.shape[1]:
            sees[:, ctx + j] = ((mask[t0:t0 + n, j // 64] >> (j % 64)) & 1) == 1
        else:
            sees[:, ctx + j] = False
    return sees


def gather_cache(cache, scale, table_row, length, h):
    page = cache.shape[2]
    pages = table_row[:(length + page - 1) // page].long()
    rows = cache[:, h]
    if rows.dtype == torch.float8_e4m3fn:
        rows = rows.view(torch.uint8)[pages].view(torch.float8_e4m3fn)
    else:
        rows = rows[pages]
    rows = rows.double().reshape(-1, cache.shape[3])[:length]
    return rows * (1.0 if scale is None else float(scale[h]))


def attention(q, k_cache, v_cache, table, context, offsets, mask, scale, k_scale, v_scale):
    """(out, bound of out, lse, bound of lse) on CPU tensors."""
    T, Hq, D = q.shape
    Hk = k_cache.shape[1]
    G = Hq // Hk
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    ltol = torch.zeros_like(lse)
    step = half_step(q.dtype)
    for b in range(table.shape[0]):
        t0, t1, ctx = int(offsets[b]), int(offsets[b + 1]), int(context[b])
        n = t1 - t0
        if n == 0:
            continue
        sees = visible(ctx, n, mask, t0)
        for h in range(Hk):
            k = gather_cache(k_cache, k_scale, table[b], ctx + n, h)
            v = gather_cache(v_cache, v_scale, table[b], ctx + n, h)
            for g in range(G):
                x = q[t0:t1, h * G + g].double()
                for i in range(n):
                    w = sees[i]
                    if not w.any():
                        continue
                    z = (k[w] @ x[i]) * scale
                    big = float((k[w].abs() @ x[i].abs()).max() * abs(scale))
                    p = torch.softmax(z, 0)
                    r = p @ v[w]
                    a = p @ v[w].abs()
                    # a score is off by (D + 8) steps of its terms: a relative
                    # error of each weight, and twice that after the division;
                    # the sums over the positions grow with their number only
                    # through rescaling (a few hundred steps at most here)
                    rel = 2 * (D + 8) * U32 * big + (256 + 2 * int(w.sum()) ** 0.5) * U32
                    out[t0 + i, h * G + g] = r
                    tol[t0 + i, h * G + g] = step * r.abs() * (1 + 2.0 ** -7) + (step + rel) * a + 1e-30
                    lse[t0 + i, h * G + g] = torch.logsumexp(z, 0)
                    ltol[t0 + i, h * G + g] = rel + 16 * U32 * (1 + abs(float(lse[t0 + i, h * G + g])))
    return out, tol, lse, ltol


def score(logits, tokens, top, temperature):
    """(logprobs, entropy, ids, top logprobs, bound)"""
    x = logits.double()
    logp = torch.log_softmax(x / temperature, -1)
    rows = torch.arange(x.shape[0])
    ok = (tokens >= 0) & (tokens < x.shape[1])
    lp = torch.where(ok, logp[rows, tokens.long().clamp(0, x.shape[1] - 1)], torch.nan)
    plogp = torch.where(logp == -math.inf, torch.zeros_like(logp), logp.exp() * logp)
    order = torch.sort(logits.float() + 0.0, dim=-1, descending=True, stable=True).indices[:, :top]
    # a lane adds at most V / 64 terms one after the other; z and its
    # difference to the maximum are off by a few steps of their size (masks of
    # a type's lowest value weigh nothing, and have their own size as results)
    finite = torch.where(x.abs() < 1e30, x, torch.zeros_like(x)).abs().max() / temperature
    n = x.shape[1] / 64 + 64
    bound = n * U32 + 8 * U32 * float(finite)
    return lp, -plogp.sum(-1), order, logp.gather(1, order), bound
