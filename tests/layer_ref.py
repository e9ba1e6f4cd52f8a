"""Plain 64-bit forms of the norm with codes and of the low-rank adapters on the
CPU, with the bounds that their tests hold the kernels to: a rounding to a
type is off by at most eps / 2 of the value (or half of the type's smallest
step), binary32 arithmetic of n steps on values of size a by n 2^-24 a."""
import torch

U32 = 2.0 ** -24
QMAX = {"fp8_token": 448.0, "int8_token": 127.0, "fp8_block": 448.0}


def rounding(value, dtype):
    """What one rounding to dtype (and that of the computed value) may cost."""
    low = 2.0 ** -25 if dtype is torch.float16 else 2.0 ** -134
    return torch.finfo(dtype).eps / 2 * value.abs() * (1 + 2.0 ** -7) + low


def norm(x, residual, weight, eps):
    """(s, y, relative error of y in binary32)"""
    s = x.double() if residual is None else x.double() + residual.double()
    y = s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    # s is off by one step; a lane adds up to 32 squares, then 6 steps over lanes and 16 over
    # waves follow, of which the root takes half; the mean, the root and the products
    # take 8 steps more
    return s, y, (1 + (32 + 6 + 16 + 2) / 2 + 10) * U32


def groups(y, kind):
    return y.view(y.shape[0], -1, 128) if kind == "fp8_block" else y[:, None, :]


def check_codes(codes, scales, y, rel, kind):
    """Codes and scales against y."""
    g = groups(y, kind)
    most = g.abs().amax(-1)
    want = torch.where(most > 0, most / QMAX[kind], torch.ones_like(most))
    got = scales.double().view(want.shape)
    assert ((got - want).abs() <= (rel + 4 * U32) * want).all()
    c = groups(codes.float().double(), kind)
    q = g / got[..., None]
    if kind == "int8_token":
        tol = 0.5 + 127 * (rel + 4 * U32) + 0 * q
    else:  # half a step of 3 bits, or of the smallest step 2^-9
        tol = 2.0 ** -4 * q.abs() + 2.0 ** -10 + 448 * (rel + 4 * U32)
    assert ((c - q).abs() <= tol).all()


def lora(x, a, b, ids, base, factors, widths):
    """(out, bound apart from the rounding of the result)"""
    T, K = x.shape
    n, N, R = b.shape
    out = torch.zeros(T, N, dtype=torch.float64) if base is None else base.double()
    err = out.abs() * U32
    x, a, b = x.double(), a.double(), b.double()
    # matrix instructions add 32 products at a time, in an order of their own
    sum_k = 2 * (K / 32 + 64) * U32
    sum_r = 2 * (R / 16 + 64) * U32
    split = 2.0 ** -16  # what the two parts of a value of h leave out
    for i in range(n):
        rows = torch.nonzero(ids == i)[:, 0]
        if not rows.numel():
            continue
        f = 1.0 if factors is None else float(factors[i])
        h, hs = x[rows] @ a[i].t(), x[rows].abs() @ a[i].abs().t()
        col = 0
        for j, w in enumerate(widths):
            part, size = h[:, j * R:(j + 1) * R], hs[:, j * R:(j + 1) * R]
            bw = b[i, col:col + w].t()
            out[rows, col:col + w] += f * (part @ bw)
            miss = size * (sum_k + U32) + part.abs() * split
            err[rows, col:col + w] += abs(f) * ((miss + sum_r * (part.abs() + miss)) @ bw.abs())
            col += w
    return out, err + 2 * U32 * out.abs()


def window_visible(ctx, n, mask, t0, window, sinks, positions):
    """bool [n, ctx + n]: which positions the nodes of a sequence see."""
    own = ctx + torch.arange(n)
    if mask is not None and positions is not None:
        own = positions[t0:t0 + n].long().clamp(ctx, ctx + n - 1)
    c = torch.arange(ctx + n)
    sees = (c < sinks) | (c > own[:, None] - window)
    if mask is None:
        return sees & (c <= own[:, None])
    for j in range(n):
        named = j // 64 < mask.shape[1]
        sees[:, ctx + j] = ((mask[t0:t0 + n, j // 64] >> (j % 64)) & 1) == 1 if named else False
    return sees


def window_attention(q, k_cache, v_cache, table, context, offsets, window, sinks, mask=None, positions=None,
                     scale=None, k_scale=None, v_scale=None, reach=None):
    """(out, bound of out, lse, bound of lse) on CPU tensors; reach: positions of
    the page table (what lies beyond is cut off)."""
    T, H, D = q.shape
    K, page = k_cache.shape[1], k_cache.shape[2]
    G = H // K
    scale = D ** -0.5 if scale is None else scale
    out, tol = torch.zeros(T, H, D, dtype=torch.float64), torch.full((T, H, D), 1e-30, dtype=torch.float64)
    lse = torch.full((T, H), -float("inf"), dtype=torch.float64)
    ltol = torch.zeros(T, H, dtype=torch.float64)
    step = torch.finfo(q.dtype).eps / 2
    for b in range(table.shape[0]):
        t0, t1, ctx = int(offsets[b]), int(offsets[b + 1]), int(context[b])
        n = t1 - t0
        if n == 0:
            continue
        sees = window_visible(ctx, n, mask, t0, window, sinks, positions)
        if reach is not None:
            sees[:, reach:] = False
        some = torch.nonzero(sees.any(0))[:, 0]
        if not some.numel():
            continue
        sees, pages, inside = sees[:, some], table[b].long()[some // page], some % page
        rows = torch.nonzero(sees.any(1))[:, 0]

        def values(cache, factor, h):
            x = cache.view(torch.uint8)[pages, h, inside].view(cache.dtype) if cache.element_size() == 1 \
                else cache[pages, h, inside]
            return x.float().double() * (1.0 if factor is None else float(factor[h]))

        for h in range(K):
            k, v = values(k_cache, k_scale, h), values(v_cache, v_scale, h)
            for g in range(h * G, (h + 1) * G):
                x = q[t0:t1, g].double()
                z = (x @ k.t() * scale).masked_fill(~sees, -float("inf"))
                big = ((x.abs() @ k.abs().t()) * abs(scale)).masked_fill(~sees, 0).amax(1)
                p = torch.softmax(z[rows], 1)
                # values that no row sees weigh nothing, whatever they are
                v0 = torch.where(v.isfinite(), v, 0.0)
                r, a = p @ v0, p @ v0.abs()
                # a score is off by (D + 8) steps of its terms: a relative error of each
                # weight, and twice that after the division; the sums over the positions grow
                # with their number only through rescaling
                rel = (2 * (D + 8) * U32 * big[rows] + (256 + 2 * sees[rows].sum(1).double().sqrt()) * U32)
                out[t0 + rows, g] = r
                tol[t0 + rows, g] = step * r.abs() * (1 + 2.0 ** -7) + (step + rel[:, None]) * a + 1e-30
                if q.dtype is torch.float16:  # the smallest steps of the result and of the weights
                    tol[t0 + rows, g] += 2.0 ** -25 + 2.0 ** -25 * v0.abs().sum(0)
                lse[t0 + rows, g] = torch.logsumexp(z[rows], 1)
                ltol[t0 + rows, g] = rel + 16 * U32 * (1 + lse[t0 + rows, g].abs())
    return out, tol, lse, ltol
