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
