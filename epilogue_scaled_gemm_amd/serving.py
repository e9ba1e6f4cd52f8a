"""The serving operators of a handle: what stands between the linear layers
when tokens are served -- per-head norms with the position rotation,
appending to a paged cache, attention of new tokens over that cache, and the
log probabilities of given tokens (C ABI in include/lin_gemm.h).

    h = Handle()
    h.kv_append(k, v, k_cache, v_cache, slots, cos_sin=table, positions=pos,
                k_weight=kw, q=q, q_out=q_rot, q_weight=qw)
    h.tree_attention(q_rot, k_cache, v_cache, out, page_table, context, offsets,
                     max_context=..., max_nodes=..., mask=mask)
    h.token_logprobs(logits, drafted, logprobs, top_ids=ids, top_logprobs=lps)

Shapes.  Heads are [tokens, heads, dim] views (any token and head strides that
are multiples of 8, dim contiguous), caches [pages, heads, page, dim] with
any order of the first three in memory; page a power of two.  Caches hold the
heads' type, or float8_e4m3fn codes with a scale per head.  Plans (positions,
slots, page tables, contexts, offsets, token ids) are int32 on the GPU.

A "node" is a new token: one per sequence in plain decoding, a tree of
drafted tokens, or a part of a prompt.  The nodes of all sequences follow
each other in one call; offsets[b] .. offsets[b + 1] are those of sequence b.
"""
import ctypes
import math
import struct

import torch

_HEADS = struct.Struct("<36qd5q")
_ATTENTION = struct.Struct("<31qd2q")
_SCORE = struct.Struct("<6qd5q")
_WINDOW = struct.Struct("<31qd5q")
_NORM = struct.Struct("<10qd5q")
_LORA = struct.Struct("<21q")
_DTYPE16 = {torch.bfloat16: 0, torch.float16: 1}
_SCORE_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_NO = (0, 0, 0)
_NORM_KIND = {"fp8_token": (0, torch.float8_e4m3fn), "int8_token": (1, torch.int8),
              "fp8_block": (2, torch.float8_e4m3fn)}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def declare(lib):
    """Argument types of the serving entry points."""
    for name in ("qk_norm_rope", "kv_append", "tree_attention", "token_logprobs", "window_attention",
                 "add_rms_norm", "lora_add"):
        f = getattr(lib, "lin_gemm_" + name)
        f.argtypes = [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p]
        f.restype = ctypes.c_int


def _at(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name}: tensors must live on the GPU")
    return t.data_ptr()


def _heads(name, t, shape, dtype):
    """(address, token stride, head stride) of a [tokens, heads, dim] view."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (no broadcasting), got {list(t.shape)}")
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    # a dimension of one is never stepped over
    return _at(name, t), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0


def _cache(name, t, shape, dtype):
    """(address, page, head and in-page strides) of a [pages, heads, page, dim] cache."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    ps, hs, ts, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    return (_at(name, t), ps if shape[0] > 1 else 0, hs if shape[1] > 1 else 0,
            ts if shape[2] > 1 else 0)


def _flat(name, t, count, dtype):
    """Address of a contiguous tensor of exactly `count` values, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != count:
        raise ValueError(f"{name} must hold {count} values (no broadcasting), got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _at(name, t)


def _rows(name, t, shape, dtype):
    """(address, row stride) of a [rows, width] view, (0, 0) for None."""
    if t is None:
        return 0, 0
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (no broadcasting), got {list(t.shape)}")
    rs, vs = t.stride()
    if vs != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the values of a row must be contiguous")
    return _at(name, t), rs if shape[0] > 1 else 0


def _cache_type(k_cache, dtype, k_scale, v_scale):
    if k_cache.dtype is torch.float8_e4m3fn:
        return 2
    if k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale are for float8_e4m3fn caches")
    return _DTYPE16[dtype]


def _forward_only(*tensors):
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise RuntimeError("the serving operators are forward only: call them under "
                                   "torch.no_grad() or on detached tensors")


def _stream_of(stream, t):
    # the current stream's address without the Stream object that
    # torch.cuda.current_stream builds: 0.2 instead of 4 us of a 10 us call
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(t.get_device())


class ServingOps:
    """Methods of Handle."""

    def _rope_part(self, T, dtype, dim, cos_sin, positions, q_weight, k_weight, eps, interleaved):
        rope, rows, rot, pos = 0, 0, 0, 0
        if cos_sin is not None:
            if cos_sin.dim() != 2:
                raise ValueError("cos_sin must be [positions, rope_dim]")
            if positions is None:
                raise ValueError("a rotation needs positions")
            rows, rot = cos_sin.shape
            rope = _flat("cos_sin", cos_sin, rows * rot, torch.float32)
            pos = _flat("positions", positions, T, torch.int32)
        return (_flat("q_weight", q_weight, dim, dtype), _flat("k_weight", k_weight, dim, dtype),
                float(eps), rope, rows, rot, pos, 1 if interleaved else 0)

    def qk_norm_rope(self, q, k, q_out, k_out, cos_sin=None, positions=None, q_weight=None,
                     k_weight=None, eps=1e-6, interleaved=False, stream=None):
        """Per-head norms (where a weight [dim] is given) and the position
        rotation (where a table is given, see rope_table) of q [T, Hq, dim]
        and k [T, Hk, dim], in one pass, into q_out and k_out (which may be q
        and k).  Returns (q_out, k_out)."""
        _forward_only(q, k, q_weight, k_weight)
        dtype = q.dtype
        if dtype not in _DTYPE16 or q.dim() != 3 or k.dim() != 3:
            raise ValueError("q and k must be [tokens, heads, dim] in bfloat16 or float16")
        T, Hq, D = qs = q.shape
        ks = k.shape
        if ks[0] != T or ks[2] != D:
            raise ValueError(f"k must be [{T}, heads, {D}], got {list(ks)}")
        args = _HEADS.pack(
            _DTYPE16[dtype], T, D, Hq, *_heads("q", q, qs, dtype),
            *_heads("q_out", q_out, qs, dtype), ks[1], *_heads("k", k, ks, dtype),
            *_heads("k_out", k_out, ks, dtype), *_NO, 0, *_NO, 0, *_NO, 0, 0, 0, 0, 0, 0,
            *self._rope_part(T, dtype, D, cos_sin, positions, q_weight, k_weight, eps,
                             interleaved))
        rc = self._lib.lin_gemm_qk_norm_rope(self._h, args, _stream_of(stream, q))
        if rc:
            self._check(rc, "lin_gemm_qk_norm_rope")
        return q_out, k_out

    def kv_append(self, k, v, k_cache, v_cache, slots, cos_sin=None, positions=None, k_weight=None,
                  eps=1e-6, interleaved=False, k_scale=None, v_scale=None, q=None, q_out=None,
                  q_weight=None, stream=None):
        """Store k and v [T, Hk, dim] at slots [T] of the caches, the keys
        normalised and rotated on the way (as in qk_norm_rope); with q and
        q_out, the queries are normalised and rotated in the same launch.
        Slots outside the cache (-1, say) are not stored.  Returns the
        caches."""
        _forward_only(k, v, q, q_weight, k_weight)
        dtype = k.dtype
        if dtype not in _DTYPE16 or k.dim() != 3 or k_cache.dim() != 4:
            raise ValueError("k must be [tokens, heads, dim] in bfloat16 or float16, caches "
                             "[pages, heads, page, dim]")
        T, Hk, D = ks = k.shape
        pages, ch, page, cd = cs = k_cache.shape
        if ch != Hk or cd != D:
            raise ValueError(f"caches must be [pages, {Hk}, page, {D}], got {list(cs)}")
        kind = _cache_type(k_cache, dtype, k_scale, v_scale)
        cdt = torch.float8_e4m3fn if kind == 2 else dtype
        if q is None:
            Hq, qp, qo = 0, _NO, _NO
            if q_out is not None or q_weight is not None:
                raise ValueError("q_out and q_weight need q")
        else:
            if q.dim() != 3 or q.shape[0] != T or q.shape[2] != D:
                raise ValueError(f"q must be [{T}, heads, {D}], got {list(q.shape)}")
            if q_out is None:
                raise ValueError("q needs q_out")
            Hq = q.shape[1]
            qp, qo = _heads("q", q, q.shape, dtype), _heads("q_out", q_out, q.shape, dtype)
        args = _HEADS.pack(
            _DTYPE16[dtype], T, D, Hq, *qp, *qo, Hk, *_heads("k", k, ks, dtype), *_NO,
            *_heads("v", v, ks, dtype), *_cache("k_cache", k_cache, cs, cdt),
            *_cache("v_cache", v_cache, cs, cdt), kind, pages, page,
            _flat("k_scale", k_scale, Hk, torch.float32),
            _flat("v_scale", v_scale, Hk, torch.float32), _flat("slots", slots, T, torch.int32),
            *self._rope_part(T, dtype, D, cos_sin, positions, q_weight, k_weight, eps,
                             interleaved))
        rc = self._lib.lin_gemm_kv_append(self._h, args, _stream_of(stream, k))
        if rc:
            self._check(rc, "lin_gemm_kv_append")
        return k_cache, v_cache

    def _attention_part(self, q, k_cache, v_cache, out, page_table, context, offsets, max_context,
                        max_nodes, mask, scale, k_scale, v_scale, lse):
        dtype = q.dtype
        if dtype not in _DTYPE16 or q.dim() != 3 or k_cache.dim() != 4 or page_table.dim() != 2:
            raise ValueError("q must be [tokens, heads, dim] in bfloat16 or float16, caches "
                             "[pages, heads, page, dim], page_table [sequences, pages]")
        T, Hq, D = qs = q.shape
        pages, Hk, page, cd = cs = k_cache.shape
        if cd != D:
            raise ValueError(f"caches must be [pages, heads, page, {D}], got {list(cs)}")
        B, mp = page_table.shape
        if page_table.dtype is not torch.int32 or (mp > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be int32 with contiguous rows")
        kind = _cache_type(k_cache, dtype, k_scale, v_scale)
        cdt = torch.float8_e4m3fn if kind == 2 else dtype
        words, mp_at = 0, 0
        if mask is not None:
            if mask.dim() != 2 or mask.shape[0] != T:
                raise ValueError(f"mask must be [{T}, words], got {list(mask.shape)}")
            words = mask.shape[1]
            if words * 64 < max_nodes:
                raise ValueError(f"mask of {words} words for up to {max_nodes} nodes")
            mp_at = _flat("mask", mask, T * words, torch.int64)
        return (
            _DTYPE16[dtype], T, Hq, Hk, D, *_heads("q", q, qs, dtype),
            *_cache("k_cache", k_cache, cs, cdt), *_cache("v_cache", v_cache, cs, cdt), kind, pages,
            page, _flat("k_scale", k_scale, Hk, torch.float32),
            _flat("v_scale", v_scale, Hk, torch.float32), B, _at("page_table", page_table),
            page_table.stride(0) if B > 1 else mp, mp, _flat("context", context, B, torch.int32),
            _flat("offsets", offsets, B + 1, torch.int32), int(max_context), int(max_nodes),
            mp_at, words, 1.0 / math.sqrt(D) if scale is None else float(scale),
            _flat("out", out, T * Hq * D, dtype), _flat("lse", lse, T * Hq, torch.float32))

    def tree_attention(self, q, k_cache, v_cache, out, page_table, context, offsets, max_context,
                       max_nodes, mask=None, scale=None, k_scale=None, v_scale=None, lse=None,
                       stream=None):
        """Attention of nodes q [T, Hq, dim] over their sequences' caches.

        page_table [B, pages per sequence], context [B] (cached tokens before
        the nodes, whose own keys and values follow them in the cache),
        offsets [B + 1].  max_context and max_nodes bound the two; they shape
        the launch only.  mask int64 [T, words]: bit j % 64 of word j // 64
        says that the node sees node j of its sequence (see tree_mask);
        without one it sees itself and the nodes before it.  scale: 1 /
        sqrt(dim) unless given.  out [T, Hq, dim] and lse [T, Hq] (fp32,
        optional) are contiguous.  Returns out."""
        _forward_only(q)
        args = _ATTENTION.pack(*self._attention_part(
            q, k_cache, v_cache, out, page_table, context, offsets, max_context, max_nodes, mask, scale,
            k_scale, v_scale, lse))
        rc = self._lib.lin_gemm_tree_attention(self._h, args, _stream_of(stream, q))
        if rc:
            self._check(rc, "lin_gemm_tree_attention")
        return out

    def window_attention(self, q, k_cache, v_cache, out, page_table, context, offsets, max_context,
                         max_nodes, window, sinks=0, mask=None, positions=None, scale=None,
                         k_scale=None, v_scale=None, lse=None, stream=None):
        """tree_attention of layers with a sliding window: of the cached
        positions a node at position p sees those below `sinks` and those
        above p - window (its own among them).  Without a mask p is context +
        node; nodes with a mask have positions int32 [T] (context + depth,
        see tree_mask; context + node without), see the nodes that the mask
        names and of the context what the window leaves.  Pages that no node
        sees may have been dropped: their table entries are not looked at
        beyond the 128 positions around the visible ones, which may hold
        anything.  Returns out."""
        _forward_only(q)
        part = self._attention_part(
            q, k_cache, v_cache, out, page_table, context, offsets, max_context, max_nodes, mask, scale,
            k_scale, v_scale, lse)
        if positions is not None and mask is None:
            raise ValueError("positions are for nodes with a mask: others follow the context")
        args = _WINDOW.pack(*part, int(window), int(sinks),
                            _flat("positions", positions, q.shape[0], torch.int32))
        rc = self._lib.lin_gemm_window_attention(self._h, args, _stream_of(stream, q))
        if rc:
            self._check(rc, "lin_gemm_window_attention")
        return out

    def token_logprobs(self, logits, tokens, logprobs, entropy=None, top_ids=None,
                       top_logprobs=None, temperature=1.0, stream=None):
        """Log probabilities of tokens [T] under logits [T, V] / temperature
        (bf16, fp16 or fp32; rows may lie apart), with the entropy [T] of each
        row and its most likely tokens: top_ids int32 and top_logprobs fp32
        [T, k], k up to 32, ties to the lower index.  Outputs are fp32 unless
        said, contiguous, optional but for logprobs.  Returns logprobs."""
        _forward_only(logits)
        if logits.dtype not in _SCORE_DTYPE or logits.dim() != 2:
            raise ValueError("logits must be [rows, vocab] in bfloat16, float16 or float32")
        T, V = logits.shape
        if V > 1 and logits.stride(1) != 1:
            raise ValueError("the logits of a row must be contiguous")
        tops = top_ids if top_ids is not None else top_logprobs
        k = 0
        if tops is not None:
            if tops.dim() != 2 or tops.shape[0] != T:
                raise ValueError(f"top_ids and top_logprobs must be [{T}, k]")
            k = tops.shape[1]
        args = _SCORE.pack(
            _SCORE_DTYPE[logits.dtype], T, V, _at("logits", logits),
            logits.stride(0) if T > 1 else V, _flat("tokens", tokens, T, torch.int32),
            float(temperature), _flat("logprobs", logprobs, T, torch.float32),
            _flat("entropy", entropy, T, torch.float32), k,
            _flat("top_ids", top_ids, T * k, torch.int32),
            _flat("top_logprobs", top_logprobs, T * k, torch.float32))
        rc = self._lib.lin_gemm_token_logprobs(self._h, args, _stream_of(stream, logits))
        if rc:
            self._check(rc, "lin_gemm_token_logprobs")
        return logprobs

    def add_rms_norm(self, x, weight, residual=None, residual_out=None, out=None, codes=None,
                     scales=None, kind="fp8_token", eps=1e-6, stream=None):
        """Norm of s = x + residual (x alone without one) over rows [T, N]:
        residual_out = s, out = s / sqrt(mean(s^2) + eps) * weight, and the
        codes [T, N] of the unrounded out with their scales, as in quantize
        (kind "fp8_token" or "int8_token": scales [T]; "fp8_block": scales
        [T, N / 128]).  Outputs that are None are not computed; one at
        least is asked for.  residual_out and out may be x or the residual
        themselves.  Returns (residual_out, out, codes, scales)."""
        _forward_only(x, weight, residual)
        dtype = x.dtype
        if dtype not in _DTYPE16 or x.dim() != 2:
            raise ValueError("x must be [rows, width] in bfloat16 or float16")
        T, N = shape = x.shape
        if kind not in _NORM_KIND:
            raise ValueError(f"kind must be one of {sorted(_NORM_KIND)}, got {kind!r}")
        code, cdt = _NORM_KIND[kind]
        if (codes is None) != (scales is None):
            raise ValueError("codes need scales, and scales codes")
        args = _NORM.pack(
            _DTYPE16[dtype], T, N, *_rows("x", x, shape, dtype),
            *_rows("residual", residual, shape, dtype),
            *_rows("residual_out", residual_out, shape, dtype),
            _flat("weight", weight, N, dtype), float(eps), *_rows("out", out, shape, dtype), code,
            _flat("codes", codes, T * N, cdt),
            _flat("scales", scales, T * (N // 128) if code == 2 else T, torch.float32))
        rc = self._lib.lin_gemm_add_rms_norm(self._h, args, _stream_of(stream, x))
        if rc:
            self._check(rc, "lin_gemm_add_rms_norm")
        return residual_out, out, codes, scales

    def lora_add(self, x, a, b, ids, out, base=None, factors=None, slices=None, stream=None):
        """Low-rank adapters beside a shared projection: out [T, N] = base +
        factors[i] (x a[i]^T) b[i]^T with i = ids[t].

        x [T, K], a [adapters, rank, K], b [adapters, N, rank], ids int32
        [T] (outside [0, adapters): the row has no adapter), factors fp32
        [adapters] (1 without).  base is the shared projection's output [T,
        N], or None for 0; out may be base.  slices: the widths of up to
        four parts of the N columns that have adapters of their own, as in
        a QKV product; a is then [adapters, slices * rank, K], the first
        rank rows for the first part.  Returns out."""
        _forward_only(x, a, b, base, factors)
        dtype = x.dtype
        if dtype not in _DTYPE16 or x.dim() != 2 or a.dim() != 3 or b.dim() != 3 or out.dim() != 2:
            raise ValueError("x must be [rows, inner] in bfloat16 or float16, a [adapters, slices * "
                             "rank, inner], b [adapters, width, rank], out [rows, width]")
        T, K = x.shape
        n, N, R = b.shape
        widths = (N,) if slices is None else tuple(int(w) for w in slices)
        if not 1 <= len(widths) <= 4 or sum(widths) != N:
            raise ValueError(f"slices must be up to four widths that add up to {N}, got {slices}")
        if a.shape != (n, len(widths) * R, K):
            raise ValueError(f"a must be {[n, len(widths) * R, K]}, got {list(a.shape)}")
        args = _LORA.pack(
            _DTYPE16[dtype], T, K, N, R, *_rows("x", x, x.shape, dtype), n,
            _flat("a", a, a.numel(), dtype), _flat("b", b, b.numel(), dtype),
            _flat("ids", ids, T, torch.int32), _flat("factors", factors, n, torch.float32),
            *_rows("base", base, (T, N), dtype), *_rows("out", out, (T, N), dtype), len(widths),
            *(widths + (0, 0, 0))[:4])
        rc = self._lib.lin_gemm_lora_add(self._h, args, _stream_of(stream, x))
        if rc:
            self._check(rc, "lin_gemm_lora_add")
        return out


# ------------------------------------------------------------------- plans

def rope_table(positions, rope_dim, theta=10000.0, device="cuda"):
    """cos_sin [positions, rope_dim] fp32 of the usual frequencies theta^(-2i /
    rope_dim): cosines, then sines.  The angles are formed in 64 bits, so far
    positions keep their phase."""
    inv = float(theta) ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / rope_dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * inv[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def tree_mask(parents, device="cuda"):
    """(mask int64 [T, words], depth int32 [T]) of drafted trees.

    parents: one list per sequence, parents[b][i] the node that node i
    follows (an earlier one), or -1 where it follows the context directly.  A
    node sees itself and its ancestors; depth is its distance from the
    context (0 for the first), so its position is context + depth."""
    words = max(1, max(((len(p) + 63) // 64 for p in parents), default=1))
    rows, depth = [], []
    for p in parents:
        seen, at = [], []
        for i, up in enumerate(p):
            if not -1 <= up < i:
                raise ValueError(f"node {i} cannot follow node {up}: parents come first")
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
            at.append(at[up] + 1 if up >= 0 else 0)
        rows += seen
        depth += at
    split = [[(r >> 64 * w) & (2 ** 64 - 1) for w in range(words)] for r in rows]
    signed = [[x - 2 ** 64 if x >= 2 ** 63 else x for x in r] for r in split]
    mask = torch.tensor(signed, dtype=torch.int64).reshape(len(rows), words)
    return mask.to(device), torch.tensor(depth, dtype=torch.int32).to(device)


def node_slots(page_table, context, offsets, page_size):
    """Cache slots int32 [T] of the nodes: node j of sequence b at position
    context[b] + j of its pages, or -1 (not stored) past the page table and
    at table entries below 0.  Elementary torch operations on the plans'
    device; T comes from offsets[-1]."""
    T = int(offsets[-1])
    t = torch.arange(T, device=offsets.device)
    b = torch.searchsorted(offsets[1:].contiguous(), t.to(offsets.dtype), right=True)
    pos = context[b].long() + t - offsets[b].long()
    at = pos // page_size
    last = page_table.shape[1] - 1
    page = page_table[b, at.clamp(0, last)].long()
    slot = page * page_size + pos % page_size
    return torch.where((at >= 0) & (at <= last) & (page >= 0), slot, -1).to(torch.int32)
