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
_DTYPE16 = {torch.bfloat16: 0, torch.float16: 1}
_SCORE_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_NO = (0, 0, 0)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def declare(lib):
    """Argument types of the serving entry points."""
    for name in ("qk_norm_rope", "kv_append", "tree_attention", "token_logprobs"):
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
        args = _ATTENTION.pack(
            _DTYPE16[dtype], T, Hq, Hk, D, *_heads("q", q, qs, dtype),
            *_cache("k_cache", k_cache, cs, cdt), *_cache("v_cache", v_cache, cs, cdt), kind, pages,
            page, _flat("k_scale", k_scale, Hk, torch.float32),
            _flat("v_scale", v_scale, Hk, torch.float32), B, _at("page_table", page_table),
            page_table.stride(0) if B > 1 else mp, mp, _flat("context", context, B, torch.int32),
            _flat("offsets", offsets, B + 1, torch.int32), int(max_context), int(max_nodes),
            mp_at, words, 1.0 / math.sqrt(D) if scale is None else float(scale),
            _flat("out", out, T * Hq * D, dtype), _flat("lse", lse, T * Hq, torch.float32))
        rc = self._lib.lin_gemm_tree_attention(self._h, args, _stream_of(stream, q))
        if rc:
            self._check(rc, "lin_gemm_tree_attention")
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
