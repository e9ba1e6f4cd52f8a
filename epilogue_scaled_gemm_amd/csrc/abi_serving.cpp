// abi_serving.cpp -- the extern "C" entry points of the serving operators
// (include/lin_gemm.h): argument checks on the host, then one or two launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>

#include "../../include/lin_gemm.h"
#include "handle.hpp"
#include "launch.hpp"

using lg::fail;
using lg::grow_size;
using lg::hip_fail;
using lg::misaligned;

namespace {

// Launches stay below 2^32 threads.
constexpr int64_t kMaxTokens = (int64_t)1 << 23;
constexpr int64_t kMaxGroups = (int64_t)1 << 23;
constexpr double kLog2e = 1.4426950408889634;

bool bad4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3) != 0; }

bool any_not_multiple(int64_t m, std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x % m != 0) return true;
  return false;
}

int log2_exact(int64_t v) {
  int l = 0;
  while (((int64_t)1 << l) < v) ++l;
  return ((int64_t)1 << l) == v ? l : -1;
}

// Nothing throws across the C boundary.
template <typename F> int guarded(lin_gemm_t h, F&& f) {
  if (!h) return LIN_ERR_INVALID_ARG;
  try {
    h->last_error.clear();
    return f();
  } catch (const std::bad_alloc&) {
    return LIN_ERR_OOM;
  } catch (...) {
    return LIN_ERR_HIP;
  }
}

int check_cache(lin_gemm_t h, int64_t dtype, int64_t type, int64_t pages, int64_t page_size,
                const void* k, const void* v, std::initializer_list<int64_t> strides) {
  if (type < LIN_CACHE_BF16 || type > LIN_CACHE_E4M3)
    return fail(h, LIN_ERR_INVALID_ARG, "unknown cache type " + std::to_string(type));
  if (type != LIN_CACHE_E4M3 && type != dtype)
    return fail(h, LIN_ERR_UNSUPPORTED, "a 16-bit cache must have the heads' type");
  if (pages < 1 || page_size < 1) return fail(h, LIN_ERR_INVALID_ARG, "an empty cache");
  if (log2_exact(page_size) < 0)
    return fail(h, LIN_ERR_UNSUPPORTED, "page_size must be a power of two");
  if (page_size > ((int64_t)1 << 30) || pages > ((int64_t)1 << 30) / page_size)
    return fail(h, LIN_ERR_UNSUPPORTED, "more than 2^30 cache slots");
  if (!k || !v) return fail(h, LIN_ERR_INVALID_ARG, "null cache");
  if (misaligned(k) || misaligned(v) ||
      any_not_multiple(type == LIN_CACHE_E4M3 ? 16 : 8, strides))
    return fail(h, LIN_ERR_UNSUPPORTED, "caches and their strides must be multiples of 16 bytes");
  return LIN_OK;
}

int run_heads(lin_gemm_t h, const lin_heads_t* p, bool append, hipStream_t s) {
  if (!p) return fail(h, LIN_ERR_INVALID_ARG, "null arguments");
  if (p->dtype != LIN_Q_BF16 && p->dtype != LIN_Q_FP16)
    return fail(h, LIN_ERR_INVALID_ARG, "dtype must be LIN_Q_BF16 or LIN_Q_FP16");
  if (p->tokens < 0 || p->q_heads < 0 || p->kv_heads < 0)
    return fail(h, LIN_ERR_INVALID_ARG, "negative size");
  if (p->dim < 16 || p->dim > 256 || p->dim % 16 != 0)
    return fail(h, LIN_ERR_UNSUPPORTED, "dim must be a multiple of 16 from 16 to 256");
  if (p->tokens > kMaxTokens || p->q_heads > 4096 || p->kv_heads > 4096)
    return fail(h, LIN_ERR_UNSUPPORTED, "more than 2^23 tokens or 4096 heads");
  if (append && p->kv_heads < 1) return fail(h, LIN_ERR_INVALID_ARG, "no key heads");
  if (!(p->eps >= 0) || !std::isfinite(p->eps))
    return fail(h, LIN_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (p->rope) {
    if (p->rope_dim < 16 || p->rope_dim > p->dim || p->rope_dim % 16 != 0)
      return fail(h, LIN_ERR_UNSUPPORTED, "rope_dim must be a multiple of 16 from 16 to dim");
    if (p->rope_rows < 1 || p->rope_rows > (int64_t)1 << 30)
      return fail(h, LIN_ERR_INVALID_ARG, "rope_rows must be in 1 .. 2^30");
    if (!p->positions && p->tokens > 0)
      return fail(h, LIN_ERR_INVALID_ARG, "a rotation needs positions");
  }
  if (append) {
    int rc = check_cache(h, p->dtype, p->cache_type, p->pages, p->page_size, p->k_cache, p->v_cache,
                         {p->k_page_stride, p->k_cache_head_stride, p->k_in_page_stride,
                          p->v_page_stride, p->v_cache_head_stride, p->v_in_page_stride});
    if (rc != LIN_OK) return rc;
  }
  if (p->tokens == 0 || p->q_heads + p->kv_heads == 0) return LIN_OK;
  if (p->q_heads > 0 && (!p->q || !p->q_out)) return fail(h, LIN_ERR_INVALID_ARG, "null q or q_out");
  if (p->kv_heads > 0 && (!p->k || (append ? !p->v || !p->slots : !p->k_out)))
    return fail(h, LIN_ERR_INVALID_ARG, append ? "null k, v or slots" : "null k or k_out");
  if (misaligned(p->q) || misaligned(p->k) || misaligned(p->q_out) || misaligned(p->q_weight) ||
      misaligned(p->k_weight) || misaligned(p->rope) ||
      (append ? misaligned(p->v) : misaligned(p->k_out)) ||
      any_not_multiple(8, {p->q_token_stride, p->q_head_stride, p->q_out_token_stride,
                           p->q_out_head_stride, p->k_token_stride, p->k_head_stride}) ||
      (append ? any_not_multiple(8, {p->v_token_stride, p->v_head_stride})
              : any_not_multiple(8, {p->k_out_token_stride, p->k_out_head_stride})))
    return fail(h, LIN_ERR_UNSUPPORTED, "head tensors and strides must be multiples of 16 bytes");
  if (bad4(p->positions) || (append && (bad4(p->slots) || bad4(p->k_scale) || bad4(p->v_scale))))
    return fail(h, LIN_ERR_UNSUPPORTED, "positions, slots and scales must be 4-byte aligned");

  lg::HeadArgs a{};
  a.Hq = (int)p->q_heads;
  a.Hk = (int)p->kv_heads;
  a.D = (int)p->dim;
  a.q = {(void*)p->q, 0, p->q_token_stride, p->q_head_stride};
  a.k = {(void*)p->k, 0, p->k_token_stride, p->k_head_stride};
  a.q_out = {p->q_out, 0, p->q_out_token_stride, p->q_out_head_stride};
  a.q_weight = (const uint16_t*)p->q_weight;
  a.k_weight = (const uint16_t*)p->k_weight;
  a.eps = (float)p->eps;
  a.table = p->rope;
  a.rot = (int)(p->rope ? p->rope_dim : 0);
  a.max_pos = (int)(p->rope ? p->rope_rows : 0);
  a.positions = p->positions;
  a.interleaved = p->interleaved != 0;
  if (append) {
    a.Hv = a.Hk;
    a.v = {(void*)p->v, 0, p->v_token_stride, p->v_head_stride};
    a.kc = {p->k_cache, p->k_page_stride, p->k_in_page_stride, p->k_cache_head_stride};
    a.vc = {p->v_cache, p->v_page_stride, p->v_in_page_stride, p->v_cache_head_stride};
    a.slots = p->slots;
    a.capacity = p->pages * p->page_size;
    a.page_log = log2_exact(p->page_size);
    a.cache8 = p->cache_type == LIN_CACHE_E4M3;
    if (a.cache8) {
      a.k_scale = p->k_scale;
      a.v_scale = p->v_scale;
    }
  } else {
    a.k_out = {p->k_out, 0, p->k_out_token_stride, p->k_out_head_stride};
  }
  hipError_t e = lg::launch_heads(a, p->tokens, p->dtype == LIN_Q_FP16, s);
  return e == hipSuccess ? LIN_OK : hip_fail(h, e, "heads kernel launch");
}

// The handle's workspace holds at least `need` bytes.
int ensure_bytes(lin_gemm_t h, size_t need, hipStream_t s) {
  if (need <= h->ws_bytes) return LIN_OK;
  hipError_t e = hipStreamSynchronize(s);  // in-flight calls may still use the old buffer
  if (e != hipSuccess) return hip_fail(h, e, "hipStreamSynchronize");
  if (h->ws) h->retired.push_back(h->ws);
  h->ws = nullptr;
  h->ws_bytes = 0;
  const size_t bytes = grow_size(need);
  h->ws = lg::device_alloc(bytes);
  if (!h->ws)
    return fail(h, LIN_ERR_OOM, "workspace allocation of " + std::to_string(bytes) + " bytes failed");
  h->ws_bytes = bytes;
  return LIN_OK;
}

// The handle's arrival counters (at zero between calls) are at least n.
int ensure_counters(lin_gemm_t h, size_t n, hipStream_t s) {
  if (n <= h->counters_n) return LIN_OK;
  hipError_t e = hipStreamSynchronize(s);  // in-flight calls may still use the old ones
  if (e != hipSuccess) return hip_fail(h, e, "hipStreamSynchronize");
  if (h->counters) h->retired.push_back(h->counters);
  h->counters = nullptr;
  h->counters_n = 0;
  const size_t bytes = grow_size(n * sizeof(int));
  h->counters = (int*)lg::device_alloc(bytes);
  if (!h->counters) return fail(h, LIN_ERR_OOM, "arrival counter allocation failed");
  e = lg::launch_fill_zero(h->counters, bytes, s);
  if (e != hipSuccess) return hip_fail(h, e, "counter zero fill");
  h->counters_n = bytes / sizeof(int);
  return LIN_OK;
}

int run_attention(lin_gemm_t h, const lin_attention_t* p, hipStream_t s) {
  if (!p) return fail(h, LIN_ERR_INVALID_ARG, "null arguments");
  if (p->dtype != LIN_Q_BF16 && p->dtype != LIN_Q_FP16)
    return fail(h, LIN_ERR_INVALID_ARG, "dtype must be LIN_Q_BF16 or LIN_Q_FP16");
  if (p->tokens < 0 || p->sequences < 0 || p->max_context < 0 || p->max_nodes < 0 ||
      p->mask_words < 0)
    return fail(h, LIN_ERR_INVALID_ARG, "negative size");
  if (p->dim != 64 && p->dim != 128 && p->dim != 256)
    return fail(h, LIN_ERR_UNSUPPORTED, "dim must be 64, 128 or 256");
  if (p->kv_heads < 1 || p->q_heads < 1 || p->q_heads % p->kv_heads != 0)
    return fail(h, LIN_ERR_UNSUPPORTED, "q_heads must be a positive multiple of kv_heads");
  if (p->tokens > kMaxTokens || p->q_heads > 4096 || p->sequences > 65535)
    return fail(h, LIN_ERR_UNSUPPORTED, "more than 2^23 tokens, 4096 heads or 65535 sequences");
  if (p->tokens > ((int64_t)1 << 25) / p->q_heads)
    return fail(h, LIN_ERR_UNSUPPORTED, "more than 2^25 rows of one head");
  if (!std::isfinite((float)(p->scale * kLog2e)))  // (what the kernels hold)
    return fail(h, LIN_ERR_INVALID_ARG, "scale must be finite, in binary32 too");
  int rc = check_cache(h, p->dtype, p->cache_type, p->pages, p->page_size, p->k_cache, p->v_cache,
                       {p->k_page_stride, p->k_head_stride, p->k_in_page_stride, p->v_page_stride,
                        p->v_head_stride, p->v_in_page_stride});
  if (rc != LIN_OK) return rc;
  if (p->tokens == 0 || p->sequences == 0) return LIN_OK;
  if (!p->q || !p->out || !p->page_table || !p->context || !p->offsets)
    return fail(h, LIN_ERR_INVALID_ARG, "null q, out, page_table, context or offsets");
  if (p->max_pages < 1 || p->table_stride < p->max_pages ||
      p->max_pages > ((int64_t)1 << 30) / p->page_size)
    return fail(h, LIN_ERR_INVALID_ARG, "the page table needs 1 .. 2^30 / page_size pages a row");
  if (p->mask_words > ((int64_t)1 << 20))
    return fail(h, LIN_ERR_UNSUPPORTED, "more than 2^20 mask words");
  // The kernels step within a page with 32-bit byte offsets.
  for (int64_t x : {p->k_page_stride, p->v_page_stride})
    if (x < 0 || x >= ((int64_t)1 << 30))
      return fail(h, LIN_ERR_UNSUPPORTED, "page strides must be in [0, 2^30)");
  for (int64_t x : {p->k_in_page_stride, p->v_in_page_stride})
    if (x < 0 || x >= ((int64_t)1 << 30) / p->page_size)
      return fail(h, LIN_ERR_UNSUPPORTED, "a page must span less than 2^30 values");
  if (misaligned(p->q) || misaligned(p->out) ||
      any_not_multiple(8, {p->q_token_stride, p->q_head_stride}))
    return fail(h, LIN_ERR_UNSUPPORTED, "q, out and strides must be multiples of 16 bytes");
  if (bad4(p->page_table) || bad4(p->context) || bad4(p->offsets) || bad4(p->lse) ||
      bad4(p->k_scale) || bad4(p->v_scale) || (reinterpret_cast<uintptr_t>(p->mask) & 7))
    return fail(h, LIN_ERR_UNSUPPORTED, "plans must be 4-byte aligned, masks 8-byte aligned");

  lg::AttnArgs a{};
  a.q = (const uint16_t*)p->q;
  a.k = p->k_cache;
  a.v = p->v_cache;
  a.out = (uint16_t*)p->out;
  a.lse = p->lse;
  a.table = p->page_table;
  a.context = p->context;
  a.offsets = p->offsets;
  a.mask = p->mask;
  const bool kv8 = p->cache_type == LIN_CACHE_E4M3;
  if (kv8) {
    a.k_scale = p->k_scale;
    a.v_scale = p->v_scale;
  }
  a.q_ts = p->q_token_stride;
  a.q_hs = p->q_head_stride;
  a.k_ps = p->k_page_stride;
  a.k_hs = p->k_head_stride;
  a.k_ts = p->k_in_page_stride;
  a.v_ps = p->v_page_stride;
  a.v_hs = p->v_head_stride;
  a.v_ts = p->v_in_page_stride;
  a.T = p->tokens;
  a.rows = p->tokens * p->q_heads;
  a.table_stride = p->table_stride;
  a.Hk = (int)p->kv_heads;
  a.G = (int)(p->q_heads / p->kv_heads);
  a.mask_words = (int)p->mask_words;
  a.max_pages = (int)p->max_pages;
  a.pages = (int)p->pages;
  a.page_log = log2_exact(p->page_size);
  a.page_mask = (int)p->page_size - 1;
  a.scale_log2e = (float)(p->scale * kLog2e);
  // The bounds shape the launch: at least one node and one position, at most
  // what the tensors can hold.
  const int64_t nodes = std::min(std::max<int64_t>(p->max_nodes, 1), p->tokens);
  const int64_t room = p->max_pages * p->page_size;
  const int64_t len = std::min(std::min(p->max_context, room) + nodes, room);
  const lg::AttnPlan plan = lg::attn_plan(p->sequences, a.Hk, a.G, (int)p->dim, nodes, len, a.rows);
  const int64_t work = p->sequences * a.Hk * plan.nsplit;
  if (work > kMaxGroups / plan.ntiles - 8)
    return fail(h, LIN_ERR_UNSUPPORTED, "too many workgroups for one launch");
  a.nwork = (int)work;
  a.ntiles = (int)plan.ntiles;
  a.nsplit = (int)plan.nsplit;
  a.chunk = (int)plan.chunk;
  if (a.nsplit > 1) {
    const size_t n = (size_t)a.nsplit * (size_t)a.rows;
    rc = ensure_bytes(h, n * (size_t)(p->dim + 2) * sizeof(float), s);
    if (rc != LIN_OK) return rc;
    a.part_o = (float*)h->ws;
    a.part_ml = a.part_o + n * (size_t)p->dim;
    if (plan.arrival) {
      rc = ensure_counters(h, (size_t)(p->sequences * a.Hk) * (size_t)a.ntiles * lg::AT_COUNTER_STEP, s);
      if (rc != LIN_OK) return rc;
      a.counters = h->counters;
    }
  }
  hipError_t e = lg::launch_attention(a, (int)p->dim, plan.shape, p->dtype == LIN_Q_FP16, kv8, s);
  return e == hipSuccess ? LIN_OK : hip_fail(h, e, "attention launch");
}

int run_score(lin_gemm_t h, const lin_score_t* p, hipStream_t s) {
  if (!p) return fail(h, LIN_ERR_INVALID_ARG, "null arguments");
  if (p->dtype < 0 || p->dtype > 2)
    return fail(h, LIN_ERR_INVALID_ARG, "dtype must be 0 (bf16), 1 (fp16) or 2 (fp32)");
  if (p->rows < 0 || p->vocab < 0 || p->top < 0)
    return fail(h, LIN_ERR_INVALID_ARG, "negative size");
  // its inverse is a factor of the logits: an infinite one would make NaN of
  // the largest, one of zero of those that are masked with -inf
  const float per_logit = (float)(kLog2e / p->temperature);
  if (!(per_logit > 0) || !std::isfinite(per_logit))
    return fail(h, LIN_ERR_INVALID_ARG,
                "temperature must be positive, and log2(e) over it within binary32");
  if (p->top > lg::SCORE_MAX_TOP || p->top > p->vocab)
    return fail(h, LIN_ERR_UNSUPPORTED, "top must be at most 32 and at most vocab");
  if (p->rows > kMaxTokens || p->vocab > ((int64_t)1 << 30))
    return fail(h, LIN_ERR_UNSUPPORTED, "more than 2^23 rows or 2^30 tokens");
  if (p->rows == 0) return LIN_OK;
  if (p->vocab < 1) return fail(h, LIN_ERR_UNSUPPORTED, "an empty vocabulary");
  if (!p->logits || !p->tokens || !p->logprobs)
    return fail(h, LIN_ERR_INVALID_ARG, "null logits, tokens or logprobs");
  if (p->row_stride < p->vocab && p->rows > 1)
    return fail(h, LIN_ERR_INVALID_ARG, "row_stride below vocab");
  if ((reinterpret_cast<uintptr_t>(p->logits) & (p->dtype == 2 ? 3 : 1)) || bad4(p->tokens) ||
      bad4(p->logprobs) || bad4(p->entropy) || bad4(p->top_ids) || bad4(p->top_logprobs))
    return fail(h, LIN_ERR_UNSUPPORTED, "operands must be aligned to their elements");
  lg::ScoreArgs a{};
  a.logits = p->logits;
  a.tokens = p->tokens;
  a.logprobs = p->logprobs;
  a.entropy = p->entropy;
  a.top_ids = p->top_ids;
  a.top_logprobs = p->top_logprobs;
  a.T = p->rows;
  a.V = p->vocab;
  a.stride = p->row_stride;
  a.k = p->top_ids || p->top_logprobs ? (int)p->top : 0;
  a.c = per_logit;
  a.inv_t = (float)(1.0 / p->temperature);
  lg::score_plan(a.T, a.V, (int)p->dtype, &a.nsplit, &a.slice);
  if (a.nsplit > 1) {
    const size_t n = (size_t)a.T * (size_t)a.nsplit;
    const size_t keys = (n * (size_t)a.k * 8 + 255) & ~(size_t)255;
    int rc = ensure_bytes(h, keys + n * 3 * sizeof(float), s);
    if (rc != LIN_OK) return rc;
    a.part_keys = (uint64_t*)h->ws;
    a.part_sums = (float*)((char*)h->ws + keys);
    rc = ensure_counters(h, (size_t)a.T * lg::SCORE_COUNTER_STEP, s);
    if (rc != LIN_OK) return rc;
    a.counters = h->counters;
  }
  hipError_t e = lg::launch_score(a, (int)p->dtype, s);
  return e == hipSuccess ? LIN_OK : hip_fail(h, e, "log-probability launch");
}

}  // namespace

extern "C" {

int lin_gemm_qk_norm_rope(lin_gemm_t h, const lin_heads_t* args, void* stream) {
  return guarded(h, [&] { return run_heads(h, args, false, (hipStream_t)stream); });
}

int lin_gemm_kv_append(lin_gemm_t h, const lin_heads_t* args, void* stream) {
  return guarded(h, [&] { return run_heads(h, args, true, (hipStream_t)stream); });
}

int lin_gemm_tree_attention(lin_gemm_t h, const lin_attention_t* args, void* stream) {
  return guarded(h, [&] { return run_attention(h, args, (hipStream_t)stream); });
}

int lin_gemm_token_logprobs(lin_gemm_t h, const lin_score_t* args, void* stream) {
  return guarded(h, [&] { return run_score(h, args, (hipStream_t)stream); });
}

}  // extern "C"
