// kernels_attn.hip -- attention of drafted tokens over a paged cache.
//
//   o[t, h] = sum_j p_j v_j,   p = softmax_j(scale * q[t, h] . k_j)
//
// over the cached positions j that node t of its sequence sees: all of the
// context, and the drafted nodes its mask names (or, without a mask, itself
// and the nodes before it).  A plain decode step is one node per sequence.
//
// One pass over the keys and values with a running maximum m, sum l and
// weighted value sum O (exp2 of scores that carry log2 e):
//   m' = max(m, s),  l' = l 2^(m - m') + sum 2^(s - m'),  O likewise.
//
// Scores are formed transposed, S^T = K Q^T, by MFMA: a lane then holds
// scores of ONE row, so the row statistics are register reductions and a few
// lane swaps, and the rounded probabilities are already the B operand of
// O^T = V^T P^T -- the contraction order over positions is permuted the same
// way on the V side, whose fragments come from LDS by transposing reads.  The
// rows of one key head (its nodes times the query heads that share it) are
// packed into one tile, so a key is read once for all heads of a group.
//
// Two kernels, by the number of those rows:
//  - stream_kernel (few rows: decode steps and small trees; bound by reading
//    the cache): every wave runs through positions of its own, 32 at a time,
//    without barriers: keys go from memory straight into MFMA operands,
//    values through the wave's own LDS.
//  - tile_kernel (many rows: large trees, parts of prompts; bound by a wait
//    for its loads in every step, see there): 32 rows per wave, all waves
//    share each tile of positions in LDS.
// Long contexts are split over workgroups; those write (m, l, O) in 32 bits,
// and join_kernel, or of few workgroups the last to arrive, joins them.
#include <type_traits>

#include "launch.hpp"

#define ALWAYS_INLINE __attribute__((always_inline))

namespace lg {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) char lds_char;

typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

constexpr float NEG_INF = -__builtin_inff();

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum / sum of the two lanes l and l ^ 32.
__device__ inline float half_max(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float half_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <bool F16> __device__ inline f32x16 mfma32(i32x4 a, i32x4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two e4m3 codes (bytes 2 HI and 2 HI + 1 of w) -> packed 16-bit floats, exact.
template <bool F16, bool HI> __device__ inline int widen2(int w) {
  if constexpr (F16) {
    typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
    f16x2 r = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w, 1.0f, HI);
    return __builtin_bit_cast(int, r);
  } else {
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)w, 1.0f, HI);
    return __builtin_bit_cast(int, r);
  }
}

// Whether one of the two 16-bit floats of w is infinite or NaN.
template <bool F16> __device__ inline bool not_finite2(int w) {
  constexpr int E = F16 ? 0x7C00 : 0x7F80;
  return (w & E) == E || ((w >> 16) & E) == E;
}

// Maximum / sum of the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ inline float quad_max(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ inline float quad_sum(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

template <bool F16> __device__ inline f32x4 mfma16(i32x4 a, i32x4 b, f32x4 c) {
  if constexpr (F16) return Mfma<QK_FP16>::mma(a, b, c);
  else return Mfma<QK_BF16>::mma(a, b, c);
}

// Eight e4m3 codes -> eight 16-bit floats.
template <bool F16> __device__ inline i32x4 widen8(int lo, int hi) {
  return i32x4{widen2<F16, false>(lo), widen2<F16, true>(lo), widen2<F16, false>(hi),
               widen2<F16, true>(hi)};
}

template <bool F16> __device__ inline bool not_finite8(i32x4 w) {
  return not_finite2<F16>(w[0]) || not_finite2<F16>(w[1]) || not_finite2<F16>(w[2]) ||
         not_finite2<F16>(w[3]);
}
// The e4m3 codes 0x7F and 0xFF are NaN; there are no infinities.
__device__ inline bool nan_codes(i32x4 w) {
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int b = 0; b < 32; b += 8) r |= ((w[i] >> b) & 0x7F) == 0x7F;
  return r;
}

// The slow product for tiles that hold infinities or NaN among drafted values:
// a weight of zero must add nothing, whatever the value.  The values are
// split into finite ones (others 0) and, one kind after the other, ones where
// a value is +inf, -inf or NaN; a row's weight on such places makes its sum
// that value.
template <bool F16> __device__ inline i32x4 finite_part(i32x4 w) {
  constexpr int E = F16 ? 0x7C00 : 0x7F80;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & E) == E) w[i] &= (int)0xFFFF0000;
    if (((w[i] >> 16) & E) == E) w[i] &= 0xFFFF;
  }
  return w;
}
template <bool F16> __device__ inline i32x4 where_kind(i32x4 w, int kind) {
  constexpr int E = F16 ? 0x7C00 : 0x7F80, ONE = F16 ? 0x3C00 : 0x3F80;
  auto is = [&](int v) {  // 0: +inf, 1: -inf, 2: NaN
    v &= 0xFFFF;
    return kind == 0 ? v == E : kind == 1 ? v == (E | 0x8000) : (v & 0x7FFF) > E;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (is(w[i]) ? ONE : 0) | (is(w[i] >> 16) ? ONE << 16 : 0);
  return w;
}
__device__ inline float kind_value(int kind) {
  return kind == 0 ? -NEG_INF : kind == 1 ? NEG_INF : __builtin_nanf("");
}

// What a workgroup works on: a sequence, a key head and a split.
struct Job {
  int b, hk, split, tile0;
  int t0, n;     // first row of q, drafted nodes
  int ctx, len;  // cached positions before the nodes, positions in all
  float sc;      // scale, key scale and log2 e: positive
  bool flip, none;  // the sign of the scale goes to q; a zero scale: q is 0
};

// What lies beyond the page table (at most 2^30 positions) is cut off.
__device__ inline void set_lengths(const AttnArgs& a, Job& j) {
  const int most = a.max_pages << a.page_log;
  j.ctx = min(max(a.context[j.b], 0), most);
  j.len = min(j.ctx + j.n, most);
}

// Workgroup -> job.  Workgroups go to the eight XCDs in turn; the row tiles
// that share keys follow each other on one XCD and find them in its L2.  A
// malformed plan gives wrong rows, never an access outside the buffers.
__device__ inline bool find_job(const AttnArgs& a, Job& j) {
  const int x = blockIdx.x >> 3;
  int work = (x / a.ntiles) * 8 + (blockIdx.x & 7);
  j.tile0 = x % a.ntiles;
  if (work >= a.nwork) return false;
  j.split = work % a.nsplit;
  work /= a.nsplit;
  j.hk = work % a.Hk;
  j.b = work / a.Hk;
  j.t0 = a.offsets[j.b];
  const int64_t t1 = a.offsets[j.b + 1];
  if (j.t0 < 0 || t1 <= j.t0 || t1 > a.T) return false;
  j.n = (int)(t1 - j.t0);
  set_lengths(a, j);
  const float sc = a.scale_log2e * (a.k_scale ? a.k_scale[j.hk] : 1.f);
  j.flip = sc < 0.f;
  j.none = sc == 0.f;
  j.sc = j.none ? 1.f : fabsf(sc);
  return true;
}

// Positions [lo, hi) of a split for the rows of a tile that ends with node
// `last`, and how many splits those rows have.
__device__ inline int split_range(const AttnArgs& a, const Job& j, int last, int& lo, int& hi) {
  const int all = a.mask ? j.len : min(j.len, j.ctx + last + 1);
  lo = j.split * a.chunk;
  // the last split takes what the bound did not foresee
  hi = j.split == a.nsplit - 1 ? all : min(all, lo + a.chunk);
  return a.nsplit == 1 ? 1 : min(a.nsplit, (all + a.chunk - 1) / a.chunk);
}

// Which of the four positions pos .. pos + 3 the row of `node` (mask words
// `mrow`) sees, as bits 0 .. 3; positions from hi on are not.
__device__ inline uint32_t sees4(const AttnArgs& a, const Job& j, int node, const int64_t* mrow,
                                 int pos, int hi) {
  const int d = pos - j.ctx;  // in nodes; the context lies below 0
  const uint32_t in = (1u << min(max(hi - pos, 0), 4)) - 1;
  if (!a.mask) return in & ((1u << min(max(node + 1 - d, 0), 4)) - 1);
  // the two words that hold the bits: all ones in the context, none past the last
  const int w = d >> 6, sh = d & 63, top = a.mask_words - 1;
  uint64_t w0 = top >= 0 ? (uint64_t)mrow[min(max(w, 0), top)] : 0;
  uint64_t w1 = top >= 0 ? (uint64_t)mrow[min(max(w + 1, 0), top)] : 0;
  w0 = w < 0 ? ~0ull : w > top ? 0 : w0;
  w1 = w + 1 < 0 ? ~0ull : w + 1 > top ? 0 : w1;
  return in & (uint32_t)((w0 >> sh) | (w1 << 1 << (63 - sh)));
}

// The signs of eight 16-bit floats, or all of them zero.
__device__ inline i32x4 scaled_q(i32x4 q, bool flip, bool zero) {
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = zero ? 0 : flip ? q[i] ^ (int)0x80008000 : q[i];
  return q;
}

// The running maximum moves only when it grows by more than 2^SLACK for some
// row of the wave: until then the weights stay below that, and the sums need
// no rescaling.  bf16 weights have binary32's range, so 2^8 costs no precision.
// fp16 ones lose bits below 2^-14 and vanish below 2^-25, which many positions
// beside a heavy one add up to (results made of such weights were off by 900
// times the bound): theirs carry a factor of 2^LIFT, as their sum does, so that
// 2^SLACK is just within the type and bits are lost only below 2^-25.  (A slack
// of 2 and a lift of 13 would move that to 2^-27, but rescales more often: 1500
// nodes over 5001 positions 375 us against 368, dim 256 1126 against 1080.)
template <bool F16> constexpr float SLACK = F16 ? 4.f : 8.f;
template <bool F16> constexpr float LIFT = F16 ? 11.f : 0.f;

// O / l, rounded, and the row's lse from m (base 2) and l.
__device__ inline float inverse_sum(float l, float vscale) {
  return l > 0.f || l != l ? vscale / l : 0.f;
}
template <bool F16> __device__ inline float row_lse(float m, float l) {
  return (m + (__builtin_amdgcn_logf(l) - LIFT<F16>)) * 0.69314718056f;
}

// x, as a value of its own: what is computed from it is not kept in registers
// over a loop that has better use for them.
__device__ inline int again(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// ------------------------------------------------- rows with far scores
// A row's exponents are s sc - M with M = m sc, rounded: all of them are off by
// what M was rounded by, which cancels as long as it is small.  Where M gets to
// 2^22 (scores of heads near their type's limits) it is not, and sums would
// overflow or vanish.  Such a row adds nothing up while its maximum is that far
// (from below zero it may still come back), and if it ends there, far_row
// computes it again: exponents (s - m) sc, all in 32 bits, one wave for one row, a
// position per lane for the scores and D / 64 values per lane for the sums.  That
// takes about 100 times as long.  (Exponents chosen within the kernels' steps
// cost all calls up to 5%, and a variable more that is carried through the
// steps up to 20%: they have no register left for it.)
constexpr float FAR = 4194304.f;
__device__ inline bool is_far(float ms) { return fabsf(ms) >= FAR && fabsf(ms) < -NEG_INF; }

// What is added to a row's scores (base 2) before the exponential.
template <bool F16> __device__ inline float weight_offset(float m, float sc) {
  const float ms = m * sc;
  return fabsf(ms) < FAR ? LIFT<F16> - ms : NEG_INF;  // (-inf also for m = -inf)
}

// What the waves of a workgroup read of the cache.
struct Cache {
  const char *k, *v;               // of the key head
  uint32_t k_ps, k_ts, v_ps, v_ts; // page and in-page strides in bytes
  const int* table;
};

// The positions [lo, hi) of the row of `node` with the query at `q`; buf, in
// LDS: D sums, then m (base 2) and l.
template <int D, bool F16, bool KV8>
__device__ void far_row(const AttnArgs& a, const Job& j, const Cache& c, const uint16_t* q, int node,
                        int lo, int hi, float* buf, int lane) {
  constexpr int VPL = D / 64;
  const int64_t* const mrow = a.mask ? a.mask + (int64_t)(j.t0 + node) * a.mask_words : nullptr;
  float m = NEG_INF, l = 0.f, o[VPL] = {};
#pragma unroll 1
  for (int base = lo; base < hi; base += 64) {
    const int pos = min(base + lane, hi - 1);
    const uint32_t page = min(max(c.table[pos >> a.page_log], 0), a.pages - 1);
    const char* const kp = c.k + (uint64_t)page * c.k_ps + (pos & a.page_mask) * c.k_ts;
    float s = 0.f;
#pragma unroll 1
    for (int d = 0; d < D; d += 8) {
      float x[8], y[8];
      unpack8<F16>(scaled_q(*(const i32x4*)(q + d), j.flip, j.none), x);
      if constexpr (KV8) {
        const i32x2 w = *(const i32x2*)(kp + d);
        unpack8<F16>(widen8<F16>(w[0], w[1]), y);
      } else {
        unpack8<F16>(*(const i32x4*)(kp + d * 2), y);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
    }
    const bool seen = base + lane < hi && (sees4(a, j, node, mrow, pos, hi) & 1);
    if (!seen) s = NEG_INF;
    float mn = s;
#pragma unroll
    for (int i = 32; i > 0; i >>= 1) mn = fmaxf(mn, __shfl_xor(mn, i));
    mn = fmaxf(m, mn);
    const float f = m == NEG_INF ? 0.f : exp2_fast((m - mn) * j.sc);
    m = mn;
    const float e = seen ? exp2_fast(fmaf(s - (m == NEG_INF ? 0.f : m), j.sc, LIFT<F16>)) : 0.f;
    float sum = e;
#pragma unroll
    for (int i = 32; i > 0; i >>= 1) sum += __shfl_xor(sum, i);
    l = l * f + sum;
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] *= f;
    for (uint64_t some = __ballot(e != 0.f); some; some &= some - 1) {
      const int i = __builtin_ctzll(some);
      const float w = __shfl(e, i);
      const char* const vp = c.v + (uint64_t)__shfl(page, i) * c.v_ps + (__shfl(pos, i) & a.page_mask) * c.v_ts;
#pragma unroll
      for (int k = 0; k < VPL; ++k) {
        const int d = lane * VPL + k;
        uint32_t bits;
        if constexpr (KV8) bits = widen2<F16, false>(((const uint8_t*)vp)[d]);
        else bits = ((const uint16_t*)vp)[d];
        o[k] = fmaf(w, h_to_f32<F16>((uint16_t)bits), o[k]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < VPL; ++k) buf[lane * VPL + k] = o[k];
  if (lane == 0) {
    buf[D] = m * j.sc;
    buf[D + 1] = l;
  }
}
// LDS between the lanes of one wave.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ------------------------------------------------------ joining the splits
struct Part {
  f32x4 o;  // four values of a row, not divided by l
  float m, l;
};
__device__ inline void join(Part& x, const Part& y) {
  const float m = fmaxf(x.m, y.m), ms = m == NEG_INF ? 0.f : m;
  const float fx = exp2_fast(x.m - ms), fy = exp2_fast(y.m - ms);
  x.m = m;
  x.l = x.l * fx + y.l * fy;
  x.o = x.o * fx + y.o * fy;
}

// A workgroup joins rows: D / 4 lanes hold one, `per` such groups take its
// splits in turn with AHEAD on their way, and the groups' sums meet in LDS.
// `r` and `nsp` are the row of this thread and its splits (0: no row).  What
// other workgroups of the same launch wrote is read with agent-scope loads.
template <int D, bool F16, bool SAME_LAUNCH, int AHEAD>
__device__ ALWAYS_INLINE void join_rows(const AttnArgs& a, int64_t r, int nsp, int per, float vscale,
                                        Part* parts) {
  constexpr int LPR = D / 4;
  const int c4 = threadIdx.x % LPR * 4, g = threadIdx.x / LPR % per;
  auto pair = [](const float* q) {
    if constexpr (SAME_LAUNCH) return __builtin_bit_cast(float2, ld_agent((const double*)q));
    else return *(const float2*)q;
  };
  auto four = [&](const float* q) {
    if constexpr (!SAME_LAUNCH) return *(const f32x4*)q;
    const float2 u = pair(q), v = pair(q + 2);
    return f32x4{u.x, u.y, v.x, v.y};
  };
  Part x = {{0.f, 0.f, 0.f, 0.f}, NEG_INF, 0.f};
#pragma unroll 1
  for (int i0 = g; i0 < nsp; i0 += AHEAD * per) {
    float2 ml[AHEAD];
    f32x4 u[AHEAD];
    float m = x.m;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      ml[i] = make_float2(NEG_INF, 0.f);
      if (i0 + i * per >= nsp) continue;
      const int64_t pr = (int64_t)(i0 + i * per) * a.rows + r;
      ml[i] = pair(a.part_ml + pr * 2);
      u[i] = four(a.part_o + pr * D + c4);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) m = fmaxf(m, ml[i].x);
    const float ms = m == NEG_INF ? 0.f : m;
    const float f0 = exp2_fast(x.m - ms);
    x.m = m;
    x.l *= f0;
    x.o *= f0;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (i0 + i * per >= nsp) continue;
      const float f = exp2_fast(ml[i].x - ms);
      x.l += f * ml[i].y;
      x.o += f * u[i];
    }
  }
  if (per > 1) {
    parts[threadIdx.x] = x;
    __syncthreads();
    if (g == 0)
      for (int i = 1; i < per; ++i) join(x, parts[threadIdx.x + i * LPR]);
    __syncthreads();
  }
  if (g > 0 || nsp == 0) return;
  const float inv = inverse_sum(x.l, vscale);
  *(i32x2*)(a.out + r * D + c4) =
      i32x2{pack2<F16>(x.o[0] * inv, x.o[1] * inv), pack2<F16>(x.o[2] * inv, x.o[3] * inv)};
  if (a.lse && c4 == 0) a.lse[r] = row_lse<F16>(x.m, x.l);
}

// After a launch whose splits were left apart: blockIdx.y the group of rows.
// With many rows it is bound by issue: 96000 rows of two splits (dim 128) take
// 25 us with two splits ahead and 36 with room for eight.
template <int D, bool F16, int AHEAD>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, int bm, int per) {
  __shared__ Part parts[256];
  const int rows = 256 / (D / 4) / per;  // of a workgroup
  const int hk = blockIdx.x % a.Hk, b = blockIdx.x / a.Hk;
  Job j;
  j.t0 = a.offsets[b];
  const int64_t t1 = a.offsets[b + 1];
  if (j.t0 < 0 || t1 <= j.t0 || t1 > a.T) return;
  j.n = (int)(t1 - j.t0);
  j.b = b;
  set_lengths(a, j);
  j.split = 0;
  const float vscale = a.v_scale ? a.v_scale[hk] : 1.f;
  for (int r0 = blockIdx.y * rows; r0 < j.n * a.G; r0 += gridDim.y * rows) {
    const int row = r0 + threadIdx.x / (D / 4) / per;
    int nsp = 0;
    int64_t r = 0;
    if (row < j.n * a.G) {
      int lo, hi;
      nsp = split_range(a, j, min(row / bm * bm + bm - 1, j.n * a.G - 1) / a.G, lo, hi);
      if (nsp == 1) nsp = 0;  // written by its workgroup
      r = (int64_t)(j.t0 + row / a.G) * (a.Hk * a.G) + hk * a.G + row % a.G;
    }
    join_rows<D, F16, false, AHEAD>(a, r, nsp, per, vscale, parts);
  }
}

// ------------------------------------------------------------ few rows
// One tile of 16 rows.  S^T tiles are 16x16 (MFMA 16x16x32): lane l holds row
// l % 16 and positions 4 (l / 16) + 0..3 of each, so two tiles of a block of
// 32 positions make the eight positions of one lane in the second product;
// the transposing reads of V take the same eight.
//
// Bound by reading the cache: 48 sequences of up to 8191 positions, 8 key
// heads of 128 values, four query heads each, in 8-bit codes take 124 us
// (5.0 TB/s) and in bf16 223 us (5.5 TB/s; a large read reaches 5.4 to 5.9).
// Four waves without a barrier keep loads of 32 KB each on their way; with a
// shared tile of 128 rows, of which 16 are used, the 8-bit call takes 231 us,
// 200 x 1000 positions 297 instead of 85.  Short calls are a chain of
// latencies (page, keys, scores, values, join): 10 us for one token over 1024.
template <int D, bool KV8> constexpr int stream_tile_bytes() { return 32 * D * (KV8 ? 1 : 2); }
template <int D, bool KV8> constexpr int stream_lds_bytes() {
  // the waves' values; at the end two waves' sums, or the parts of the splits;
  // behind them all waves' m and l
  return std::max({4 * stream_tile_bytes<D, KV8>(), 2 * 16 * D * 4, 256 * (int)sizeof(Part)}) +
         4 * 16 * 8;
}

// (Dim 128 over codes just fits three workgroups on a CU: 200 x 1000 positions take
// 86 us, and 96 with two.)
template <int D, bool F16, bool KV8>
__global__ __launch_bounds__(256, D == 256 ? 1 : D == 128 && KV8 ? 3 : 2) void stream_kernel(AttnArgs a) {
  constexpr int ES = KV8 ? 1 : 2;
  constexpr int RB = D * ES;           // bytes of a cache row
  constexpr int KS = D / 32;           // steps of the first product
  constexpr int DT = D / 16;           // tiles of the second
  constexpr int NK = RB / 64;          // 16-byte loads of a key row per lane
  constexpr int RPI = 1024 / RB;       // value rows of one load instruction
  constexpr int NV = 32 / RPI;         // load instructions of a block's values
  constexpr int CPR = RB / 16;         // chunks of a row
  constexpr int VT = stream_tile_bytes<D, KV8>();

  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = lane >> 4, col = lane & 15;
  char* const sv = smem + wave * VT;
  float* const st = (float*)(smem + stream_lds_bytes<D, KV8>() - 4 * 16 * 8);

  Job j;
  if (!find_job(a, j)) return;
  const int* const table = a.table + (int64_t)j.b * a.table_stride;
  const char* const kb = (const char*)a.k + j.hk * a.k_hs * ES;
  const char* const vb = (const char*)a.v + j.hk * a.v_hs * ES;
  // a page's bytes fit 32 bits (checked on the host), a cache's need not
  const uint32_t k_ps = a.k_ps * ES, k_ts = a.k_ts * ES, v_ps = a.v_ps * ES, v_ts = a.v_ts * ES;
  const Cache cache = {kb, vb, k_ps, k_ts, v_ps, v_ts, table};
  const int nrows = j.n * a.G;

  for (int tile = j.tile0; tile * 16 < nrows; tile += a.ntiles) {
    const int row0 = tile * 16;
    const int last = min(row0 + 16 - 1, nrows - 1) / a.G;
    int lo, hi;
    int nsp = split_range(a, j, last, lo, hi);
    if (tile >= a.ntiles && a.counters) {
      // more nodes than the call's bound: there is no arrival counter, and
      // the first split takes the whole row tile
      lo = 0;
      hi = a.mask ? j.len : min(j.len, j.ctx + last + 1);
      nsp = 1;
    }
    if (j.split >= nsp) continue;
    const int nblk = (hi - lo + 31) / 32;

    // this lane's rows, as operands of the first product
    const bool live = row0 + col < nrows;
    const int node = live ? (row0 + col) / a.G : 0;
    const int64_t t = j.t0 + node;
    const int64_t* const mrow = a.mask ? a.mask + t * a.mask_words : nullptr;
    i32x4 qf[KS];
    {
      const int head = j.hk * a.G + (live ? (row0 + col) % a.G : 0);
      const uint16_t* qp = a.q + t * a.q_ts + head * a.q_hs;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        // a lane's 16 bytes of codes are two steps' operands
        const int d = KV8 ? (ks >> 1) * 64 + grp * 16 + (ks & 1) * 8 : ks * 32 + grp * 8;
        qf[ks] = scaled_q(*(const i32x4*)(qp + d), j.flip, j.none || !live);
      }
    }

    float m = NEG_INF, l = 0.f;
    f32x4 o[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[dt] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Pages of a block's 32 positions, one per lane (twice).
    auto load_pages = [&](int blk) {
      const int pos = min(lo + blk * 32 + (lane & 31), hi - 1);
      return table[pos >> a.page_log];  // not looked at before it is used: no wait here
    };
    i32x4 kr[2][NK], vr[NV];
    auto load_block = [&](int blk, int pg) {
      const int base = lo + blk * 32;
      pg = min(max(pg, 0), a.pages - 1);
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const int r = min(base + kt * 16 + col, hi - 1) - base;
        const int p = __shfl(pg, r);
        const char* at = kb + (uint64_t)(uint32_t)p * k_ps +
                         (((base + r) & a.page_mask) * k_ts + grp * 16);
#pragma unroll
        for (int i = 0; i < NK; ++i) kr[kt][i] = *(const i32x4*)(at + i * 64);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = min(base + i * RPI + lane / CPR, hi - 1) - base;
        const int p = __shfl(pg, r);
        vr[i] = *(const i32x4*)(vb + (uint64_t)(uint32_t)p * v_ps +
                                (((base + r) & a.page_mask) * v_ts + (lane % CPR) * 16));
      }
    };
    // Chunks of a value row are XOR-ed with the row, so that the transposing
    // reads of 16 rows spread over the banks.
    auto v_at = [&](int row, int chunk) {
      return sv + row * RB + ((chunk ^ ((KV8 ? row : 2 * row) & (CPR - 1))) << 4);
    };

    int blk = wave;
    int pg = 0;
    if (blk < nblk) {
      load_block(blk, load_pages(blk));
      if (blk + 4 < nblk) pg = load_pages(blk + 4);
    }
    for (; blk < nblk; blk += 4) {
      const int base = lo + blk * 32;
      const bool tail = base + 32 > min(j.ctx, hi);
      bool odd = false;
      // Values past the end read as zero.  Drafted values that some rows do
      // not see must not reach them: an infinity or NaN among those takes
      // the slow product below.
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = i * RPI + lane / CPR;
        if (tail) {
          if (base + r >= hi) vr[i] = i32x4{0, 0, 0, 0};
          else if (base + r >= j.ctx) odd |= KV8 ? nan_codes(vr[i]) : not_finite8<F16>(vr[i]);
        }
        *(i32x4*)v_at(r, lane % CPR) = vr[i];
      }
      odd = __any(odd);
      f32x4 s[2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        s[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          i32x4 kf;
          if constexpr (KV8)
            kf = widen8<F16>(kr[kt][ks >> 1][2 * (ks & 1)], kr[kt][ks >> 1][2 * (ks & 1) + 1]);
          else
            kf = kr[kt][ks];
          s[kt] = mfma16<F16>(kf, qf[ks], s[kt]);
        }
      }
      if (blk + 4 < nblk) {
        load_block(blk + 4, pg);
        if (blk + 8 < nblk) pg = load_pages(blk + 8);
      }
      if (tail) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          const uint32_t vis = sees4(a, j, node, mrow, base + kt * 16 + grp * 4, hi);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[kt][i] = (vis >> i) & 1 ? s[kt][i] : NEG_INF;
        }
      }
      float mx = s[0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i >> 2][i & 3]);
      const float mn = fmaxf(m, quad_max(mx));
      if (__any((mn - m) * j.sc > SLACK<F16>)) {
        const float f = mn == NEG_INF ? 1.f : exp2_fast((m - mn) * j.sc);
        m = mn;
        l *= f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[dt][i] *= f;
      }
      const float at = weight_offset<F16>(m, j.sc);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[i >> 2][i & 3] = exp2_fast(fmaf(s[i >> 2][i & 3], j.sc, at));
        sum += s[i >> 2][i & 3];
      }
      l += sum;
      // rounded to the value type: the products are then exact in the MFMA and
      // summed in 32 bits
      i32x4 pf;
#pragma unroll
      for (int w = 0; w < 4; ++w) pf[w] = pack2<F16>(s[w >> 1][2 * (w & 1)], s[w >> 1][2 * (w & 1) + 1]);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();  // the lanes' values are in LDS
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      auto value = [&](int dt) {
        if constexpr (KV8) {
          const int r8 = col >> 1;
          const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(lds_char*)(
              v_at((r8 & 3) + 4 * grp + (r8 >> 2) * 16, dt) + (col & 1) * 8));
          return widen8<F16>(w[0], w[1]);
        } else {
          const int r = 4 * grp + (col >> 2), c = 2 * dt + ((col & 3) >> 1), b8 = (col & 1) * 8;
          const i32x2 w0 = __builtin_bit_cast(
              i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)(v_at(r, c) + b8)));
          const i32x2 w1 = __builtin_bit_cast(
              i32x2,
              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)(v_at(r + 16, c) + b8)));
          return i32x4{w0[0], w0[1], w1[0], w1[1]};
        }
      };
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        i32x4 vf = value(dt);
        if (odd) {
#pragma unroll 1
          for (int kind = 0; kind < 3; ++kind) {
            const f32x4 x = mfma16<F16>(where_kind<F16>(vf, kind), pf, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int i = 0; i < 4; ++i) o[dt][i] += x[i] > 0.f ? kind_value(kind) : 0.f;
          }
          vf = finite_part<F16>(vf);
        }
        o[dt] = mfma16<F16>(vf, pf, o[dt]);
      }
      __builtin_amdgcn_wave_barrier();  // read before the next block's are written
    }

    // Join the four waves.
    l = quad_sum(l);
    m *= j.sc;
    if (grp == 0) *(float2*)(st + (wave * 16 + col) * 2) = make_float2(m, l);
    __syncthreads();
    {
      float M = NEG_INF, L = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, st[(w * 16 + col) * 2]);
      const float ms = M == NEG_INF ? 0.f : M;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        L += st[(w * 16 + col) * 2 + 1] * exp2_fast(st[(w * 16 + col) * 2] - ms);
      const float f = exp2_fast(m - ms);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[dt][i] *= f;
      m = M;
      l = L;
    }
    f32x4* const sums = (f32x4*)smem;
#pragma unroll
    for (int step = 2; step > 0; step >>= 1) {
      if (wave >= step && wave < 2 * step) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) sums[((wave - step) * DT + dt) * 64 + lane] = o[dt];
      }
      __syncthreads();
      if (wave < step) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] += sums[(wave * DT + dt) * 64 + lane];
      }
      __syncthreads();
    }
    if (wave == 0) {
      uint64_t rows = __ballot(live && is_far(m)) & 0xFFFF;
      while (__builtin_expect(rows != 0, 0)) {
        const int r = __builtin_ctzll(rows), row = row0 + r, ln = again(lane);
        float* const buf = (float*)smem;
        far_row<D, F16, KV8>(a, j, cache, a.q + (int64_t)(j.t0 + row / a.G) * a.q_ts +
                             (int64_t)(j.hk * a.G + row % a.G) * a.q_hs, row / a.G, lo, hi, buf, ln);
        wave_sync();
        if ((ln & 15) == r) {
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) o[dt] = *(const f32x4*)(buf + dt * 16 + (ln >> 4) * 4);
          m = buf[D];
          l = buf[D + 1];
        }
        wave_sync();
        rows &= rows - 1;
      }
    }
    const int heads = a.Hk * a.G;
    auto row_of = [&](int row) {  // of q and out
      return (int64_t)(j.t0 + row / a.G) * heads + j.hk * a.G + row % a.G;
    };
    const float vscale = a.v_scale ? a.v_scale[j.hk] : 1.f;
    if (wave == 0 && live) {
      const int64_t r = row_of(row0 + col);
      const int64_t pr = (int64_t)j.split * a.rows + r;
      if (nsp == 1) {
        const float inv = inverse_sum(l, vscale);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
          *(i32x2*)(a.out + r * D + dt * 16 + grp * 4) =
              i32x2{pack2<F16>(o[dt][0] * inv, o[dt][1] * inv),
                    pack2<F16>(o[dt][2] * inv, o[dt][3] * inv)};
        if (a.lse && grp == 0) a.lse[r] = row_lse<F16>(m, l);
      } else if (!a.counters) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) *(f32x4*)(a.part_o + pr * D + dt * 16 + grp * 4) = o[dt];
        if (grp == 0) *(float2*)(a.part_ml + pr * 2) = make_float2(m, l);
      } else {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int i = 0; i < 4; i += 2)
            st_agent((double*)(a.part_o + pr * D + dt * 16 + grp * 4 + i),
                     __builtin_bit_cast(double, make_float2(o[dt][i], o[dt][i + 1])));
        if (grp == 0) st_agent((double*)(a.part_ml + pr * 2), __builtin_bit_cast(double, make_float2(m, l)));
      }
    }
    // (past the last barrier smem has had no use but far_row's, in wave 0's own part)
    if (nsp == 1 || !a.counters) continue;

    // Arrival: the workgroup that comes last joins the splits.  Partials are
    // written and read with agent-scope atomics, which are coherent across the
    // XCDs' L2s by themselves; the wave waits for its stores to be
    // acknowledged before it counts itself.  (A release / acquire of that
    // scope would write back and invalidate the whole L2 every time.)
    int* const counter = a.counters + ((int64_t)(j.b * a.Hk + j.hk) * a.ntiles + tile) * AT_COUNTER_STEP;
    int* const arrival = (int*)st;
    if (wave == 0) {
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_s_waitcnt(0);
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      if (lane == 0)
        *arrival = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    const bool is_last = *arrival == nsp - 1;
    __syncthreads();  // smem is written again for the next row tile
    if (!is_last) continue;
    const int end = min(row0 + 16, nrows);
    int per = 256 / (D / 4);  // groups of lanes per row
    while (per > 1 && 256 / (D / 4) / per < end - row0) per >>= 1;
    const int g = threadIdx.x / (D / 4);
    for (int r0 = row0; r0 < end; r0 += 256 / (D / 4) / per) {
      const int row = r0 + g / per;
      join_rows<D, F16, true, 8>(a, row < end ? row_of(row) : 0, row < end ? nsp : 0, per, vscale,
                              (Part*)smem);
    }
    if (threadIdx.x == 0) st_agent(counter, 0);  // kept at zero between calls
  }
}

// ------------------------------------------------------------ many rows
// A tile in LDS holds its rows as 16-byte chunks; the chunk index is XOR-ed
// with the row so that 32 lanes that read one chunk of 32 rows (K) or four
// rows of four chunks (V, transposing reads) use all banks, of which a row of
// 64 values covers half.  (No conflicts are counted; with the row shifted by
// one for V at dim 128 and 256 there were two cycles of them per transposing
// read, which cost 4 to 8% at dim 256 and 1% at most at 128.)
template <int D> __device__ inline int k_off(int row, int chunk) {
  return row * (D * 2) + ((chunk ^ (row & (D / 8 - 1))) << 4);
}
template <int D> __device__ inline int v_xor(int row) {
  return (row << (D == 64 ? 1 : 2)) & (D / 8 - 1);
}
template <int D> __device__ inline int v_off(int row, int chunk) {
  return row * (D * 2) + ((chunk ^ v_xor<D>(row)) << 4);
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;

// The value fragment f of a block of 32 positions that starts at row `r0` of
// a tile: sixteen positions (f / DT) by 32 values (f % DT), by two transposing
// reads per lane.
template <int D> __device__ inline i32x4 value_frag(const char* sv, int r0, int f, int lane) {
  constexpr int DT = D / 32;
  const int i16 = lane & 15;
  const int r = r0 + 16 * (f / DT) + 4 * (lane >> 5) + (i16 >> 2);
  const int c = 4 * (f % DT) + 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
  const int b8 = (i16 & 1) * 8;
  const i32x2 w0 = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                 (lds_s16x4*)(lds_char*)(sv + v_off<D>(r, c) + b8)));
  const i32x2 w1 =
      __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                    (lds_s16x4*)(lds_char*)(sv + v_off<D>(r + 8, c) + b8)));
  return i32x4{w0[0], w0[1], w1[0], w1[1]};
}

__device__ inline void clear(f32x16& p) {
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = 0.f;
}

// One wave's 32 rows: what the tile kernels keep of them.
template <int D, bool F16> struct Rows {
  static constexpr int DT = D / 32, KS = D / 16;
  i32x4 q[KS];
  f32x16 o[DT];
  float m, l;

  // Scores of a block of 32 positions.  Key fragments are read a few ahead of
  // the products that use them.
  __device__ inline ALWAYS_INLINE void scores(f32x16& p, const char* sk, int r0, int lane) {
    constexpr int KA = 4;
    if constexpr (D == 256) lane = again(lane);
    const int col = lane & 31, half = lane >> 5;
    i32x4 kf[KS];
    clear(p);
#pragma unroll
    for (int f = 0; f < KA; ++f) kf[f] = *(const i32x4*)(sk + k_off<D>(r0 + col, 2 * f + half));
#pragma unroll
    for (int f = 0; f < KS; ++f) {
      p = mfma32<F16>(kf[f], q[f], p);
      if (f + KA < KS) kf[f + KA] = *(const i32x4*)(sk + k_off<D>(r0 + col, 2 * (f + KA) + half));
    }
  }
  // Masks (for the positions pos + ... of the block), running maximum and sum;
  // p becomes the probabilities, rounded to the value type, in pf.
  template <bool TAIL>
  __device__ inline ALWAYS_INLINE void softmax(f32x16& p, i32x4 (&pf)[2], const AttnArgs& a,
                                               const Job& j, int node, const int64_t* mrow, int pos,
                                               int hi, int lane) {
    if constexpr (TAIL) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t vis = sees4(a, j, node, mrow, pos + 8 * b + 4 * (lane >> 5), hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[b * 4 + i] = (vis >> i) & 1 ? p[b * 4 + i] : NEG_INF;
      }
    }
    float mx = p[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) mx = fmaxf(mx, p[i]);
    const float mn = fmaxf(m, half_max(mx));
    if (__any((mn - m) * j.sc > SLACK<F16>)) {
      const float f = mn == NEG_INF ? 1.f : exp2_fast((m - mn) * j.sc);
      m = mn;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] *= f;
    }
    const float at = weight_offset<F16>(m, j.sc);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      p[i] = exp2_fast(fmaf(p[i], j.sc, at));
      sum += p[i];
    }
    l += sum;
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int w = 0; w < 4; ++w) pf[tt][w] = pack2<F16>(p[8 * tt + 2 * w], p[8 * tt + 2 * w + 1]);
  }
  // O^T += V^T P^T for the block.  TAIL: values that some rows do not see, or
  // that lie past the end, may be infinite or NaN.
  template <bool TAIL>
  __device__ inline ALWAYS_INLINE void values(const i32x4 (&pf)[2], const char* sv, int r0, int lane) {
    constexpr int NF = 2 * DT, VA = 4 < NF ? 4 : NF;
    if constexpr (D == 256) lane = again(lane);
    if constexpr (TAIL) {
      bool odd = false;
#pragma unroll
      for (int f = 0; f < NF; ++f) odd |= not_finite8<F16>(value_frag<D>(sv, r0, f, lane));
      if (__any(odd)) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
#pragma unroll 1
          for (int kind = 0; kind < 3; ++kind) {
            f32x16 t;
            clear(t);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
              t = mfma32<F16>(where_kind<F16>(value_frag<D>(sv, r0, tt * DT + dt, lane), kind),
                              pf[tt], t);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[dt][i] += t[i] > 0.f ? kind_value(kind) : 0.f;
          }
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
            o[dt] = mfma32<F16>(finite_part<F16>(value_frag<D>(sv, r0, tt * DT + dt, lane)), pf[tt],
                                o[dt]);
        }
        return;
      }
    }
    i32x4 vf[NF];
#pragma unroll
    for (int f = 0; f < VA; ++f) vf[f] = value_frag<D>(sv, r0, f, lane);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      o[f % DT] = mfma32<F16>(vf[f], pf[f / DT], o[f % DT]);
      if (f + VA < NF) vf[f + VA] = value_frag<D>(sv, r0, f + VA, lane);
    }
  }
  // Writes a finished row, or its part of a split one.
  __device__ inline void write(const AttnArgs& a, const Job& j, int64_t r, bool whole, int half) {
    if (whole) {
      const float inv = inverse_sum(l, a.v_scale ? a.v_scale[j.hk] : 1.f);
      uint16_t* const op = a.out + r * D + half * 4;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *(i32x2*)(op + dt * 32 + b * 8) =
              i32x2{pack2<F16>(o[dt][b * 4] * inv, o[dt][b * 4 + 1] * inv),
                    pack2<F16>(o[dt][b * 4 + 2] * inv, o[dt][b * 4 + 3] * inv)};
      if (a.lse && half == 0) a.lse[r] = row_lse<F16>(m, l);
    } else {
      const int64_t pr = (int64_t)j.split * a.rows + r;
      float* const op = a.part_o + pr * D + half * 4;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *(f32x4*)(op + dt * 32 + b * 8) =
              f32x4{o[dt][b * 4], o[dt][b * 4 + 1], o[dt][b * 4 + 2], o[dt][b * 4 + 3]};
      if (half == 0) *(float2*)(a.part_ml + pr * 2) = make_float2(m, l);
    }
  }
};

// s_waitcnt immediate for "vmcnt <= n" (other counters not waited for).
constexpr int vmcnt_imm(int n) { return (n & 15) | 0x0F70 | ((n >> 4) << 14); }

// A barrier that waits for the wave's LDS accesses, but for none of its loads.
__device__ inline void tile_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Positions of a tile, and buffers of the tile kernel: 128 KB of LDS.
template <int D> constexpr int tile_positions() { return 8192 / D; }
constexpr int TILE_BUFS = 4;
template <int D> constexpr int tile_waves() { return D == 256 ? 4 : 8; }
template <int D> constexpr int tile_lds_bytes() { return TILE_BUFS * tile_positions<D>() * D * 4; }

// Eight waves of 32 rows.  S^T tiles are 32x32 (MFMA 32x32x16): lane l holds
// row l % 32 and positions 8 b + 4 (l / 32) + 0..3 of each.  CW = 1: 256 rows;
// CW = 2: 128 rows, waves 4..7 take the second half of each tile's positions
// and their sums are joined at the end.
//
// One barrier per tile: past the one that ends step it, every wave has read
// tile it to the end (its buffer may be refilled) and waited for its own
// loads of tile it + 1 (which may be read).  16-bit caches go from memory to
// LDS directly, issued three tiles ahead; 8-bit codes pass through registers
// one tile ahead, where they are widened.  Waves 4..7 have the higher issue
// priority, which keeps the two waves of a SIMD out of step: one's products
// run under the other's exponentials.
//
// What bounds the 16-bit forms: of the three tiles ahead the compiled loop keeps
// none.  The compiler takes the transposing reads of the values for reads of
// what the direct loads still write, and waits for all loads before those of
// each block of 32 positions; and the page numbers, which are loaded after the
// newest tile and used at the next step's start, are waited for there, with
// everything issued before them.  So each tile's way from memory is covered by
// half a softmax only, the counted waits in `finish` never bind, and the matrix
// units are busy 36% of the time.  Open: reads that carry no such dependence, and
// page numbers that are loaded earlier.
//   Four trees of 64 nodes with four heads to a key head over 32000 positions
// (dim 128, bf16): 181 us in this kernel, of which the tiles' way into LDS alone
// takes 103 (5.1 TB/s) and the arithmetic alone 143 (0.94 PFLOP/s); 1500 nodes over
// 5001: 0.84 PFLOP/s.  Over e4m3 codes 171 us and 0.85 PFLOP/s: nothing waits for
// LDS there, but widening costs registers (dim 128 spills 3 to 5 of 256, dim 256
// 8 or 9 of 512).
// Dim 256 has four waves, one per SIMD: O and Q of 32 rows take 200 registers.
// 16 trees of 64 nodes over 2000 positions: 168 us (0.40 PFLOP/s: nothing runs
// beside a wave's exponentials), and 25 more with the LDS offsets of the
// fragments kept over the loop, for which O went to memory.
// Measured and not kept, all with the waits described above, so that other
// results are possible without them: strict alternation of the two waves
// between barriers (215 us), the first product of the next block inside the
// softmax of this one (spills), fragments of the values read before the
// softmax (spills), page numbers by scalar loads (their counter is the LDS
// reads' too: 195 us).
template <int D, int CW, bool F16, bool KV8>
__global__ __launch_bounds__(64 * tile_waves<D>()) void tile_kernel(AttnArgs a) {
  constexpr int THREADS = 64 * tile_waves<D>();
  constexpr int BM = THREADS / 2 / CW, BN = tile_positions<D>();
  constexpr int NB = BN / 32 / CW;
  constexpr int ES = KV8 ? 1 : 2;
  constexpr int CPR = D * ES / 16;       // 16-byte chunks of a cache row
  constexpr int NI = BN * CPR / THREADS; // chunks per thread, tile and operand
  constexpr int TILE = BN * D * 2;       // bytes of one operand's tile
  static_assert(NI * THREADS == BN * CPR, "whole chunks per thread");

  extern __shared__ __align__(16) char smem[];  // [TILE_BUFS][keys, values]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  const int grp = wave >> 2, rw = CW == 1 ? wave : wave & 3, b0 = CW == 1 ? 0 : grp * NB;

  Job j;
  if (!find_job(a, j)) return;
  const int* const table = a.table + (int64_t)j.b * a.table_stride;
  const char* const kb = (const char*)a.k + j.hk * a.k_hs * ES;
  const char* const vb = (const char*)a.v + j.hk * a.v_hs * ES;
  // a page's bytes fit 32 bits (checked on the host), a cache's need not
  const uint32_t k_ps = a.k_ps * ES, k_ts = a.k_ts * ES, v_ps = a.v_ps * ES, v_ts = a.v_ts * ES;
  const Cache cache = {kb, vb, k_ps, k_ts, v_ps, v_ts, table};
  const int nrows = j.n * a.G;
  if (grp) __builtin_amdgcn_s_setprio(1);

  for (int tile = j.tile0; tile * BM < nrows; tile += a.ntiles) {
    const int row0 = tile * BM;
    const int last = min(row0 + BM - 1, nrows - 1) / a.G;
    int lo, hi;
    const int nsp = split_range(a, j, last, lo, hi);
    if (j.split >= nsp) continue;
    const int ntl = (hi - lo + BN - 1) / BN;
    // tiles that every row sees whole
    const int all = min(a.mask ? j.ctx : j.ctx + row0 / a.G + 1, hi);
    const int full = max(0, (all - lo) / BN);

    // this lane's row (rows past the end stand for the first and are not stored)
    struct Row { bool live; int node, head; };
    auto my_row = [&]() ALWAYS_INLINE {
      const int row = row0 + rw * 32 + (again(lane) & 31);
      const bool live = row < nrows;
      const int node = live ? row / a.G : 0;
      return Row{live, node, j.hk * a.G + (live ? row - node * a.G : 0)};
    };
    Rows<D, F16> w;
    {
      const Row r = my_row();
      const uint16_t* qp = a.q + (int64_t)(j.t0 + r.node) * a.q_ts + r.head * a.q_hs + half * 8;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        w.q[ks] = scaled_q(*(const i32x4*)(qp + ks * 16), j.flip, j.none || !r.live);
    }
    w.m = NEG_INF;
    w.l = 0.f;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) clear(w.o[dt]);

    // The cache rows that this thread loads of a tile: chunk idx of the tile
    // in LDS order is row idx / CPR (and, loaded directly, holds the chunk
    // that the XOR puts there).
    auto chunk_row = [&](int i, int ln) ALWAYS_INLINE { return ((wave * NI + i) * 64 + ln) / CPR; };
    struct Pages { int p[NI]; };
    auto load_pages = [&](int it) ALWAYS_INLINE {
      Pages g;
      const int ln = again(lane);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        g.p[i] = table[min(lo + it * BN + chunk_row(i, ln), hi - 1) >> a.page_log];
      return g;  // not looked at before it is used: no wait here
    };
    auto buffer = [&](int it) ALWAYS_INLINE { return smem + (it % TILE_BUFS) * 2 * TILE; };
    i32x4 rk[NI], rv[NI];  // 8-bit caches
    auto issue = [&](int it, const Pages& g) ALWAYS_INLINE {
      char* const sk = buffer(it);
      const int ln = again(lane);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = chunk_row(i, ln), c = ln % CPR;
        const int in = min(lo + it * BN + r, hi - 1) & a.page_mask;
        const uint32_t page = min(max(g.p[i], 0), a.pages - 1);
        const char* ka = kb + (uint64_t)page * k_ps + in * k_ts;
        const char* va = vb + (uint64_t)page * v_ps + in * v_ts;
        if constexpr (KV8) {
          rk[i] = *(const i32x4*)(ka + c * 16);
          rv[i] = *(const i32x4*)(va + c * 16);
        } else {
          char* const at = sk + (wave * NI + i) * 1024;
          __builtin_amdgcn_global_load_lds((global_void*)(ka + ((c ^ (r & (CPR - 1))) << 4)),
                                           (lds_void*)at, 16, 0, 0);
          __builtin_amdgcn_global_load_lds((global_void*)(va + ((c ^ v_xor<D>(r)) << 4)),
                                           (lds_void*)(at + TILE), 16, 0, 0);
        }
      }
    };
    // 8-bit: widen what was loaded into its buffer.
    auto store = [&](int it) ALWAYS_INLINE {
      char* const sk = buffer(it);
      char* const sv = sk + TILE;
      const int ln = again(lane);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = chunk_row(i, ln), c = ln % CPR;
        *(i32x4*)(sk + k_off<D>(r, 2 * c)) = widen8<F16>(rk[i][0], rk[i][1]);
        *(i32x4*)(sk + k_off<D>(r, 2 * c + 1)) = widen8<F16>(rk[i][2], rk[i][3]);
        *(i32x4*)(sv + v_off<D>(r, 2 * c)) = widen8<F16>(rv[i][0], rv[i][1]);
        *(i32x4*)(sv + v_off<D>(r, 2 * c + 1)) = widen8<F16>(rv[i][2], rv[i][3]);
      }
    };
    Pages pg;
    // Tile `it` is in LDS as far as this wave loads it.  `behind`: tiles whose
    // loads were issued after its own (16-bit), if all of them were.
    auto finish = [&](int it, int behind) ALWAYS_INLINE {
      if (it >= ntl) return;
      if constexpr (KV8) {
        store(it);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): written
        if (it + 1 < ntl) {
          issue(it + 1, pg);
          if (it + 2 < ntl) pg = load_pages(it + 2);
        }
      } else if (it + behind >= ntl) {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      } else if (behind == 2) {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(4 * NI));
      } else {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * NI));
      }
    };

    if constexpr (KV8) {
      pg = load_pages(0);
      issue(0, pg);
      if (ntl > 1) pg = load_pages(1);
      finish(0, 0);

    } else {
      const Pages g0 = load_pages(0), g1 = load_pages(1), g2 = load_pages(2);
      pg = load_pages(3);
      issue(0, g0);
      if (ntl > 1) issue(1, g1);
      if (ntl > 2) issue(2, g2);
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    }
    __syncthreads();

    f32x16 p;
    i32x4 pf[2];
    const bool busy = row0 + rw * 32 < nrows;  // any live row in this wave
    w.scores(p, buffer(0), b0 * 32, lane);
    auto step = [&](int it, auto tail_tag) ALWAYS_INLINE {
      constexpr bool TAIL = decltype(tail_tag)::value;
      const char* const sk = buffer(it);
      if (!KV8 && it + 3 < ntl) {
        issue(it + 3, pg);
        pg = load_pages(it + 4);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (busy) {
          int node = 0;
          const int64_t* mrow = nullptr;
          if constexpr (TAIL) {
            node = my_row().node;
            if (a.mask) mrow = a.mask + (int64_t)(j.t0 + node) * a.mask_words;
          }
          w.template softmax<TAIL>(p, pf, a, j, node, mrow, lo + it * BN + (b0 + k) * 32, hi, lane);
          w.template values<TAIL>(pf, sk + TILE, (b0 + k) * 32, lane);
          if (k + 1 < NB) w.scores(p, sk, (b0 + k + 1) * 32, lane);
        }
      }
      finish(it + 1, 2);
      tile_barrier();
      // (past the last block: of whatever the next buffer holds, not used)
      if (busy) w.scores(p, buffer(it + 1), b0 * 32, lane);
    };
    int it = 0;
    for (; it < full; ++it) step(it, std::false_type{});
    for (; it < ntl; ++it) step(it, std::true_type{});
    __syncthreads();

    w.l = half_sum(w.l);
    w.m *= j.sc;
    if constexpr (CW == 2) {
      // the second halves' sums go to the first through LDS
      float* const st = (float*)(smem + 4 * 32 * D * 4);  // [4][32][2]
      f32x4* const sums = (f32x4*)smem + rw * (32 * D / 4);
      if (grp == 1) {
        if (half == 0) *(float2*)(st + (rw * 32 + col) * 2) = make_float2(w.m, w.l);
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            sums[(dt * 4 + b) * 64 + lane] =
                f32x4{w.o[dt][b * 4], w.o[dt][b * 4 + 1], w.o[dt][b * 4 + 2], w.o[dt][b * 4 + 3]};
      }
      __syncthreads();
      if (grp == 0) {
        const float2 ml = *(const float2*)(st + (rw * 32 + col) * 2);
        const float M = fmaxf(w.m, ml.x), ms = M == NEG_INF ? 0.f : M;
        const float f0 = exp2_fast(w.m - ms), f1 = exp2_fast(ml.x - ms);
        w.m = M;
        w.l = w.l * f0 + ml.y * f1;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const f32x4 x = sums[(dt * 4 + b) * 64 + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) w.o[dt][b * 4 + i] = w.o[dt][b * 4 + i] * f0 + x[i] * f1;
          }
      }
    }
    const Row r = my_row();
    if (CW == 1 || grp == 0) {
      uint64_t rows = __ballot(r.live && is_far(w.m)) & 0xFFFFFFFF;
      // (behind the sums of the second halves, which other waves may still read)
      float* const buf = (float*)(smem + TILE_BUFS * 2 * TILE) - (wave + 1) * (D + 4);
      while (__builtin_expect(rows != 0, 0)) {
        const int i = __builtin_ctzll(rows), row = row0 + rw * 32 + i, ln = again(lane);
        far_row<D, F16, KV8>(a, j, cache, a.q + (int64_t)(j.t0 + row / a.G) * a.q_ts +
                             (int64_t)(j.hk * a.G + row % a.G) * a.q_hs, row / a.G, lo, hi, buf, ln);
        wave_sync();
        if ((ln & 31) == i) {
#pragma unroll
          for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const f32x4 x = *(const f32x4*)(buf + dt * 32 + b * 8 + (ln >> 5) * 4);
#pragma unroll
              for (int e = 0; e < 4; ++e) w.o[dt][b * 4 + e] = x[e];
            }
          w.m = buf[D];
          w.l = buf[D + 1];
        }
        wave_sync();
        rows &= rows - 1;
      }
    }
    if (r.live && (CW == 1 || grp == 0))
      w.write(a, j, (int64_t)(j.t0 + r.node) * (a.Hk * a.G) + r.head, nsp == 1, half);
    __syncthreads();  // smem is written again for the next row tile
  }
}

template <int D, int SHAPE, bool F16, bool KV8>
hipError_t launch_one(const AttnArgs& a, hipStream_t s) {
  const int64_t grid = (int64_t)((a.nwork + 7) / 8 * 8) * a.ntiles;
  hipError_t e;
  if constexpr (SHAPE == AT_STREAM16) {
    constexpr size_t lds = stream_lds_bytes<D, KV8>();
    e = opt_in_lds((const void*)stream_kernel<D, F16, KV8>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((stream_kernel<D, F16, KV8>), dim3((unsigned)grid), dim3(256), lds, s, a);
  } else {
    constexpr int CW = SHAPE == AT_TILE128 && D < 256 ? 2 : 1;
    constexpr size_t lds = tile_lds_bytes<D>();
    e = opt_in_lds((const void*)tile_kernel<D, CW, F16, KV8>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((tile_kernel<D, CW, F16, KV8>), dim3((unsigned)grid),
                       dim3(64 * tile_waves<D>()), lds, s, a);
  }
  e = hipGetLastError();
  if (e != hipSuccess || a.nsplit == 1 || a.counters) return e;
  const int bm = attn_rows(SHAPE);
  int per = 1;  // groups of lanes per row: with eight splits each, all loads are on their way at once
  while (per < 256 / (D / 4) && per * 8 < a.nsplit) per *= 2;
  const int rpb = 256 / (D / 4) / per;
  const int64_t groups = std::min<int64_t>(((int64_t)a.ntiles * bm + rpb - 1) / rpb, 65535);
  const dim3 join_grid((unsigned)(a.nwork / a.nsplit), (unsigned)groups);
  if (a.nsplit == 2)
    hipLaunchKernelGGL((join_kernel<D, F16, 2>), join_grid, dim3(256), 0, s, a, bm, per);
  else
    hipLaunchKernelGGL((join_kernel<D, F16, 8>), join_grid, dim3(256), 0, s, a, bm, per);
  return hipGetLastError();
}

template <int D, int SHAPE>
hipError_t launch_types(const AttnArgs& a, bool f16, bool kv8, hipStream_t s) {
  if (f16) return kv8 ? launch_one<D, SHAPE, true, true>(a, s) : launch_one<D, SHAPE, true, false>(a, s);
  return kv8 ? launch_one<D, SHAPE, false, true>(a, s) : launch_one<D, SHAPE, false, false>(a, s);
}

template <int D>
hipError_t launch_dim(const AttnArgs& a, int shape, bool f16, bool kv8, hipStream_t s) {
  switch (shape) {
    case AT_STREAM16: return launch_types<D, AT_STREAM16>(a, f16, kv8, s);
    case AT_TILE128: return launch_types<D, AT_TILE128>(a, f16, kv8, s);
  }
  if constexpr (D < 256) {
    if (shape == AT_TILE256) return launch_types<D, AT_TILE256>(a, f16, kv8, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

AttnPlan attn_plan(int64_t B, int Hk, int G, int D, int64_t max_nodes, int64_t max_len,
                   int64_t all_rows) {
  AttnPlan p;
  const int64_t rows = max_nodes * G;
  // (Measured at dim 128 over 16-bit caches of thousands of positions; the other
  // dims, codes and short contexts follow the same borders unmeasured.)
  // 8 trees over 8000 positions (dim 128, bf16), rows of a key head: 32 rows
  // take 67 us in tiles of 128 and 83 in two tiles of the streaming kernel, 128
  // rows 82 and (tiles of 256) 88, 192 rows 118 and 101.  16 rows stream: 48
  // sequences of 8-bit codes take 127 us, and 231 in tiles of 128.
  if (D == 256) p.shape = rows <= 16 ? AT_STREAM16 : AT_TILE128;  // what fits the registers
  else p.shape = rows <= 16 ? AT_STREAM16 : rows <= 128 ? AT_TILE128 : AT_TILE256;
  const int bm = attn_rows(p.shape);
  p.ntiles = (rows + bm - 1) / bm;
  const int64_t units = B * Hk * p.ntiles;
  const int64_t step = p.shape == AT_STREAM16 ? 128 : 64;  // positions of one round of the waves
  const int64_t steps = (max_len + step - 1) / step;
  // Parts of splits take 128 MB at most, so that a call's workspace is bounded.
  // (With 32 heads of 128: 2100 nodes over 5000 positions take 390 us in nine
  // splits of 35 MB and 322 in three; 3 x 1400 over 2000 432 and 289; 4200 over
  // 12000 1254 in four of 70 MB, and 1353 whole.)
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 27) / (all_rows * (D + 2) * (int64_t)sizeof(float)));
  int64_t ns;
  if (p.shape == AT_STREAM16) {
    // A workgroup for each CU; more make more parts to join (one sequence of
    // 8000 positions: 14.8 us with 256, 17.9 with 512).  Lengths may differ,
    // though: up to 1536 where a split is longer than 2048 positions (48
    // sequences of up to 8191, 8-bit: 143 us with 768, 127 with 1536).
    ns = (256 + units - 1) / units;
    if (units * ns < 1536) ns = std::max(ns, std::min((1536 + units - 1) / units, (max_len + 2047) / 2048));
    ns = std::min({ns, steps, most});
  } else {
    // as many as fill whole rounds best; splits of four tiles at least
    const int64_t slots = 256;
    double best = 0;
    ns = 1;
    for (int64_t n = 1; n <= std::min({(int64_t)16, (steps + 3) / 4, most}); ++n) {
      const int64_t rounds = (units * n + slots - 1) / slots;
      const double use = (double)(units * n) / (double)(rounds * slots) - 0.01 * (double)n;
      if (use > best + 1e-9) { best = use; ns = n; }
    }
  }
  ns = std::max<int64_t>(1, ns);
  p.chunk = (steps + ns - 1) / ns * step;
  p.nsplit = std::max<int64_t>(1, (max_len + p.chunk - 1) / p.chunk);
  // Joined by the last workgroup, a call of one token over 1024 positions
  // takes 10.3 instead of 12 us; of 1536 workgroups (48 sequences of up to 8191)
  // the arrivals and the narrower stores cost 5 us more than a second launch.
  p.arrival = p.shape == AT_STREAM16 && units * p.nsplit <= 512;
  return p;
}

hipError_t launch_attention(const AttnArgs& a, int D, int shape, bool f16, bool kv8, hipStream_t s) {
  if (D == 64) return launch_dim<64>(a, shape, f16, kv8, s);
  if (D == 128) return launch_dim<128>(a, shape, f16, kv8, s);
  return launch_dim<256>(a, shape, f16, kv8, s);
}

}  // namespace lg
