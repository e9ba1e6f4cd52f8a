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
// Layout.  The rows of one key head (its nodes times the query heads that
// share it) are packed into tiles of 32 per wave, so a key is read once for
// all heads of a group.  Scores are formed transposed, S^T = K Q^T, with
// the 32x32x16 MFMA: a lane then holds 16 scores of ONE row, so the row
// statistics are register reductions and one half-wave swap, and the
// rounded probabilities are already the B operand of O^T = V^T P^T -- the
// contraction order over positions is permuted the same way on the V side,
// whose fragments come from LDS by transposing reads.
//
// Four waves of a workgroup share each tile of keys and values in LDS.  They
// are arranged as RW row tiles x CW shares of the positions: few rows split
// the positions (1 x 4), many rows split the rows (4 x 1).  Long contexts
// are split over workgroups too; those write (m, l, O) in 32 bits and a
// second kernel joins them.
#include "launch.hpp"

namespace lg {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) char lds_char;

constexpr int AT_THREADS = 256;
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

// Two fp32 -> packed 16-bit floats.
template <bool F16> __device__ inline int pack2(float a, float b) {
  return (int)((uint32_t)f32_to_h<F16>(a) | ((uint32_t)f32_to_h<F16>(b) << 16));
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

// ------------------------------------------------------------ LDS tiles
// A tile holds its rows as 16-byte chunks (8 values); the chunk index is
// XOR-ed with the row so that 32 lanes that read one chunk of 32 rows (K) or
// four rows of two chunks (V, transposing reads) use all banks.
template <int D> __device__ inline int k_off(int row, int chunk) {
  return row * (D * 2) + ((chunk ^ (row & (D / 8 - 1))) << 4);
}
template <int D> __device__ inline int v_off(int row, int chunk) {
  return row * (D * 2) + ((chunk ^ ((row << 1) & (D / 8 - 1))) << 4);
}

struct Seq {
  int t0, n;     // first row of q, drafted nodes
  int ctx, len;  // cached positions before the nodes, positions in all
};

template <int D, int RW, bool F16, bool KV8>
__global__ __launch_bounds__(AT_THREADS) void attn_kernel(AttnArgs a) {
  constexpr int CW = 4 / RW;
  constexpr int BM = 32 * RW;             // rows per workgroup
  constexpr int BN = CW == 4 ? 128 : 64;  // positions per tile
  constexpr int NS = BN / (32 * CW);      // 32-position blocks per wave and tile
  constexpr int DT = D / 32, KS = D / 16;
  constexpr int CPR = KV8 ? D / 16 : D / 8;  // 16-byte chunks of a cache row
  constexpr int NI = BN * CPR / AT_THREADS;  // chunks per thread, tile and operand
  constexpr int TILE = BN * D * 2;           // bytes of one operand's tile

  extern __shared__ __align__(16) char smem[];
  char* const sk = smem;
  char* const sv = smem + TILE;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int half = lane >> 5, col = lane & 31;
  const int rw = wave / CW, cw = wave % CW;

  // Workgroup -> (sequence, key head, split, row tile).  Workgroups go to
  // the eight XCDs in turn; the row tiles that share keys follow each other
  // on one XCD and find them in its L2.
  const int id = blockIdx.x;
  const int x = id >> 3;
  int work = (x / a.ntiles) * 8 + (id & 7);
  const int tile0 = x % a.ntiles;
  if (work >= a.nwork) return;
  const int split = work % a.nsplit;
  work /= a.nsplit;
  const int hk = work % a.Hk, b = work / a.Hk;

  Seq s;
  s.t0 = a.offsets[b];
  s.n = a.offsets[b + 1] - s.t0;
  s.ctx = a.context[b];
  // A malformed plan gives wrong rows, never an access outside the buffers.
  if (s.t0 < 0 || s.n <= 0 || (int64_t)s.t0 + s.n > a.T) return;
  s.ctx = max(s.ctx, 0);
  const int64_t room = (int64_t)a.max_pages << a.page_log;
  s.len = (int)min((int64_t)s.ctx + s.n, room);
  if (s.len <= 0) return;
  const int G = a.G;
  const int* const table = a.table + (int64_t)b * a.table_stride;
  const float kscale = a.k_scale ? a.k_scale[hk] : 1.f;
  const float vscale = a.v_scale ? a.v_scale[hk] : 1.f;
  const float sc = a.scale_log2e * kscale;

  const int nrows = s.n * G;
  for (int tile = tile0; tile * BM < nrows; tile += a.ntiles) {
    const int row0 = tile * BM;
    const int last_node = min(row0 + BM - 1, nrows - 1) / G;
    const int kv_all = a.mask ? s.len : min(s.len, s.ctx + last_node + 1);
    const int nsp = a.nsplit == 1 ? 1 : min(a.nsplit, (kv_all + a.chunk - 1) / a.chunk);
    if (split >= nsp) continue;
    const int kv_lo = split * a.chunk;
    // the last split takes what the bound did not foresee
    const int kv_hi = split == a.nsplit - 1 ? kv_all : min(kv_all, kv_lo + a.chunk);
    const int ntl = (kv_hi - kv_lo + BN - 1) / BN;

    // this lane's row
    const int row = row0 + rw * 32 + col;
    const bool live = row < nrows;
    const int node = live ? row / G : 0;
    const int64_t t = s.t0 + node;
    const int head = hk * G + (live ? row % G : 0);
    i32x4 qf[KS];
    {
      const uint16_t* qp = a.q + t * a.q_ts + head * a.q_hs + half * 8;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[ks] = *(const i32x4*)(qp + ks * 16);
        if (!live) qf[ks] = i32x4{0, 0, 0, 0};
      }
    }
    const int64_t* const mrow = a.mask ? a.mask + t * a.mask_words : nullptr;

    float m = NEG_INF, l = 0.f;
    f32x16 o[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;

    int pg[NI];         // pages of the rows this thread loads next
    i32x4 rk[NI], rv[NI];
    auto load_pages = [&](int it) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int pos = min(kv_lo + it * BN + (tid + i * AT_THREADS) / CPR, kv_hi - 1);
        pg[i] = min(max(table[pos >> a.page_log], 0), a.pages - 1);
      }
    };
    auto load_tile = [&](int it) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int idx = tid + i * AT_THREADS;
        const int r = idx / CPR, c = idx % CPR;
        const int pos = min(kv_lo + it * BN + r, kv_hi - 1);
        const int in = pos & a.page_mask;
        const int64_t ko = pg[i] * a.k_ps + hk * a.k_hs + in * a.k_ts;
        const int64_t vo = pg[i] * a.v_ps + hk * a.v_hs + in * a.v_ts;
        rk[i] = *(const i32x4*)((const char*)a.k + (KV8 ? ko : ko * 2) + c * 16);
        rv[i] = *(const i32x4*)((const char*)a.v + (KV8 ? vo : vo * 2) + c * 16);
      }
    };
    load_pages(0);
    load_tile(0);
    if (ntl > 1) load_pages(1);

    for (int it = 0; it < ntl; ++it) {
      const int base = kv_lo + it * BN;
      // Positions past the end read as zero; drafted values that some rows
      // do not see must not reach them, so an infinity or NaN among those
      // takes the slow product below.
      const bool tail = base + BN > min(s.ctx, kv_hi);
      bool odd = false;
      __syncthreads();  // the previous tile is read
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int idx = tid + i * AT_THREADS;
        const int r = idx / CPR, c = idx % CPR;
        if (tail && base + r >= kv_hi) {
          rk[i] = i32x4{0, 0, 0, 0};
          rv[i] = i32x4{0, 0, 0, 0};
        }
        if constexpr (KV8) {
          i32x4 lo, hi;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            lo[2 * w] = widen2<F16, false>(rk[i][w]);
            lo[2 * w + 1] = widen2<F16, true>(rk[i][w]);
            hi[2 * w] = widen2<F16, false>(rk[i][w + 2]);
            hi[2 * w + 1] = widen2<F16, true>(rk[i][w + 2]);
          }
          *(i32x4*)(sk + k_off<D>(r, 2 * c)) = lo;
          *(i32x4*)(sk + k_off<D>(r, 2 * c + 1)) = hi;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            lo[2 * w] = widen2<F16, false>(rv[i][w]);
            lo[2 * w + 1] = widen2<F16, true>(rv[i][w]);
            hi[2 * w] = widen2<F16, false>(rv[i][w + 2]);
            hi[2 * w + 1] = widen2<F16, true>(rv[i][w + 2]);
          }
          *(i32x4*)(sv + v_off<D>(r, 2 * c)) = lo;
          *(i32x4*)(sv + v_off<D>(r, 2 * c + 1)) = hi;
          if (tail && base + r >= s.ctx)
#pragma unroll
            for (int w = 0; w < 4; ++w) odd |= not_finite2<F16>(lo[w]) || not_finite2<F16>(hi[w]);
        } else {
          *(i32x4*)(sk + k_off<D>(r, c)) = rk[i];
          *(i32x4*)(sv + v_off<D>(r, c)) = rv[i];
          if (tail && base + r >= s.ctx)
#pragma unroll
            for (int w = 0; w < 4; ++w) odd |= not_finite2<F16>(rv[i][w]);
        }
      }
      if (tail) odd = __syncthreads_or(odd);
      else __syncthreads();
      if (it + 1 < ntl) {
        load_tile(it + 1);
        if (it + 2 < ntl) load_pages(it + 2);
      }

#pragma unroll
      for (int ns = 0; ns < NS; ++ns) {
        const int sub = (cw * NS + ns) * 32;  // first row of this block in the tile
        f32x16 p;
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const i32x4 kf = *(const i32x4*)(sk + k_off<D>(sub + col, 2 * ks + half));
          p = mfma32<F16>(kf, qf[ks], p);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] *= sc;
        if (tail) {
#pragma unroll
          for (int bb = 0; bb < 4; ++bb) {
            const int pos0 = base + sub + 8 * bb + 4 * half;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int pos = pos0 + i, j = pos - s.ctx;
              bool sees = pos < kv_hi;
              if (sees && j >= 0) {
                if (mrow)
                  sees = (j >> 6) < a.mask_words && ((mrow[j >> 6] >> (j & 63)) & 1);
                else
                  sees = j <= node;
              }
              if (!sees) p[bb * 4 + i] = NEG_INF;
            }
          }
        }
        float mx = p[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, p[i]);
        const float mn = fmaxf(m, half_max(mx));
        const float ms = mn == NEG_INF ? 0.f : mn;  // nothing seen yet: all weights are 0
        const float f = exp2_fast(m - ms);
        m = mn;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[i] = exp2_fast(p[i] - ms);
          sum += p[i];
        }
        l = l * f + sum;
        if (__any(f != 1.f)) {
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[dt][i] *= f;
        }
        if (odd) {
          // One position at a time: a weight of zero adds nothing, whatever
          // the value there is.
          for (int j = 0; j < 32; ++j) {
            float pj = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if ((j >> 3) * 4 + (j & 3) == i) pj = p[i];
            pj = __shfl(pj, col + ((j >> 2) & 1) * 32);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int d = dt * 32 + (i >> 2) * 8 + half * 4 + (i & 3);
                const float v = h_to_f32<F16>(
                    *(const uint16_t*)(sv + v_off<D>(sub + j, d >> 3) + (d & 7) * 2));
                if (pj != 0.f) o[dt][i] += pj * v;
              }
          }
        } else {
          // The probabilities of 16 positions, rounded to the value type: the
          // products are exact in the MFMA and summed in 32 bits.
          i32x4 pf[2];
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int w = 0; w < 4; ++w)
              pf[tt][w] = pack2<F16>(p[8 * tt + 2 * w], p[8 * tt + 2 * w + 1]);
          const int i16 = lane & 15;
          const int vr = sub + 4 * half + (i16 >> 2);
          const int vc = 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
              s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (lds_s16x4*)(lds_char*)(sv + v_off<D>(vr + 16 * tt, vc + 4 * dt) + (i16 & 1) * 8));
              s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (lds_s16x4*)(lds_char*)(sv + v_off<D>(vr + 16 * tt + 8, vc + 4 * dt) + (i16 & 1) * 8));
              const i32x2 w0 = __builtin_bit_cast(i32x2, v0), w1 = __builtin_bit_cast(i32x2, v1);
              o[dt] = mfma32<F16>(i32x4{w0[0], w0[1], w1[0], w1[1]}, pf[tt], o[dt]);
            }
        }
      }
    }

    // Join the waves that share rows.
    l = half_sum(l);
    if constexpr (CW > 1) {
      __syncthreads();  // the tiles are read
      float* const st = (float*)smem;  // [4][32][2]
      if (half == 0) {
        st[(wave * 32 + col) * 2] = m;
        st[(wave * 32 + col) * 2 + 1] = l;
      }
      __syncthreads();
      float M = NEG_INF, L = 0.f;
#pragma unroll
      for (int c = 0; c < CW; ++c) M = fmaxf(M, st[((rw * CW + c) * 32 + col) * 2]);
      const float ms = M == NEG_INF ? 0.f : M;
#pragma unroll
      for (int c = 0; c < CW; ++c)
        L += st[((rw * CW + c) * 32 + col) * 2 + 1] *
             exp2_fast(st[((rw * CW + c) * 32 + col) * 2] - ms);
      const float f = exp2_fast(m - ms);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] *= f;
      m = M;
      l = L;
      // pairwise: the upper half of the waves hands its sums to the lower
#pragma unroll
      for (int step = CW / 2; step > 0; step >>= 1) {
        __syncthreads();
        if (cw >= step && cw < 2 * step) {
          float* const dst = (float*)smem + (rw * step + (cw - step)) * (DT * 16 * 64) + lane;
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[(dt * 16 + i) * 64] = o[dt][i];
        }
        __syncthreads();
        if (cw < step) {
          const float* const src = (const float*)smem + (rw * step + cw) * (DT * 16 * 64) + lane;
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[dt][i] += src[(dt * 16 + i) * 64];
        }
      }
    }
    if (cw == 0 && live) {
      const int64_t r = t * ((int64_t)a.Hk * G) + head;
      if (a.nsplit > 1 && half == 0 && split == 0) a.nsp[r] = nsp;
      if (nsp == 1) {
        const float inv = l > 0.f || l != l ? vscale / l : 0.f;
        uint16_t* const op = a.out + r * D;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int bb = 0; bb < 4; ++bb) {
            i32x2 w;
            w[0] = pack2<F16>(o[dt][bb * 4] * inv, o[dt][bb * 4 + 1] * inv);
            w[1] = pack2<F16>(o[dt][bb * 4 + 2] * inv, o[dt][bb * 4 + 3] * inv);
            *(i32x2*)(op + dt * 32 + bb * 8 + half * 4) = w;
          }
        if (a.lse && half == 0) a.lse[r] = (m + __log2f(l)) * 0.69314718056f;
      } else {
        const int64_t pr = (int64_t)split * a.rows + r;
        float* const op = a.part_o + pr * D;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int bb = 0; bb < 4; ++bb)
            *(f32x4*)(op + dt * 32 + bb * 8 + half * 4) =
                f32x4{o[dt][bb * 4], o[dt][bb * 4 + 1], o[dt][bb * 4 + 2], o[dt][bb * 4 + 3]};
        if (half == 0) {
          a.part_ml[pr * 2] = m;
          a.part_ml[pr * 2 + 1] = l;
        }
      }
    }
    __syncthreads();  // smem is written again for the next row tile
  }
}

// Joins the splits of each row: one wave per row, D / 64 values per lane.
template <int D, bool F16>
__global__ __launch_bounds__(AT_THREADS) void attn_join_kernel(AttnArgs a) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= a.rows) return;
  const int lane = threadIdx.x & 63;
  // Rows that no sequence owns, and rows that one workgroup finished, are
  // not touched: nsp was cleared before and set by the row's first split.
  const int nsp = a.nsp[r];
  if (nsp <= 1 || nsp > a.nsplit) return;
  float M = NEG_INF;
  for (int i = 0; i < nsp; ++i) M = fmaxf(M, a.part_ml[(i * a.rows + r) * 2]);
  const float ms = M == NEG_INF ? 0.f : M;
  float L = 0.f, o[D / 64];
#pragma unroll
  for (int c = 0; c < D / 64; ++c) o[c] = 0.f;
  for (int i = 0; i < nsp; ++i) {
    const int64_t pr = i * a.rows + r;
    const float f = exp2_fast(a.part_ml[pr * 2] - ms);
    L += f * a.part_ml[pr * 2 + 1];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) o[c] += f * a.part_o[pr * D + c * 64 + lane];
  }
  const int hk = (int)(r % (a.Hk * a.G)) / a.G;
  const float vscale = a.v_scale ? a.v_scale[hk] : 1.f;
  const float inv = L > 0.f || L != L ? vscale / L : 0.f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) a.out[r * D + c * 64 + lane] = f32_to_h<F16>(o[c] * inv);
  if (a.lse && lane == 0) a.lse[r] = (M + __log2f(L)) * 0.69314718056f;
}

template <int D, int RW, bool F16, bool KV8>
hipError_t launch_one(const AttnArgs& a, hipStream_t s) {
  constexpr int BN = RW == 1 ? 128 : 64;
  constexpr size_t lds = (size_t)BN * D * 4;
  const void* fn = (const void*)attn_kernel<D, RW, F16, KV8>;
  hipError_t e = opt_in_lds(fn, lds);
  if (e != hipSuccess) return e;
  const int64_t grid = (int64_t)((a.nwork + 7) / 8 * 8) * a.ntiles;
  hipLaunchKernelGGL((attn_kernel<D, RW, F16, KV8>), dim3((unsigned)grid), dim3(AT_THREADS), lds,
                     s, a);
  e = hipGetLastError();
  if (e != hipSuccess || a.nsplit == 1) return e;
  hipLaunchKernelGGL((attn_join_kernel<D, F16>), dim3((unsigned)((a.rows + 3) / 4)),
                     dim3(AT_THREADS), 0, s, a);
  return hipGetLastError();
}

template <int D, int RW>
hipError_t launch_types(const AttnArgs& a, bool f16, bool kv8, hipStream_t s) {
  if (f16) return kv8 ? launch_one<D, RW, true, true>(a, s) : launch_one<D, RW, true, false>(a, s);
  return kv8 ? launch_one<D, RW, false, true>(a, s) : launch_one<D, RW, false, false>(a, s);
}

template <int D>
hipError_t launch_dim(const AttnArgs& a, int rw, bool f16, bool kv8, hipStream_t s) {
  if (rw == 1) return launch_types<D, 1>(a, f16, kv8, s);
  if (rw == 2) return launch_types<D, 2>(a, f16, kv8, s);
  return launch_types<D, 4>(a, f16, kv8, s);
}

}  // namespace

AttnPlan attn_plan(int64_t B, int Hk, int G, int D, int64_t max_nodes, int64_t max_len) {
  AttnPlan p;
  const int64_t rows = max_nodes * G;
  p.rw = rows <= 32 ? 1 : rows <= 64 ? 2 : 4;
  const int bm = 32 * p.rw, bn = p.rw == 1 ? 128 : 64;
  p.ntiles = (rows + bm - 1) / bm;
  // Enough workgroups for two on each of the 256 CUs; a split takes at
  // least two tiles.
  const int64_t units = B * Hk * p.ntiles;
  int64_t ns = (512 + units - 1) / units;
  ns = std::max<int64_t>(1, std::min(ns, (max_len + 2 * bn - 1) / (2 * bn)));
  p.chunk = ((max_len + ns - 1) / ns + bn - 1) / bn * bn;
  p.nsplit = std::max<int64_t>(1, (max_len + p.chunk - 1) / p.chunk);
  return p;
}

hipError_t launch_attention(const AttnArgs& a, int D, int rw, bool f16, bool kv8, hipStream_t s) {
  if (a.nsplit > 1) {
    hipError_t e = launch_fill_zero(a.nsp, (size_t)a.rows * sizeof(int), s);
    if (e != hipSuccess) return e;
  }
  if (D == 64) return launch_dim<64>(a, rw, f16, kv8, s);
  if (D == 128) return launch_dim<128>(a, rw, f16, kv8, s);
  return launch_dim<256>(a, rw, f16, kv8, s);
}

}  // namespace lg
