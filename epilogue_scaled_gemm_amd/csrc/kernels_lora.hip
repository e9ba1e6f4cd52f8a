// kernels_lora.hip -- low-rank adapters of many requests beside a shared
// projection:
//
//   out[t, n] = base[t, n] + f[id] sum_r h[t, r] B[id, n, r],
//   h[t, r] = sum_k x[t, k] A[id, r, k],        id = ids[t]
//
// (a QKV product's slices have their own rows of A: h then is [slices][rank]).
// Two launches: shrink_kernel forms h in 32 bits, expand_kernel adds its
// product with B to the base and rounds once.
//
// Rows name their adapters in any order.  A window of 64 rows is one id per lane,
// so that the rows of one adapter are a ballot: a workgroup takes adapters whose
// first row of the window lies in its slot, gathers their rows as MFMA columns
// and so reads an adapter's weights once for all its rows of the window.  Rows
// and weights go from memory straight into MFMA operands (16x16x32: weights are
// the rows, tokens the columns); every wave has loads of several steps on their
// way.
//
// Bound by bytes: of the adapters in use for a decode step, of x, base and out
// for prompts.
#include "launch.hpp"

namespace lg {
namespace {

constexpr int LR_THREADS = 256, LR_WAVES = 4, LR_WINDOW = 64;

template <bool F16> __device__ inline f32x4 mma(i32x4 w, i32x4 x, f32x4 c) {
  if constexpr (F16) return Mfma<QK_FP16>::mma(w, x, c);
  else return Mfma<QK_BF16>::mma(w, x, c);
}

__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Calls f(id, mask of its rows, first row) for every adapter, -1 among them,
// whose first row of the window lies in the slot; id and mask are scalar.
template <typename F> __device__ inline void each_adapter(const LoraArgs& a, int64_t row0, int slot, F f) {
  const int lane = threadIdx.x & 63;
  const bool live = row0 + lane < a.T;
  int id = live ? a.ids[row0 + lane] : -1;
  if (id < 0 || id >= a.n) id = -1;
  const uint64_t all = __ballot(live);
  const int span = LR_WINDOW / a.slots;
  uint64_t todo = all & (span == 64 ? ~0ull : ((1ull << span) - 1) << (slot * span));
  while (todo) {
    const int r = __builtin_ctzll(todo);
    const int mine = __builtin_amdgcn_readlane(id, r);
    const uint64_t rows = __ballot(id == mine) & all;
    todo &= ~rows;
    if (__builtin_ctzll(rows) == r) f(mine, rows);
  }
}

// The rows of a mask in order, in LDS.
__device__ inline void list_rows(uint64_t rows, uint8_t* list) {
  const int lane = threadIdx.x & 63;
  wave_sync();  // (the last one's readers are done)
  if ((rows >> lane) & 1) list[__popcll(rows & ((1ull << lane) - 1))] = lane;
  wave_sync();
}

// ------------------------------------------------------------------ shrink
// A workgroup: JT tiles of 16 rows of A and a part of k, which its waves share
// out 64 at a time.
template <bool F16, int JT, int GR>
__device__ void shrink_rows(const LoraArgs& a, const uint16_t* A, int j0, int64_t row0, const uint8_t* list,
                            int count, int g0, float* out, f32x4* sums) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const uint16_t* xp[GR];
#pragma unroll
  for (int g = 0; g < GR; ++g)
    xp[g] = a.x + (row0 + list[min((g0 + g) * 16 + col, count - 1)]) * a.x_s + q * 16;
  const uint16_t* ap[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j)
    ap[j] = A + (int64_t)min(j0 + j * 16 + col, a.SR - 1) * a.K + q * 16;

  f32x4 acc[JT][GR];
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int g = 0; g < GR; ++g) acc[j][g] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Steps of 64 values of k: a lane's 32 bytes are two products' operands.
  const int steps = (a.K + 63) >> 6, whole = a.K >> 6;
  const int lo = (int)((int64_t)steps * blockIdx.z / a.ksplit), hi = (int)((int64_t)steps * (blockIdx.z + 1) / a.ksplit);
  auto products = [&](const i32x4 (&xa)[GR][2], const i32x4 (&aa)[JT][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int g = 0; g < GR; ++g) acc[j][g] = mma<F16>(aa[j][h], xa[g][h], acc[j][g]);
  };
  constexpr int AHEAD = JT + GR <= 5 ? 4 : 2;
#pragma unroll AHEAD
  for (int st = lo + wave; st < min(hi, whole); st += LR_WAVES) {
    i32x4 xa[GR][2], aa[JT][2];
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) aa[j][h] = *(const i32x4*)(ap[j] + st * 64 + h * 8);
#pragma unroll
    for (int g = 0; g < GR; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) xa[g][h] = *(const i32x4*)(xp[g] + st * 64 + h * 8);
    products(xa, aa);
  }
  // the last, partial step: its wave is the one whose turn it is
  if (hi > whole && (whole - lo) % LR_WAVES == wave) {
    i32x4 xa[GR][2], aa[JT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = whole * 64 + q * 16 + h * 8 < a.K;
      const int at = in ? whole * 64 + h * 8 : -q * 16;  // (the row's first values stand in)
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        aa[j][h] = *(const i32x4*)(ap[j] + at);
        if (!in) aa[j][h] = i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int g = 0; g < GR; ++g) {
        xa[g][h] = *(const i32x4*)(xp[g] + at);
        if (!in) xa[g][h] = i32x4{0, 0, 0, 0};
      }
    }
    products(xa, aa);
  }

  // The waves' sums meet in LDS, 16 token rows at a time, in the order of the waves.
#pragma unroll
  for (int g = 0; g < GR; ++g) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < JT; ++j) sums[(wave * JT + j) * 64 + lane] = acc[j][g];
    __syncthreads();
    const int p = (g0 + g) * 16 + col;
    for (int j = wave; j < JT; j += LR_WAVES) {
      f32x4 v = sums[j * 64 + lane];
#pragma unroll
      for (int w = 1; w < LR_WAVES; ++w) v += sums[(w * JT + j) * 64 + lane];
      const int r = j0 + j * 16 + q * 4;
      if (p < count && r < a.SR) *(f32x4*)(out + (row0 + list[p]) * a.SR + r) = v;
    }
  }
}

template <bool F16, int JT>
__global__ __launch_bounds__(LR_THREADS, 2) void shrink_kernel(LoraArgs a) {
  __shared__ f32x4 sums[LR_WAVES * JT * 64];
  __shared__ uint8_t lists[LR_WAVES][LR_WINDOW];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const list = lists[wave];
  const int64_t row0 = (int64_t)(blockIdx.x / a.slots) * LR_WINDOW;
  const int j0 = blockIdx.y * JT * 16;
  float* const out = a.h + (int64_t)blockIdx.z * a.T * a.SR;
  each_adapter(a, row0, blockIdx.x % a.slots, [&](int id, uint64_t rows) {
    if (id < 0) return;
    list_rows(rows, list);
    const int count = __popcll(rows);
    const uint16_t* const A = a.a + (int64_t)id * a.SR * a.K;
    if (count <= 16) shrink_rows<F16, JT, 1>(a, A, j0, row0, list, count, 0, out, sums);
    else if (count <= 32) shrink_rows<F16, JT, 2>(a, A, j0, row0, list, count, 0, out, sums);
    else shrink_rows<F16, JT, 4>(a, A, j0, row0, list, count, 0, out, sums);
  });
}

// ------------------------------------------------------------------ expand
// h of a row is rounded to 16 bits twice, as a leading and a remaining part (16 and
// more bits of it in bf16, 22 in fp16): of one part alone the sum would be off by
// its rounding, which is of the size of the output's own.  fp16 has no range
// for it, so a row's h is brought to below 2^14 by a power of two first.
//
// KS: steps of 32 ranks; 0: ranks up to 16, both parts in one step.
template <bool F16, int KS, int GR>
__device__ void expand_rows(const LoraArgs& a, int id, int64_t row0, const uint8_t* list, int count, int slice,
                            int col0, int width, int blk0, int blk1) {
  constexpr int STEPS = KS ? KS : 1, PARTS = KS ? 2 : 1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int R = a.R;
  // operands of the tokens: this lane's row of each group, ranks 8 q .. of a step
  i32x4 hf[GR][STEPS][PARTS];
  float fac[GR];
  int64_t row[GR];
  const float f = id < 0 ? 0.f : a.factors ? a.factors[id] : 1.f;
#pragma unroll
  for (int g = 0; g < GR; ++g) {
    row[g] = row0 + list[min(g * 16 + col, count - 1)];
    fac[g] = f;
    if (id < 0) continue;
    float h[STEPS][8];
    float big = 0.f;
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      // KS = 0: lanes of q = R / 8 and beyond hold the remaining parts of the first
      const int r = KS ? st * 32 + q * 8 : (q * 8) % R;
      const bool in = KS ? r < R : q * 8 < 2 * R;
      const float* at = a.h + row[g] * a.SR + slice * R + (in ? r : 0);
      f32x4 u = {0.f, 0.f, 0.f, 0.f}, v = u;
#pragma unroll 4
      for (int k = 0; k < a.ksplit; ++k) {
        u += *(const f32x4*)(at + k * a.T * a.SR);
        v += *(const f32x4*)(at + k * a.T * a.SR + 4);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[st][e] = in ? (e < 4 ? u[e] : v[e - 4]) : 0.f;
        big = fmaxf(big, fabsf(h[st][e]));
      }
    }
    int up = 0;
    if constexpr (F16) {
      big = fmaxf(big, __shfl_xor(big, 16));
      big = fmaxf(big, __shfl_xor(big, 32));
      if (big > 0.f && big < __builtin_inff()) up = 14 - __builtin_amdgcn_frexp_expf(big);
      fac[g] = ldexpf(f, -up);
    }
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      float top[8], rest[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = F16 ? ldexpf(h[st][e], up) : h[st][e];
        top[e] = h_to_f32<F16>(f32_to_h<F16>(x));
        rest[e] = fabsf(top[e]) < __builtin_inff() ? x - top[e] : 0.f;
      }
      i32x4 t, m;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        t[w] = pack2<F16>(top[2 * w], top[2 * w + 1]);
        m[w] = pack2<F16>(rest[2 * w], rest[2 * w + 1]);
      }
      if constexpr (KS) {
        hf[g][st][0] = t;
        hf[g][st][1] = m;
      } else {
        hf[g][0][0] = q * 8 < R ? t : m;
      }
    }
  }

  // Blocks of 64 columns: row m of tile j of the weights is column 16 (m / 4) + 4 j
  // + m % 4, so that a lane ends up with 16 neighbours of one token.
  const uint16_t* const B = a.b + ((int64_t)max(id, 0) * a.N + col0) * R;
#pragma unroll 1
  for (int blk = blk0 + wave; blk < blk1; blk += LR_WAVES) {
    const int n0 = blk * 64;
    i32x4 wf[4][STEPS];
    if (id >= 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = min(n0 + 16 * (col >> 2) + 4 * j + (col & 3), width - 1);
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
          const int r = KS ? st * 32 + q * 8 : (q * 8) % R;
          const bool in = KS ? r < R : q * 8 < 2 * R;
          wf[j][st] = *(const i32x4*)(B + (int64_t)n * R + (in ? r : 0));
          if (!in) wf[j][st] = i32x4{0, 0, 0, 0};
        }
      }
    }
    const int n = n0 + q * 16;  // this lane's columns of the slice
    const bool vec = a.vec && n + 16 <= width;
#pragma unroll
    for (int g = 0; g < GR; ++g) {
      const bool live = g * 16 + col < count;
      uint16_t* const op = a.out + row[g] * a.out_s + col0 + n;
      const uint16_t* const bp = a.base ? a.base + row[g] * a.base_s + col0 + n : nullptr;
      float y[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0.f;
      if (bp && live) {
        if (vec) {
          load_h<8, F16>(bp, y);
          load_h<8, F16>(bp + 8, y + 8);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (n + i < width) y[i] = h_to_f32<F16>(bp[i]);
        }
      }
      if (id >= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int st = 0; st < STEPS; ++st)
#pragma unroll
            for (int p = 0; p < PARTS; ++p) acc = mma<F16>(wf[j][st], hf[g][st][p], acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[4 * j + i] = fmaf(acc[i], fac[g], y[4 * j + i]);
        }
      }
      if (!live) continue;
      if (vec) {
        store_h<8, F16>(op, y);
        store_h<8, F16>(op + 8, y + 8);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (n + i < width) op[i] = f32_to_h<F16>(y[i]);
      }
    }
  }
}

template <bool F16, int KS>
__global__ __launch_bounds__(LR_THREADS, 2) void expand_kernel(LoraArgs a) {
  __shared__ uint8_t lists[LR_WAVES][LR_WINDOW];
  uint8_t* const list = lists[__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)];
  const int64_t row0 = (int64_t)(blockIdx.x / a.slots) * LR_WINDOW;
  // chunk of columns -> slice, blocks of 64 in it
  int slice = 0, at = blockIdx.y, col0 = 0;
  while (slice < a.S - 1) {
    const int chunks = ((a.width[slice] + 63) / 64 + a.blocks - 1) / a.blocks;
    if (at < chunks) break;
    at -= chunks;
    col0 += a.width[slice++];
  }
  const int width = a.width[slice];
  const int blk0 = at * a.blocks, blk1 = min(blk0 + a.blocks, (width + 63) / 64);
  each_adapter(a, row0, blockIdx.x % a.slots, [&](int id, uint64_t rows) {
    if (id < 0 && a.base == a.out && a.base_s == a.out_s) return;  // there already
    list_rows(rows, list);
    const int count = __popcll(rows);
    if (count <= 16) expand_rows<F16, KS, 1>(a, id, row0, list, count, slice, col0, width, blk0, blk1);
    else if (count <= 32) expand_rows<F16, KS, 2>(a, id, row0, list, count, slice, col0, width, blk0, blk1);
    else expand_rows<F16, KS, 4>(a, id, row0, list, count, slice, col0, width, blk0, blk1);
  });
}

template <bool F16> hipError_t launch_type(const LoraArgs& a, const LoraPlan& p, hipStream_t s) {
  const unsigned windows = (unsigned)((a.T + LR_WINDOW - 1) / LR_WINDOW * a.slots);
  const dim3 grid(windows, (unsigned)((a.SR + 16 * p.tiles - 1) / (16 * p.tiles)), a.ksplit);
  switch (p.tiles) {
    case 1: hipLaunchKernelGGL((shrink_kernel<F16, 1>), grid, dim3(LR_THREADS), 0, s, a); break;
    case 2: hipLaunchKernelGGL((shrink_kernel<F16, 2>), grid, dim3(LR_THREADS), 0, s, a); break;
    case 3: hipLaunchKernelGGL((shrink_kernel<F16, 3>), grid, dim3(LR_THREADS), 0, s, a); break;
    case 4: hipLaunchKernelGGL((shrink_kernel<F16, 4>), grid, dim3(LR_THREADS), 0, s, a); break;
    default: hipLaunchKernelGGL((shrink_kernel<F16, 6>), grid, dim3(LR_THREADS), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  unsigned chunks = 0;
  for (int i = 0; i < a.S; ++i) chunks += ((a.width[i] + 63) / 64 + a.blocks - 1) / a.blocks;
  const dim3 egrid(windows, chunks);
  switch (a.R <= 16 ? 0 : (a.R + 31) / 32) {
    case 0: hipLaunchKernelGGL((expand_kernel<F16, 0>), egrid, dim3(LR_THREADS), 0, s, a); break;
    case 1: hipLaunchKernelGGL((expand_kernel<F16, 1>), egrid, dim3(LR_THREADS), 0, s, a); break;
    case 2: hipLaunchKernelGGL((expand_kernel<F16, 2>), egrid, dim3(LR_THREADS), 0, s, a); break;
    case 3: hipLaunchKernelGGL((expand_kernel<F16, 3>), egrid, dim3(LR_THREADS), 0, s, a); break;
    default: hipLaunchKernelGGL((expand_kernel<F16, 4>), egrid, dim3(LR_THREADS), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

LoraPlan lora_plan(int64_t T, int64_t K, const int* width, int S, int SR, int64_t n) {
  LoraPlan p;
  const int64_t windows = (T + LR_WINDOW - 1) / LR_WINDOW;
  // An adapter of a window is one workgroup's: as many slots as give each
  // possible one its own, up to about 256 workgroups.
  p.slots = 1;
  const int64_t distinct = std::min({T, n + 1, (int64_t)LR_WINDOW});
  while (p.slots < distinct && p.slots * windows < 256) p.slots *= 2;
  if (p.slots > 1 && p.slots < LR_WINDOW && windows == 1)
    while (p.slots < T && p.slots < LR_WINDOW) p.slots *= 2;
  const int tiles = (SR + 15) / 16;
  p.tiles = tiles <= 4 ? tiles : tiles == 5 || tiles == 6 || tiles >= 9 ? 6 : 4;
  const int64_t parts = (tiles + p.tiles - 1) / p.tiles;
  // k is split until about 512 workgroups have work, but for no less than two steps
  // of 64 for each wave.
  const int64_t busy = windows * std::min(distinct, (int64_t)p.slots) * parts;
  const int64_t most = std::max<int64_t>(1, (K + 511) / 512);
  p.ksplit = std::max<int64_t>(1, std::min({most, (512 + busy - 1) / busy, (int64_t)32}));
  // columns: blocks of 64, a workgroup takes 4 at least
  int64_t blocks = 0;
  for (int i = 0; i < S; ++i) blocks += (width[i] + 63) / 64;
  const int64_t groups = windows * std::min(distinct, (int64_t)p.slots);
  int64_t per = 4;
  while (per < 64 && groups * (blocks / per) > 2048) per *= 2;
  p.blocks = per;
  return p;
}

hipError_t launch_lora(const LoraArgs& a, const LoraPlan& p, bool f16, hipStream_t s) {
  return f16 ? launch_type<true>(a, p, s) : launch_type<false>(a, p, s);
}

}  // namespace lg
