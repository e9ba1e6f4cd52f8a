// kernels_lora.hip -- low-rank adapters of many requests beside a shared
// projection:
//
//   out[t, n] = base[t, n] + f[id] sum_r h[t, r] B[id, n, r],
//   h[t, r] = sum_k x[t, k] A[id, r, k],        id = ids[t]
//
// (a QKV product's slices have their own rows of A: h then is [slices][rank]).
// Two launches: shrink_kernel forms h in 32 bits, expand_kernel adds its product
// with B to the base and rounds once; few rows take both steps in one launch
// (step_kernel).
//
// Rows name their adapters in any order.  A window of 64 rows is one id per lane,
// so that the rows of one adapter are a ballot: a workgroup takes adapters of a
// window, gathers their rows as MFMA columns (16x16x32: rows of A and B are the
// rows, tokens the columns) and so reads an adapter's weights once for all its rows
// of the window.
//
// Bound by bytes: x once, base and out once, the weights of the adapters in use.
// 8191 rows of a 6144-wide QKV product (K = 4096, rank 32, bf16) take 21 us for h
// (3.2 TB/s of x; A comes from the caches for every window) and 46 for the rest (4.4
// TB/s; a large copy reaches 5.1); 300 rows of N = 4099, whose rows are not aligned,
// 7 and 13.  A decode step is a chain of latencies: ids, rows of x and A (131 KB
// for one CU at rank 16), the waves' sums, parts, output: 8.7 us in the kernel for one
// row, of which a workgroup's first to last instruction take 6.8.
#include "launch.hpp"

namespace lg {
namespace {

constexpr int LR_WINDOW = 64;

template <bool F16> __device__ inline f32x4 mma(i32x4 w, i32x4 x, f32x4 c) {
  if constexpr (F16) return Mfma<QK_FP16>::mma(w, x, c);
  else return Mfma<QK_BF16>::mma(w, x, c);
}

__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A barrier that waits for the waves' LDS accesses, but for none of their loads.
__device__ inline void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Calls f(id, mask of its rows) for the adapters of the window, -1 among them, that
// are a slot's: the i-th in the order of their first rows belongs to slot i % slots.
// id and mask are scalar.
//
// Workgroups of one slot follow each other over the windows (the other way round
// the later slots, often empty, would leave whole XCDs idle: workgroups go to
// those in turn).
template <typename F> __device__ inline void each_adapter(const LoraArgs& a, int64_t row0, int slot, F f) {
  const int lane = threadIdx.x & 63;
  const bool live = row0 + lane < a.T;
  int id = live ? a.ids[row0 + lane] : -1;
  if (id < 0 || id >= a.n) id = -1;
  uint64_t todo = __ballot(live);
  for (int i = 0; todo; i = i + 1 == a.slots ? 0 : i + 1) {
    const int mine = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t rows = __ballot(id == mine) & todo;
    todo &= ~rows;
    if (i == slot) f(mine, rows);
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
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;

// Groups of 16 rows, of x or A, that a wave holds in LDS: 64 values of k each, 2 KB.
constexpr int STAGE_GROUPS = 8;
constexpr int staged_groups(int jt, int gr) { return gr == 1 ? jt : jt + gr; }
constexpr int steps_ahead(int jt, int gr) { return STAGE_GROUPS / staged_groups(jt, gr); }

// The products of JT tiles of 16 rows of A with GR groups of 16 tokens over this
// wave's share of the steps [lo, hi) of 64 values of k.  Rows go from memory to
// the wave's own part of LDS, eight lanes to the 128 bytes of a row (16 rows loaded
// straight into operands, a row to a lane, cost 64 accesses of the vector cache for a
// load instead of 8, which bound prompts and decode steps alike); chunks of 16
// bytes are XOR-ed with the row, so that 16 lanes that read one chunk of 16
// rows spread over the banks.  AHEAD steps are on their way at once.  One group of
// tokens, often a single row, goes straight into operands and leaves the room to A.
template <bool F16, int JT, int GR, int WAVES>
__device__ inline void shrink_products(const LoraArgs& a, const uint16_t* A, int j0, int64_t row0,
                                       const uint8_t* list, int count, int g0, int lo, int hi,
                                       char* stage, f32x4 (&acc)[JT][GR]) {
  constexpr int AHEAD = steps_ahead(JT, GR), STAGED = staged_groups(JT, GR), XS = STAGED - JT;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4, r8 = lane >> 3, c = (lane & 7) ^ r8;
  const uint16_t* from[STAGED][2];  // tokens, then rows of A
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int g = 0; g < XS; ++g)
      from[g][i] = a.x + (row0 + list[min((g0 + g) * 16 + i * 8 + r8, count - 1)]) * a.x_s;
#pragma unroll
    for (int j = 0; j < JT; ++j)
      from[XS + j][i] = A + (int64_t)min(j0 + j * 16 + i * 8 + r8, a.SR - 1) * a.K;
  }
  const uint16_t* const xp = a.x + (row0 + list[min(g0 * 16 + col, count - 1)]) * a.x_s;
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int g = 0; g < GR; ++g) acc[j][g] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll 1
  for (int st = lo + wave; st < hi; st += AHEAD * WAVES) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the last batch has been read
    i32x4 x[GR == 1 ? AHEAD : 1][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (u > 0 && st + u * WAVES >= hi) break;
      const int k0 = (st + u * WAVES) * 64, k = k0 + c * 8;
      // (past the end of k a row's first values stand in)
#pragma unroll
      for (int g = 0; g < STAGED; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          __builtin_amdgcn_global_load_lds((global_void*)(from[g][i] + (k < a.K ? k : 0)),
                                           (lds_void*)(stage + (u * STAGED + g) * 2048 + i * 1024), 16, 0, 0);
      if constexpr (GR == 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = k0 + h * 32 + q * 8;
          x[u][h] = *(const i32x4*)(xp + (at < a.K ? at : 0));
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    wave_sync();
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (u > 0 && st + u * WAVES >= hi) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = (st + u * WAVES) * 64 + h * 32 + q * 8 < a.K;
        i32x4 f[STAGED];
#pragma unroll
        for (int g = 0; g < STAGED; ++g) {
          f[g] = *(const i32x4*)(stage + (u * STAGED + g) * 2048 + col * 128 + (((h * 4 + q) ^ (col & 7)) << 4));
          if (!in) f[g] = i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int g = 0; g < GR; ++g) {
            if constexpr (GR == 1) acc[j][g] = mma<F16>(f[j], in ? x[u][h] : i32x4{0, 0, 0, 0}, acc[j][g]);
            else acc[j][g] = mma<F16>(f[XS + j], f[g], acc[j][g]);
          }
      }
    }
    wave_sync();
  }
}

constexpr int SH_WAVES = 4;

// A workgroup: JT tiles of rows of A and a part of k, which its waves share out.
template <bool F16, int JT, int GR>
__device__ void shrink_rows(const LoraArgs& a, const uint16_t* A, int64_t row0, const uint8_t* list, int count,
                            float* out, char* lds) {
  f32x4* const sums = (f32x4*)lds;  // (after the loops over k)
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j0 = blockIdx.y * JT * 16;
  f32x4 acc[JT][GR];
  const int lo = blockIdx.z * a.ksteps, hi = min(lo + a.ksteps, (a.K + 63) >> 6);
  shrink_products<F16, JT, GR, SH_WAVES>(a, A, j0, row0, list, count, 0, lo, hi,
                                             lds + wave * STAGE_GROUPS * 2048, acc);
  // The waves' sums meet in LDS, 16 token rows at a time, in the order of the waves.
#pragma unroll
  for (int g = 0; g < GR; ++g) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < JT; ++j) sums[(wave * JT + j) * 64 + lane] = acc[j][g];
    __syncthreads();
    const int p = g * 16 + (lane & 15);
#pragma unroll 1
    for (int j = wave; j < JT; j += SH_WAVES) {
      f32x4 v = sums[j * 64 + lane];
#pragma unroll
      for (int w = 1; w < SH_WAVES; ++w) v += sums[(w * JT + j) * 64 + lane];
      const int r = j0 + j * 16 + (lane >> 4) * 4;
      if (p < count && r < a.SR) *(f32x4*)(out + (row0 + list[p]) * a.SR + r) = v;
    }
  }
}

template <bool F16, int JT>
__global__ __launch_bounds__(64 * SH_WAVES, 2) void shrink_kernel(LoraArgs a) {
  __shared__ __align__(16) char lds[SH_WAVES * STAGE_GROUPS * 2048];
  __shared__ uint8_t lists[SH_WAVES][LR_WINDOW];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const list = lists[wave];
  const unsigned windows = gridDim.x / a.slots;
  const int64_t row0 = (int64_t)(blockIdx.x % windows) * LR_WINDOW;
  float* const out = a.h + (int64_t)blockIdx.z * a.T * a.SR;
  each_adapter(a, row0, blockIdx.x / windows, [&](int id, uint64_t rows) {
    if (id < 0) return;
    list_rows(rows, list);
    __syncthreads();  // (the last adapter's sums are not read any more)
    const int count = __popcll(rows);
    const uint16_t* const A = a.a + (int64_t)id * a.SR * a.K;
    if (count <= 16) shrink_rows<F16, JT, 1>(a, A, row0, list, count, out, lds);
    else if (count <= 32) shrink_rows<F16, JT, 2>(a, A, row0, list, count, out, lds);
    else shrink_rows<F16, JT, 4>(a, A, row0, list, count, out, lds);
  });
}

// ------------------------------------------------------------------ expand
// h of a row is rounded to 16 bits twice, as a leading and a remaining part (16 and
// more bits of it in bf16, 22 in fp16): of one part alone the sum would be off by
// its rounding, which is of the size of the output's own.  fp16 has no range
// for it, so a row's h is brought to below 2^14 by a power of two first.
//
// In LDS the parts of 64 rows stand as the operands of the product: KS steps of 32
// ranks for each part, or, for ranks up to 16 (KS = 0), both parts in one step.
template <int KS> struct Parts {
  static constexpr int STEPS = KS ? KS : 1, COUNT = KS ? 2 : 1;
  static constexpr int ROW = STEPS * 64 + 16;  // bytes; rows spread over the banks
  static constexpr int BYTES = COUNT * LR_WINDOW * ROW;
};

// Rows p0 up to `end` of h -> parts and factors: at(p, r) gives eight values of row p.
template <bool F16, int KS, int THREADS, typename At>
__device__ inline void split_rows(const LoraArgs& a, float f, int p0, int end, char* parts, float* factor, At at) {
  constexpr int CHUNKS = Parts<KS>::STEPS * 4;  // of eight ranks
  constexpr int ROW = Parts<KS>::ROW;
  // CHUNKS is 4, 8, 12 or 16: lanes of a row
  constexpr int LPR = CHUNKS <= 4 ? 4 : CHUNKS <= 8 ? 8 : 16;
  const int c = threadIdx.x % LPR;
#pragma unroll 1
  for (int p = p0 + threadIdx.x / LPR; p < (end + 15) / 16 * 16; p += THREADS / LPR) {
    const int r = KS ? c * 8 : c * 8 % a.R;  // KS = 0: chunks from R / 8 on hold the remaining parts
    const bool in = p < end && (KS ? r < a.R : c * 8 < 2 * a.R);
    float h[8] = {};
    if (in) at(p, r, h);
    int up = 0;
    if constexpr (F16) {
      float big = amax8(h);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, LPR));
      if (big > 0.f && big < __builtin_inff()) up = 14 - __builtin_amdgcn_frexp_expf(big);
    }
    if (c == 0) factor[p] = F16 ? ldexpf(f, -up) : f;
    i32x4 top, rest;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float x[2], t[2], m[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[e] = F16 ? ldexpf(h[2 * w + e], up) : h[2 * w + e];
        t[e] = h_to_f32<F16>(f32_to_h<F16>(x[e]));
        m[e] = fabsf(t[e]) < __builtin_inff() ? x[e] - t[e] : 0.f;
      }
      top[w] = pack2<F16>(t[0], t[1]);
      rest[w] = pack2<F16>(m[0], m[1]);
    }
    if constexpr (KS) {
      if (c < CHUNKS) {
        *(i32x4*)(parts + p * ROW + c * 16) = top;
        *(i32x4*)(parts + (LR_WINDOW + p) * ROW + c * 16) = rest;
      }
    } else {
      *(i32x4*)(parts + p * ROW + c * 16) = c * 8 < a.R ? top : rest;
    }
  }
}

constexpr int TILE_STRIDE = 68;  // values of a token's 64 columns in LDS
constexpr int TILE_VALUES = 16 * TILE_STRIDE;

// base + factor h B^T for the blocks [blk0, blk1) of 64 columns of a slice.  The
// waves take units of a block and GROUPS groups of 16 tokens in turn; load() of a
// wave's first unit, which needs nothing of h, goes out before h is formed.  A
// product goes through the wave's LDS, so that eight lanes hold the 128 bytes
// of a token's row (or, where rows are not aligned, 64 lanes 64 neighbouring
// values).
template <bool F16, int KS, bool VEC, int WAVES> struct Adder {
  static constexpr int STEPS = Parts<KS>::STEPS, COUNT = Parts<KS>::COUNT, ROW = Parts<KS>::ROW;
  static constexpr int GROUPS = VEC ? 2 : 1;
  const LoraArgs& a;
  const uint16_t* B;
  const uint8_t* list;
  int64_t row0;
  int count, col0, width, blk0, gs, unit, units;
  i32x4 w[4][STEPS];
  i32x4 wide[GROUPS][2];                // VEC: eight values of rows lane / 8 and 8 further
  uint16_t single[VEC ? 1 : 16];        // or a value of each row

  __device__ inline Adder(const LoraArgs& args, int id, int64_t r0, const uint8_t* rows, int n, int c0, int wd,
                          int b0, int b1)
      : a(args), B(args.b + ((int64_t)id * args.N + c0) * args.R), list(rows), row0(r0), count(n), col0(c0),
        width(wd), blk0(b0) {
    gs = (count + 16 * GROUPS - 1) / (16 * GROUPS);
    units = gs * (b1 - b0);
    unit = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (unit < units) load();
  }
  __device__ inline int lane() const { return threadIdx.x & 63; }
  // columns of this lane, from the slice's first
  __device__ inline int column() const { return (blk0 + unit / gs) * 64 + (VEC ? (lane() & 7) * 8 : lane()); }
  __device__ inline bool inside(int n) const { return VEC ? n + 8 <= width : n < width; }
  __device__ inline int64_t row_of(int p) const { return row0 + list[min(p, count - 1)]; }

  __device__ inline void load() {
    const int n0 = (blk0 + unit / gs) * 64, g0 = unit % gs * GROUPS, col = lane() & 15, q = lane() >> 4;
    const int n = column();
    if (a.base) {  // (lanes without a value load another instead: see run())
      if constexpr (VEC) {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint16_t* const from =
                a.base + row_of((g0 + g) * 16 + i * 8 + (lane() >> 3)) * a.base_s + col0 + n;
            wide[g][i] = *(const i32x4*)(inside(n) ? from : B);
          }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) single[i] = a.base[row_of(g0 * 16 + i) * a.base_s + col0 + min(n, width - 1)];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const int r = KS ? st * 32 + q * 8 : q * 8 % a.R;
        const bool in = KS ? r < a.R : q * 8 < 2 * a.R;
        w[j][st] = *(const i32x4*)(B + (int64_t)min(n0 + 16 * j + col, width - 1) * a.R + (in ? r : 0));
      }
  }
  __device__ inline void finish(const char* parts, const float* factor, float* tile) {
    const int g0 = unit % gs * GROUPS, col = lane() & 15, q = lane() >> 4, n = column();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
        if (KS ? st * 32 + q * 8 >= a.R : q * 8 >= 2 * a.R) w[j][st] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const float f = factor[(g0 + g) * 16 + col];
      f32x4 acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
#pragma unroll
        for (int p = 0; p < COUNT; ++p) {
          const i32x4 h = *(const i32x4*)(parts + (p * LR_WINDOW + (g0 + g) * 16 + col) * ROW + st * 64 + q * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mma<F16>(w[j][st], h, acc[j]);
        }
      wave_sync();  // (the last tile's readers are done)
#pragma unroll
      for (int j = 0; j < 4; ++j) *(f32x4*)(tile + col * TILE_STRIDE + 16 * j + 4 * q) = acc[j] * f;
      wave_sync();
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = (g0 + g) * 16 + i * 8 + (lane() >> 3);
          if (p >= count || n >= width) continue;
          const float* const src = tile + (i * 8 + (lane() >> 3)) * TILE_STRIDE + (lane() & 7) * 8;
          uint16_t* const op = a.out + row_of(p) * a.out_s + col0 + n;
          if (inside(n)) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = src[e];
            if (a.base) {
              float x[8];
              unpack8<F16>(wide[g][i], x);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] += x[e];
            }
            store_h<8, F16>(op, y);
          } else {  // the last, partial eight of the slice
            const uint16_t* const bp = a.base + row_of(p) * a.base_s + col0 + n;
#pragma unroll 1
            for (int e = 0; n + e < width; ++e)
              op[e] = f32_to_h<F16>(src[e] + (a.base ? h_to_f32<F16>(bp[e]) : 0.f));
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (g0 * 16 + i < count && inside(n))
            a.out[row_of(g0 * 16 + i) * a.out_s + col0 + n] =
                f32_to_h<F16>(tile[i * TILE_STRIDE + lane()] + (a.base ? h_to_f32<F16>(single[i]) : 0.f));
      }
    }
  }
  __device__ inline void run(const char* parts, const float* factor, float* tile) {
    // Matrix instructions write all lanes, whether or not they are switched off, so a
    // wave stays together here.  A condition of a lane's own between one turn and the
    // next (as "this lane's column is inside" at load()'s loads was) let the compiler
    // make a loop of its own for the lanes outside, whose products overwrote registers
    // of the waiting ones, addresses among them.
    while (unit < units) {
      finish(parts, factor, tile);
      __builtin_amdgcn_wave_barrier();
      unit += WAVES;
      if (unit < units) load();
      __builtin_amdgcn_wave_barrier();
    }
  }
};

// Rows without an adapter: the base, or zeros.
template <bool VEC, int WAVES>
__device__ inline void copy_rows(const LoraArgs& a, int64_t row0, const uint8_t* list, int count, int n0, int n1) {
  if (a.base == a.out && a.base_s == a.out_s) return;  // there already
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll 1
  for (int p = wave; p < count; p += WAVES) {
    const int64_t row = row0 + list[p];
    const uint16_t* const bp = a.base ? a.base + row * a.base_s : nullptr;
    uint16_t* const op = a.out + row * a.out_s;
    const int whole = VEC ? n0 + (n1 - n0) / 8 * 8 : n0;
    for (int n = n0 + lane * 8; n < whole; n += 512)
      *(i32x4*)(op + n) = bp ? *(const i32x4*)(bp + n) : i32x4{0, 0, 0, 0};
    for (int n = whole + lane; n < n1; n += 64) op[n] = bp ? bp[n] : 0;
  }
}

// What a workgroup of column chunk `at` covers: blocks [blk0, blk1) of a slice.
struct Chunk {
  int slice, col0, width, blk0, blk1;
};
__device__ inline Chunk find_chunk(const LoraArgs& a, int at) {
  Chunk c;
  c.slice = c.col0 = 0;
  while (c.slice < a.S - 1) {
    const int chunks = ((a.width[c.slice] + 63) / 64 + a.blocks - 1) / a.blocks;
    if (at < chunks) break;
    at -= chunks;
    c.col0 += a.width[c.slice++];
  }
  c.width = a.width[c.slice];
  c.blk0 = at * a.blocks;
  c.blk1 = min(c.blk0 + a.blocks, (c.width + 63) / 64);
  return c;
}

constexpr int EX_WAVES = 4;

template <bool F16, int KS, bool VEC>
__global__ __launch_bounds__(64 * EX_WAVES, 4) void expand_kernel(LoraArgs a) {
  __shared__ uint8_t lists[EX_WAVES][LR_WINDOW];
  __shared__ __align__(16) float tiles[EX_WAVES][TILE_VALUES];
  __shared__ __align__(16) char parts[Parts<KS>::BYTES];
  __shared__ float factor[LR_WINDOW];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const list = lists[wave];
  const unsigned windows = gridDim.x / a.slots;
  const int64_t row0 = (int64_t)(blockIdx.x % windows) * LR_WINDOW;
  const Chunk c = find_chunk(a, blockIdx.y);
  each_adapter(a, row0, blockIdx.x / windows, [&](int id, uint64_t rows) {
    list_rows(rows, list);
    const int count = __popcll(rows);
    if (id < 0) {
      copy_rows<VEC, EX_WAVES>(a, row0, list, count, c.col0 + c.blk0 * 64, c.col0 + min(c.blk1 * 64, c.width));
      return;
    }
    Adder<F16, KS, VEC, EX_WAVES> adder(a, id, row0, list, count, c.col0, c.width, c.blk0, c.blk1);
    lds_barrier();  // (the last adapter's parts are not read any more)
    split_rows<F16, KS, 64 * EX_WAVES>(a, a.factors ? a.factors[id] : 1.f, 0, count, parts, factor,
                                       [&](int p, int r, float* h) {
      const float* at = a.h + (row0 + list[p]) * a.SR + c.slice * a.R + r;
      f32x4 u = {0.f, 0.f, 0.f, 0.f}, v = u;
#pragma unroll 4
      for (int k = 0; k < a.ksplit; ++k, at += a.T * a.SR) {
        u += *(const f32x4*)at;
        v += *(const f32x4*)(at + 4);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = e < 4 ? u[e] : v[e - 4];
    });
    lds_barrier();
    adder.run(parts, factor, tiles[wave]);
  });
}

// --------------------------------------------------------------- few rows
// Both products in one launch: a workgroup forms h of its slice by itself, eight
// waves sharing k, and adds its columns.  The rows of A are read once for every
// chunk of columns instead of once, but from the caches, and there is no second
// launch to wait for.
constexpr int ST_WAVES = 8;

template <bool F16, int KS> struct StepLds {
  static constexpr int JT = KS ? KS * 2 : 1;  // tiles of 16 ranks
  static constexpr int H_ROW = JT * 16 + 4;
  static constexpr int H = 16 * H_ROW * 4;
  // rows on their way, then the waves' sums, then the tiles of the second product
  static constexpr int STAGE = steps_ahead(JT, 1) * JT * 2048;
  static constexpr int SHARED = ST_WAVES * STAGE;
  static constexpr int BYTES = SHARED + Parts<KS>::BYTES + H + LR_WINDOW * 4 + ST_WAVES * LR_WINDOW;
  static_assert(ST_WAVES * JT * 1024 <= SHARED && ST_WAVES * TILE_VALUES * 4 <= SHARED, "");
};

template <bool F16, int KS, bool VEC>
__global__ __launch_bounds__(64 * ST_WAVES, 1) void step_kernel(LoraArgs a) {
  using L = StepLds<F16, KS>;
  extern __shared__ __align__(16) char shared[];
  f32x4* const sums = (f32x4*)shared;
  char* const parts = shared + L::SHARED;
  float* const hs = (float*)(parts + Parts<KS>::BYTES);
  float* const factor = (float*)((char*)hs + L::H);
  uint8_t* const lists = (uint8_t*)(factor + LR_WINDOW);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const list = lists + wave * LR_WINDOW;
  const unsigned windows = gridDim.x / a.slots;
  const int64_t row0 = (int64_t)(blockIdx.x % windows) * LR_WINDOW;
  const Chunk c = find_chunk(a, blockIdx.y);
  each_adapter(a, row0, blockIdx.x / windows, [&](int id, uint64_t rows) {
    list_rows(rows, list);
    const int count = __popcll(rows);
    if (id < 0) {
      copy_rows<VEC, ST_WAVES>(a, row0, list, count, c.col0 + c.blk0 * 64, c.col0 + min(c.blk1 * 64, c.width));
      return;
    }
    const uint16_t* const A = a.a + (int64_t)id * a.SR * a.K;
    const float f = a.factors ? a.factors[id] : 1.f;
    Adder<F16, KS, VEC, ST_WAVES> adder(a, id, row0, list, count, c.col0, c.width, c.blk0, c.blk1);
#pragma unroll 1
    for (int g = 0; g * 16 < count; ++g) {
      f32x4 acc[L::JT][1];
      lds_barrier();  // (tiles and sums of before are not read any more)
      shrink_products<F16, L::JT, 1, ST_WAVES>(a, A, c.slice * a.R, row0, list, count, g, 0, (a.K + 63) >> 6,
                                               shared + wave * L::STAGE, acc);
      lds_barrier();
#pragma unroll
      for (int j = 0; j < L::JT; ++j) sums[(wave * L::JT + j) * 64 + lane] = acc[j][0];
      lds_barrier();
      for (int j = wave; j < L::JT; j += ST_WAVES) {
        f32x4 v = sums[j * 64 + lane];
#pragma unroll
        for (int w = 1; w < ST_WAVES; ++w) v += sums[(w * L::JT + j) * 64 + lane];
        *(f32x4*)(hs + (lane & 15) * L::H_ROW + j * 16 + (lane >> 4) * 4) = v;
      }
      lds_barrier();
      split_rows<F16, KS, 64 * ST_WAVES>(a, f, g * 16, min(g * 16 + 16, count), parts, factor,
                                         [&](int p, int r, float* h) {
        const float* const at = hs + (p & 15) * L::H_ROW + r;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = at[e];
      });
    }
    lds_barrier();
    adder.run(parts, factor, (float*)shared + wave * TILE_VALUES);
  });
}

template <bool F16, int KS, bool VEC> hipError_t launch_step(const LoraArgs& a, dim3 grid, hipStream_t s) {
  constexpr size_t lds = StepLds<F16, KS>::BYTES;
  const hipError_t e = opt_in_lds((const void*)step_kernel<F16, KS, VEC>, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((step_kernel<F16, KS, VEC>), grid, dim3(64 * ST_WAVES), lds, s, a);
  return hipGetLastError();
}

template <bool F16, bool VEC> hipError_t launch_type(const LoraArgs& a, const LoraPlan& p, hipStream_t s) {
  const unsigned windows = (unsigned)((a.T + LR_WINDOW - 1) / LR_WINDOW * a.slots);
  unsigned chunks = 0;
  for (int i = 0; i < a.S; ++i) chunks += ((a.width[i] + 63) / 64 + a.blocks - 1) / a.blocks;
  const int ks = a.R <= 16 ? 0 : (a.R + 31) / 32;
  const dim3 out_grid(windows, chunks);
  if (p.step) {
    return ks ? launch_step<F16, 1, VEC>(a, out_grid, s) : launch_step<F16, 0, VEC>(a, out_grid, s);
  }
  const dim3 grid(windows, (unsigned)((a.SR + 16 * p.tiles - 1) / (16 * p.tiles)), a.ksplit);
  const dim3 in_block(64 * SH_WAVES), block(64 * EX_WAVES);
  switch (p.tiles) {
    case 1: hipLaunchKernelGGL((shrink_kernel<F16, 1>), grid, in_block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((shrink_kernel<F16, 2>), grid, in_block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((shrink_kernel<F16, 3>), grid, in_block, 0, s, a); break;
    default: hipLaunchKernelGGL((shrink_kernel<F16, 4>), grid, in_block, 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  switch (ks) {
    case 0: hipLaunchKernelGGL((expand_kernel<F16, 0, VEC>), out_grid, block, 0, s, a); break;
    case 1: hipLaunchKernelGGL((expand_kernel<F16, 1, VEC>), out_grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((expand_kernel<F16, 2, VEC>), out_grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((expand_kernel<F16, 3, VEC>), out_grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((expand_kernel<F16, 4, VEC>), out_grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

LoraPlan lora_plan(int64_t T, int64_t K, const int* width, int S, int R, int64_t n) {
  LoraPlan p;
  const int SR = S * R;
  const int64_t windows = (T + LR_WINDOW - 1) / LR_WINDOW;
  // A workgroup for each adapter that a window can have, up to about 256 of them; one
  // for all from 64 windows on.  That is for runs of rows, where most of the others
  // would find none (4096 rows, three slices of 6144 columns, rank 16, 16 adapters: 46 us
  // and 62 with four slots a window); for rows in any order it costs (198 us and 112).
  const int64_t distinct = std::min({T, n + 1, (int64_t)LR_WINDOW});
  p.slots = windows >= 64 ? 1 : std::max<int64_t>(1, std::min(distinct, 256 / windows));
  const int64_t groups = windows * p.slots;
  int64_t blocks = 0;
  for (int i = 0; i < S; ++i) blocks += (width[i] + 63) / 64;
  // One launch for few rows.  Each of its workgroups reads its slice of A by itself and
  // takes 16 rows of an adapter at a time, and a CU holds one: up to two rounds of
  // them, ranks up to 32.  (K = N = 4096, rank 16, us a call in one launch and in two: 1
  // row 8 and 10, 16 rows of 16 adapters 9 and 11, 48 of 24 10 and 17, 64 of 64 22 and
  // 27.  N = 6144: 504 workgroups for 42 rows 20 and 23, 528 for 44 28 and 20; 32 rows of
  // 32 with N = 14336 35 and 19.  Rank 64: 1 row 12.5 and 12.4, 16 of 16 14 and 12.)
  // Beyond 16 rows, up to eight rows for each adapter that there is: how many of
  // them the rows name is on the device.  Rows that name them all or any at random fit
  // that (64 rows of 64 adapters, of which 40 are named: 20 and 22 us, 16 16 and 16, 8
  // 15 and 14; two adapters 23 and 11: two launches by the rule).  One that many rows
  // share does not: 64 rows of 4 of the 64 take 19 and 14 us, of one 34 and 15, 16 rows
  // at a time in one workgroup for each 512 columns.
  p.step = T <= LR_WINDOW && R <= 32 && (T <= 16 || T <= 8 * n) && groups * ((blocks + 7) / 8) <= 2 * 256;
  p.tiles = p.ksteps = p.ksplit = 1;
  p.blocks = 8;
  if (p.step) return p;
  const int tiles = (SR + 15) / 16;
  const int64_t parts = (tiles + 3) / 4;
  p.tiles = (tiles + parts - 1) / parts;
  // k is split until there are about 512 workgroups (8191 rows of K = 4096, three slices
  // of rank 32, both launches: 67 us, and 74 with 256, 75 with 1024), but for no less
  // than two steps of 64 for each wave.  Slots that find no adapter count too (300 rows
  // of 5 of 64 adapters, rank 16: 21 us, and 23 if only windows count; 1000 rows of 10, rank
  // 32: 27 and 26).
  const int64_t steps = (K + 63) / 64, busy = groups * parts;
  const int64_t want = std::min<int64_t>((512 + busy - 1) / busy, 32);
  p.ksteps = std::max<int64_t>((steps + want - 1) / want, 2 * SH_WAVES);
  p.ksplit = (steps + p.ksteps - 1) / p.ksteps;
  // blocks of columns per workgroup: about 2048 workgroups (the same call: 84 us with 512,
  // 71 with 4096; 2000 rows of rank 64 54, 35 and 33)
  p.blocks = 1;
  while (p.blocks < 64 && groups * (blocks / p.blocks) > 2048) p.blocks *= 2;
  return p;
}

hipError_t launch_lora(const LoraArgs& a, const LoraPlan& p, bool f16, bool vec, hipStream_t s) {
  if (f16) return vec ? launch_type<true, true>(a, p, s) : launch_type<true, false>(a, p, s);
  return vec ? launch_type<false, true>(a, p, s) : launch_type<false, false>(a, p, s);
}

}  // namespace lg
