// kernels_score.hip -- log probabilities of given tokens, the entropy of each
// row's distribution and its most likely tokens, from logits [T][V].
//
//   z = x / temperature,  lse = log sum exp z,  logprob = z[token] - lse,
//   entropy = -sum p log p = log S - W / S,
//   S = sum exp(z - m),  W = sum exp(z - m) (z - m)
//
// One pass: every lane keeps its own running maximum m, S and W (rescaled
// when its maximum grows) in 32 bits and base 2, so the values read are
// used once and the row is never written back.
//
// The top k of a row are kept per wave as a sorted list of 64-bit keys, one
// per lane: the value's bits in an order-preserving map above the inverted
// index, so all keys differ, larger means "before", and equal logits go to
// the lower index.  A batch of values is compared with the wave's k-th value
// only by its maximum; the few values that pass are collected in LDS and
// merged into the list by a bitonic network.  The first batch has no k-th
// value yet: the k-th largest of the 64 lane maxima is a lower bound of it.
//
// Memory bound for many rows.  Few rows are split over workgroups; each
// slice writes its sums and list, and a second kernel joins them.
#include "launch.hpp"

namespace lg {
namespace {

constexpr int SC_THREADS = 256;
constexpr int SC_WAVES = 4;
constexpr float LOWEST = -3.402823466e38f;
constexpr float LN2 = 0.693147180559945f;

// Larger key: larger value, then lower index.  -0 and +0 are one value.
__device__ inline uint64_t make_key(float x, uint32_t idx) {
  uint32_t b = __float_as_uint(x + 0.0f);
  b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return ((uint64_t)b << 32) | (uint32_t)~idx;
}
__device__ inline float key_value(uint64_t k) {
  uint32_t b = (uint32_t)(k >> 32);
  b = (b & 0x80000000u) ? b & 0x7FFFFFFFu : ~b;
  return __uint_as_float(b);
}

__device__ inline uint64_t shfl_xor64(uint64_t v, int mask) {
  const uint32_t lo = __shfl_xor((uint32_t)v, mask), hi = __shfl_xor((uint32_t)(v >> 32), mask);
  return ((uint64_t)hi << 32) | lo;
}
__device__ inline uint64_t shfl64(uint64_t v, int lane) {
  const uint32_t lo = __shfl((uint32_t)v, lane), hi = __shfl((uint32_t)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}
__device__ inline uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// One compare-exchange of lanes l and l ^ mask; `up` lanes keep the larger.
__device__ inline uint64_t exchange(uint64_t v, int mask, bool keep_max) {
  const uint64_t w = shfl_xor64(v, mask);
  return (v > w) == keep_max ? v : w;
}
// Bitonic sort of the 64 lanes, descending.
__device__ inline uint64_t sort64(uint64_t v, int lane) {
#pragma unroll
  for (int size = 2; size <= 64; size <<= 1)
#pragma unroll
    for (int m = size >> 1; m > 0; m >>= 1)
      v = exchange(v, m, ((lane & m) == 0) == ((lane & size) == 0 || size == 64));
  return v;
}
// The 64 largest of two descending lists of 64, descending.
__device__ inline uint64_t merge64(uint64_t a, uint64_t b, int lane) {
  uint64_t v = max64(a, shfl64(b, 63 - lane));
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = exchange(v, m, (lane & m) == 0);
  return v;
}

// Sums of one lane, wave or slice: m in logit units, base-2 exponents.
struct Sums {
  float m, s, w;
};
__device__ inline Sums join(const Sums& a, const Sums& b, float c) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float da = fmaxf((a.m - r.m) * c, -1e4f), db = fmaxf((b.m - r.m) * c, -1e4f);
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  r.s = a.s * fa + b.s * fb;
  r.w = fa * (a.w + da * a.s) + fb * (b.w + db * b.s);
  return r;
}

template <int ET> struct Elem;  // 0 bf16, 1 fp16, 2 fp32
template <> struct Elem<0> { static constexpr int SIZE = 2; };
template <> struct Elem<1> { static constexpr int SIZE = 2; };
template <> struct Elem<2> { static constexpr int SIZE = 4; };

template <int ET> __device__ inline float load_one(const void* p, int64_t i) {
  if constexpr (ET == 2) return ((const float*)p)[i];
  else return h_to_f32<ET == 1>(((const uint16_t*)p)[i]);
}

// What a row's results are written from.
template <int ET>
__device__ inline void write_row(const ScoreArgs& a, int64_t t, Sums r, uint64_t list, int lane) {
  const float ls = __builtin_amdgcn_logf(r.s);  // log2
  if (lane == 0) {
    const int tok = a.tokens[t];
    float lp = __builtin_nanf("");
    if (tok >= 0 && tok < a.V) {
      const float x = load_one<ET>(a.logits, t * a.stride + tok);
      lp = (x - r.m) * a.inv_t - ls * LN2;
    }
    a.logprobs[t] = lp;
    if (a.entropy) a.entropy[t] = (ls - r.w / r.s) * LN2;
  }
  if (lane < a.k) {
    if (a.top_ids) a.top_ids[t * a.k + lane] = (int)~(uint32_t)list;
    if (a.top_logprobs)
      a.top_logprobs[t * a.k + lane] = (key_value(list) - r.m) * a.inv_t - ls * LN2;
  }
}

template <int ET>
__global__ __launch_bounds__(SC_THREADS) void score_kernel(ScoreArgs a) {
  constexpr int ES = Elem<ET>::SIZE, EPV = 16 / ES;
  constexpr int U = 32 / EPV;  // 16-byte loads in flight: 32 values a lane
  __shared__ uint64_t found[SC_WAVES][64];
  __shared__ uint64_t lists[SC_WAVES][64];
  __shared__ Sums sums[SC_WAVES];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x / a.nsplit;
  const int split = blockIdx.x % a.nsplit;
  const char* row = (const char*)a.logits + t * a.stride * ES;
  // Rows start at any element: up to EPV - 1 values before the first whole
  // 16 bytes and after the last are taken one by one.
  int head = (int)((16 - ((uintptr_t)row & 15)) & 15) / ES;
  if (head > a.V) head = (int)a.V;
  const int64_t nvec = (a.V - head) / EPV;
  const int rest = (int)(a.V - head - nvec * EPV);
  const int64_t v0 = split * a.slice, v1 = min(nvec, v0 + a.slice);
  const char* body = row + head * ES;
  const int k = a.k;
  const float c = a.c;

  Sums r = {LOWEST, 0.f, 0.f};
  uint64_t list = 0, tau = 0;    // 0 is below every key
  float tau_x = -__builtin_inff();
  int cnt = 0;
  uint64_t* const buf = found[wave];

  // Merge what was found into the list.
  auto flush = [&]() {
    __builtin_amdgcn_wave_barrier();
    uint64_t v = lane < cnt ? buf[lane] : 0;
    __builtin_amdgcn_wave_barrier();
    list = merge64(list, sort64(v, lane), lane);
    cnt = 0;
    const uint64_t kth = shfl64(list, k - 1);
    if (kth > tau) {
      tau = kth;
      tau_x = key_value(kth);
    }
  };
  // Offer one value per lane.
  auto offer = [&](float x, bool valid, uint32_t idx) {
    bool in = valid && x >= tau_x;
    if (!__any(in)) return;
    const uint64_t key = make_key(x, idx);
    in = in && key > tau;
    const uint64_t who = __ballot(in);
    const int n = __popcll(who);
    if (n == 0) return;
    if (cnt + n > 64) flush();
    // the list's k-th may have grown, but what passed before still may stay
    if (in) buf[cnt + __popcll(who & ((1ull << lane) - 1))] = key;
    cnt += n;
  };
  auto add = [&](float x, float m) {
    const float d = (x - m) * c;
    const float e = __builtin_amdgcn_exp2f(d);
    r.s += e;
    r.w += e * fmaxf(d, -1e4f);  // 0 * -inf is no term; a NaN stays in e
  };
  auto grow = [&](float mx) {
    const float m = fmaxf(r.m, mx);
    const float d = fmaxf((r.m - m) * c, -1e4f);
    const float f = __builtin_amdgcn_exp2f(d);
    r.w = f * (r.w + d * r.s);
    r.s *= f;
    r.m = m;
  };

  bool first = true;
  for (int64_t g = v0 + wave * (int64_t)(64 * U); g < v1; g += SC_WAVES * 64 * U) {
    i32x4 raw[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = g + u * 64 + lane;
      ok[u] = v < v1;
      raw[u] = *(const i32x4*)(body + min(v, v1 - 1) * 16);
    }
    float x[U * EPV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (ET == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[u * 4 + i] = __int_as_float(raw[u][i]);
      } else {
        unpack8<ET == 1>(raw[u], x + u * 8);
      }
      if (!ok[u])
#pragma unroll
        for (int i = 0; i < EPV; ++i) x[u * EPV + i] = -__builtin_inff();
    }
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < U * EPV; ++i) mx = fmaxf(mx, x[i]);
    grow(mx);
#pragma unroll
    for (int i = 0; i < U * EPV; ++i) add(x[i], r.m);
    if (k > 0) {
      if (first) {
        const uint64_t kth = shfl64(sort64(make_key(mx, 0), lane), k - 1);
        tau = kth & 0xFFFFFFFF00000000ull;
        tau_x = key_value(kth);
      }
      // Later batches have higher indices: an equal value comes after.
      if (__any(first ? true : mx > tau_x)) {
        const uint32_t base = (uint32_t)(head + g * EPV);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < EPV; ++i)
            offer(x[u * EPV + i], ok[u], base + (u * 64 + lane) * EPV + i);
        if (first || cnt > 32) flush();
      }
    }
    first = false;
  }
  if (split == 0 && wave == 0 && head + rest > 0) {
    const bool ok = lane < head + rest;
    const int64_t at = lane < head ? lane : a.V - rest + (lane - head);
    const float x = ok ? load_one<ET>(row, at) : -__builtin_inff();
    grow(x);
    add(x, r.m);
    if (k > 0) offer(x, ok, (uint32_t)at);
  }
  if (k > 0 && cnt > 0) flush();
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    Sums o = {__shfl_xor(r.m, off), __shfl_xor(r.s, off), __shfl_xor(r.w, off)};
    r = join(r, o, c);
  }
  if (lane == 0) sums[wave] = r;
  lists[wave][lane] = list;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < SC_WAVES; ++w) {
    r = join(r, sums[w], c);
    if (k > 0) list = merge64(list, lists[w][lane], lane);
  }
  if (a.nsplit == 1) {
    write_row<ET>(a, t, r, list, lane);
    return;
  }
  const int64_t p = t * a.nsplit + split;
  if (lane == 0) {
    a.part_sums[p * 3] = r.m;
    a.part_sums[p * 3 + 1] = r.s;
    a.part_sums[p * 3 + 2] = r.w;
  }
  if (lane < k) a.part_keys[p * k + lane] = list;
}

// Joins the slices of a row: one workgroup per row.
template <int ET>
__global__ __launch_bounds__(SC_THREADS) void score_join_kernel(ScoreArgs a) {
  __shared__ uint64_t lists[SC_WAVES][64];
  __shared__ Sums sums[SC_WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  const int k = a.k;
  Sums r = {LOWEST, 0.f, 0.f};
  uint64_t list = 0;
  for (int i = threadIdx.x; i < a.nsplit; i += SC_THREADS) {
    const float* p = a.part_sums + (t * a.nsplit + i) * 3;
    r = join(r, Sums{p[0], p[1], p[2]}, a.c);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    Sums o = {__shfl_xor(r.m, off), __shfl_xor(r.s, off), __shfl_xor(r.w, off)};
    r = join(r, o, a.c);
  }
  if (k > 0) {
    for (int i = wave; i < a.nsplit; i += SC_WAVES) {
      const uint64_t v = lane < k ? a.part_keys[(t * a.nsplit + i) * k + lane] : 0;
      list = merge64(list, v, lane);
    }
  }
  if (lane == 0) sums[wave] = r;
  lists[wave][lane] = list;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < SC_WAVES; ++w) {
    r = join(r, sums[w], a.c);
    if (k > 0) list = merge64(list, lists[w][lane], lane);
  }
  write_row<ET>(a, t, r, list, lane);
}

template <int ET> hipError_t launch_score_t(const ScoreArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((score_kernel<ET>), dim3((unsigned)(a.T * a.nsplit)), dim3(SC_THREADS), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.nsplit == 1) return e;
  hipLaunchKernelGGL((score_join_kernel<ET>), dim3((unsigned)a.T), dim3(SC_THREADS), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Slices of a row: enough workgroups for a few on each of the 256 CUs, and at
// least one batch of every wave in each.
void score_plan(int64_t T, int64_t V, int elem, int* nsplit, int64_t* slice) {
  const int64_t nvec = V / (elem == 2 ? 4 : 8) + 1;
  const int64_t batch = SC_THREADS * (elem == 2 ? 8 : 4);  // 16-byte chunks
  int64_t ns = std::min<int64_t>((1024 + T - 1) / T, (nvec + batch - 1) / batch);
  if (T >= 512) ns = 1;
  ns = std::max<int64_t>(ns, 1);
  *slice = ((nvec + ns - 1) / ns + batch - 1) / batch * batch;
  *nsplit = (int)((nvec + *slice - 1) / *slice);
}

hipError_t launch_score(const ScoreArgs& a, int elem, hipStream_t s) {
  if (elem == 0) return launch_score_t<0>(a, s);
  if (elem == 1) return launch_score_t<1>(a, s);
  return launch_score_t<2>(a, s);
}

}  // namespace lg
