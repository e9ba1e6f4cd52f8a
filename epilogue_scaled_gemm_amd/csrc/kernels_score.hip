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
// The top k of a row: keys of 64 bits, the value's bits in an order-preserving
// map above the inverted index, so all differ, larger means "before", and
// equal logits go to the lower index.  The pass over the row only notes the
// maximum of every 16 lanes of every batch.  The k-th largest of (groups of)
// those maxima is a lower bound of the k-th value; the few batches that reach
// it are read again, and their values at or above it collected in LDS, sorted
// by a bitonic network into the wave's list, and the lists merged.
//
// Memory bound for many rows (2048 of 131072 logits in bf16, top 8: 111 us,
// 4.8 TB/s); a chain of latencies for few, which are split over workgroups (one
// row of 32003: 10 us with the call around it; 48 rows of 128259 in 32 bits, top
// 20: 21 us, of which reading is 5).  A slice writes its sums and list, and the
// workgroup that arrives last joins the row's slices.
#include "launch.hpp"

namespace lg {
namespace {

constexpr int SC_THREADS = 256;
constexpr int SC_WAVES = 4;
constexpr int FOUND = 128;  // keys a wave collects between merges
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

// The value of lane l ^ M: moves within a row of 16 lanes and swaps of rows,
// without a trip through LDS.
template <int M> __device__ inline uint32_t lane_xor(uint32_t v) {
  if constexpr (M == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
  if constexpr (M == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
  if constexpr (M == 4)  // mirrored within 8, then within 4
    return __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true), 0x1B, 0xF,
                                    0xF, true);
  if constexpr (M == 8) return __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, true);
  if constexpr (M == 16) {
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return threadIdx.x & 16 ? r[0] : r[1];
  }
  if constexpr (M == 32) {
    auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return threadIdx.x & 32 ? r[0] : r[1];
  }
}
template <int M> __device__ inline float lane_xor(float v) {
  return __uint_as_float(lane_xor<M>(__float_as_uint(v)));
}
template <int M> __device__ inline uint64_t lane_xor(uint64_t v) {
  return ((uint64_t)lane_xor<M>((uint32_t)(v >> 32)) << 32) | lane_xor<M>((uint32_t)v);
}
__device__ inline uint64_t shfl64(uint64_t v, int lane) {
  const uint32_t lo = __shfl((uint32_t)v, lane), hi = __shfl((uint32_t)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}

// Bitonic steps: lanes of `size` in descending order after step 1.  T is a
// key or a value.
template <int SIZE, int M, typename T> __device__ inline T bitonic(T v, int lane) {
  const T w = lane_xor<M>(v);
  const bool keep_max = ((lane & M) == 0) == ((lane & SIZE) == 0 || SIZE == 64);
  v = (v > w) == keep_max ? v : w;
  if constexpr (M > 1) return bitonic<SIZE, M / 2>(v, lane);
  return v;
}
// The 64 lanes' values (or those of the first LAST), descending.
template <int SIZE = 2, int LAST = 64, typename T> __device__ inline T sort64(T v, int lane) {
  v = bitonic<SIZE, SIZE / 2>(v, lane);
  if constexpr (SIZE < LAST) return sort64<SIZE * 2, LAST>(v, lane);
  return v;
}
// The 64 largest of two descending lists of 64, descending.
__device__ inline uint64_t merge64(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = shfl64(b, 63 - lane);
  return bitonic<64, 32>(a > r ? a : r, lane);
}
// A value that at least k of the wave's values are not below, if k lanes have
// one: the least maximum of 8 groups of lanes, of 16, or the k-th lane's value.
// (Six steps instead of the 21 of a sort, for about 22 values above the bound
// instead of 9, at k = 8.)
__device__ inline float at_least(float mx, int k, int lane) {
  if (k > 16) return __shfl(sort64(mx, lane), k - 1);
  mx = fmaxf(mx, lane_xor<1>(mx));
  mx = fmaxf(mx, lane_xor<2>(mx));
  const float other = lane_xor<4>(mx);
  mx = k <= 8 ? fmaxf(mx, other) : fminf(mx, other);
  mx = fminf(mx, lane_xor<8>(mx));
  mx = fminf(mx, lane_xor<16>(mx));
  return fminf(mx, lane_xor<32>(mx));
}

// Sums of one lane, wave or slice, relative to the maximum m (a logit).
// Exponents are base 2: a value's is x c - M with c = log2(e) / temperature and
// M = m c, rounded; the product x c is exact in the FMA, so the difference is
// rounded once.  All of them are then off by what M was rounded by, which
// cancels in the results as long as it is no large exponent itself: it is
// below one for M up to 2^24.  Beyond that (logits that an additive mask has
// moved far from zero) exponents are (x - m) c.
struct Sums {
  float m, s, w;
};
__device__ inline float frame(float m, float c) {
  float mc = m * c;
  asm volatile("" : "+v"(mc));  // rounded here: never part of another FMA
  return mc;
}
__device__ inline bool in_range(float mc) { return fabsf(mc) < 16777216.f; }
__device__ inline float rel(float x, float m, float c) {
  const float mc = frame(m, c);
  return in_range(mc) ? fmaf(x, c, -mc) : (x - m) * c;
}
// What exponents relative to `from` lose when they are taken relative to `to`.
__device__ inline float shift(float from, float to, float c) {
  const float f = frame(from, c), t = frame(to, c);
  return fmaxf(in_range(f) && in_range(t) ? f - t : (from - to) * c, -1e4f);
}
__device__ inline Sums join(const Sums& a, const Sums& b, float c) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float da = shift(a.m, r.m, c), db = shift(b.m, r.m, c);
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  r.s = a.s * fa + b.s * fb;
  r.w = fa * (a.w + da * a.s) + fb * (b.w + db * b.s);
  return r;
}
template <int M, typename T> __device__ inline T max_lanes(T v) {
  const T w = lane_xor<M>(v);
  v = v < w ? w : v;
  if constexpr (M > 1) return max_lanes<M / 2>(v);
  return v;
}
template <int M> __device__ inline float add_lanes(float v) {
  v += lane_xor<M>(v);
  if constexpr (M > 1) return add_lanes<M / 2>(v);
  return v;
}
// The 64 lanes' sums as one: taken relative to the common maximum, then added.
__device__ inline Sums join_lanes(Sums r, float c) {
  const float m = max_lanes<32>(r.m);
  const float d = shift(r.m, m, c);
  const float f = __builtin_amdgcn_exp2f(d);
  return Sums{m, add_lanes<32>(r.s * f), add_lanes<32>(f * (r.w + d * r.s))};
}

template <int ET> struct Elem;  // 0 bf16, 1 fp16, 2 fp32
template <> struct Elem<0> { static constexpr int SIZE = 2; };
template <> struct Elem<1> { static constexpr int SIZE = 2; };
template <> struct Elem<2> { static constexpr int SIZE = 4; };

template <int ET> __device__ inline float load_one(const void* p, int64_t i) {
  if constexpr (ET == 2) return ((const float*)p)[i];
  else return h_to_f32<ET == 1>(((const uint16_t*)p)[i]);
}

// A row's results.  A row with NaN can have fewer values in order than places:
// those that are left hold their own number for an index (k is at most the
// vocabulary's size), and the key 0 stands for NaN.
template <int ET>
__device__ inline void write_row(const ScoreArgs& a, int64_t t, Sums r, uint64_t list, int lane) {
  const float ls = __builtin_amdgcn_logf(r.s);  // log2
  auto logprob = [&](float x) {
    const float d = rel(x, r.m, a.c);
    // (the lowest finite values overflow in base 2 before they do in base e)
    return fabsf(d) < 1e30f || d != d ? (d - ls) * LN2 : (x - r.m) * a.inv_t - ls * LN2;
  };
  if (lane == 0) {
    const int tok = a.tokens[t];
    a.logprobs[t] = tok >= 0 && tok < a.V ? logprob(load_one<ET>(a.logits, t * a.stride + tok))
                                          : __builtin_nanf("");
    if (a.entropy) a.entropy[t] = (ls - r.w / r.s) * LN2;
  }
  if (lane < a.k) {
    if (a.top_ids) a.top_ids[t * a.k + lane] = list ? (int)~(uint32_t)list : lane;
    if (a.top_logprobs) a.top_logprobs[t * a.k + lane] = logprob(key_value(list));
  }
}

// Keys that a wave collects in LDS (in any order) and the 64 largest of what it
// merged before, descending.
struct Best {
  uint64_t* buf;         // FOUND keys
  uint64_t list = 0;
  int cnt = 0;
  bool merged = false;   // the list holds something

  __device__ inline void put(uint64_t key, bool in, int lane) {  // there is room for 64
    const uint64_t who = __ballot(in);
    if (in) buf[cnt + __popcll(who & ((1ull << lane) - 1))] = key;
    cnt += __popcll(who);
  }
  __device__ inline void merge(int lane) {
    __builtin_amdgcn_wave_barrier();
    for (int at = 0; at < cnt; at += 64) {
      uint64_t v = at + lane < cnt ? buf[at + lane] : 0;
      // few keys lie in the first lanes; the others' zeros are in order
      v = cnt - at <= 16   ? sort64<2, 16>(v, lane)
          : cnt - at <= 32 ? sort64<2, 32>(v, lane)
                           : sort64<2, 64>(v, lane);
      list = merged ? merge64(list, v, lane) : v;
      merged = true;
    }
    __builtin_amdgcn_wave_barrier();
    cnt = 0;
  }
};

template <int ET> constexpr int batch_loads() { return ET == 2 ? 4 : 2; }  // 16 values a lane

template <int ET>
__global__ __launch_bounds__(SC_THREADS, ET == 2 ? 6 : 8) void score_kernel(ScoreArgs a) {
  constexpr int ES = Elem<ET>::SIZE, EPV = 16 / ES;
  constexpr int U = batch_loads<ET>(), N = U * EPV;
  __shared__ uint64_t found[SC_WAVES][FOUND];
  __shared__ __align__(16) float tops[SCORE_BATCHES * SC_WAVES * 4];  // of 16 lanes each
  __shared__ Sums sums[SC_WAVES];
  __shared__ int counts[SC_WAVES];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x / a.nsplit;
  const int split = blockIdx.x % a.nsplit;
  const char* row = (const char*)a.logits + t * a.stride * ES;
  // Rows start at any element: up to EPV - 1 values before the first whole
  // 16 bytes and after the last are taken one by one.
  int head = (int)((16 - ((uintptr_t)row & 15)) & 15) / ES;
  if (head > a.V) head = (int)a.V;
  const int nvec = ((int)a.V - head) / EPV;  // V is at most 2^30
  const int rest = (int)a.V - head - nvec * EPV;
  const int v0 = split * (int)a.slice, v1 = min(nvec, v0 + (int)a.slice);
  const char* body = row + head * ES;
  const int k = a.k;
  const float c = a.c;
  // batches of this wave: every fourth of the slice's
  auto start = [&](int b) { return v0 + (b * SC_WAVES + wave) * (64 * U); };
  const int batches = (v1 - v0 + 64 * U - 1) / (64 * U) - wave;
  const int nb = v1 > v0 && batches > 0 ? (int)((batches + SC_WAVES - 1) / SC_WAVES) : 0;
  const int nb_most = v1 > v0 ? (int)((batches + wave + SC_WAVES - 1) / SC_WAVES) : 0;  // wave 0's

  Sums r = {LOWEST, 0.f, 0.f};
  auto add = [&](float d) {
    const float e = __builtin_amdgcn_exp2f(d);
    r.s += e;
    r.w += e * fmaxf(d, -1e4f);  // 0 * -inf is no term; a NaN stays in e
  };
  auto grow = [&](float mx) {
    const float m = fmaxf(r.m, mx);
    const float d = shift(r.m, m, c);
    const float f = __builtin_amdgcn_exp2f(d);
    r.w = f * (r.w + d * r.s);
    r.s *= f;
    r.m = m;
  };
  i32x4 raw[U];
  auto load = [&](int g) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      raw[u] = *(const i32x4*)(body + (int64_t)min(g + u * 64 + lane, v1 - 1) * 16);
  };
  // The loaded batch's values; places past the slice hold -inf.
  auto unpack = [&](int g, float* x) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (ET == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[u * 4 + i] = __int_as_float(raw[u][i]);
      } else {
        unpack8<ET == 1>(raw[u], x + u * 8);
      }
    }
    if (g + 64 * U > v1) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (g + u * 64 + lane >= v1)
#pragma unroll
          for (int i = 0; i < EPV; ++i) x[u * EPV + i] = -__builtin_inff();
    }
  };

  float lane_max = -__builtin_inff();
  if (nb > 0) load(start(0));
  for (int b = 0; b < nb; ++b) {
    float x[N];
    unpack(start(b), x);
    if (b + 1 < nb) load(start(b + 1));
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mx = fmaxf(mx, x[i]);
    grow(mx);
    const float mc = frame(r.m, c);
    if (__any(!in_range(mc))) {
#pragma unroll
      for (int i = 0; i < N; ++i) add(rel(x[i], r.m, c));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) add(fmaf(x[i], c, -mc));
    }
    if (k > 0) {
      lane_max = fmaxf(lane_max, mx);
      const float top = max_lanes<8>(mx);
      if ((lane & 15) == 0) tops[(b * SC_WAVES + wave) * 4 + (lane >> 4)] = top;
    }
  }
  const bool ends = split == 0 && wave == 0 && head + rest > 0;
  const bool end_ok = lane < head + rest;
  const int end_at = lane < head ? lane : (int)a.V - rest + (lane - head);
  float end_x = -__builtin_inff();
  if (ends) {
    if (end_ok) end_x = load_one<ET>(row, end_at);
    grow(end_x);
    add(rel(end_x, r.m, c));
  }

  Best best;
  best.buf = found[wave];
  if (k > 0) {
    // The lower bound: a lane takes every 64th maximum of 16 lanes, in batch
    // order over all waves; of few batches, its own maximum, and the best of
    // the waves' bounds counts.
    for (int b = nb; b < nb_most; ++b)
      if (lane < 4) tops[(b * SC_WAVES + wave) * 4 + lane] = -__builtin_inff();
    float tau_x = -__builtin_inff();
    const bool few = nb_most < 4;
    if (few) {
      tau_x = at_least(lane_max, k, lane);
      if (lane == 0) sums[wave].m = tau_x;
    }
    __syncthreads();
    if (few) {
#pragma unroll
      for (int w = 0; w < SC_WAVES; ++w) tau_x = fmaxf(tau_x, sums[w].m);
      __syncthreads();
    } else {
      float mx = -__builtin_inff();
      for (int e = lane; e < nb_most * SC_WAVES * 4; e += 64) mx = fmaxf(mx, tops[e]);
      tau_x = __shfl(sort64(mx, lane), k - 1);
    }
    uint64_t tau = make_key(tau_x, 0) & 0xFFFFFFFF00000000ull;  // below every key of its value
    auto merge = [&]() {
      best.merge(lane);
      const uint64_t kth = shfl64(best.list, k - 1);
      if (kth > tau) {
        tau = kth;
        tau_x = key_value(kth);
      }
    };
    // Note one value per lane; there is room.
    auto note = [&](float x, bool valid, uint32_t idx) {
      const bool in = valid && x >= tau_x;
      if (!__any(in)) return;
      const uint64_t key = make_key(x, idx);
      best.put(key, in && key > tau, lane);
    };
    float top = -__builtin_inff();  // of batch `lane`
    if (lane < nb) {
      const f32x4 v = *(const f32x4*)(tops + (lane * SC_WAVES + wave) * 4);
      top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
    }
    uint64_t hit = __ballot(lane < nb && top >= tau_x);
    while (hit) {
      const int b = __builtin_ctzll(hit);
      hit &= hit - 1;
      const int g = start(b);
      if (nb > 1) load(g);  // (a single batch is still there)
      float x[N];
      unpack(g, x);
      float mx = x[0];
#pragma unroll
      for (int i = 1; i < N; ++i) mx = fmaxf(mx, x[i]);
      const uint32_t base = (uint32_t)(head + g * EPV);
      const bool tight = best.cnt + __popcll(__ballot(mx >= tau_x)) * N > FOUND;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (tight && best.cnt > FOUND - 64) merge();
        note(x[i], g + i / EPV * 64 + lane < v1, base + (i / EPV * 64 + lane) * EPV + i % EPV);
      }
      if (best.cnt > FOUND - 64) merge();
    }
    if (ends) note(end_x, end_ok, (uint32_t)end_at);
    if (best.merged) {  // more than fits: the k first stand for all
      merge();
      best.put(best.list, lane < k, lane);
    }
    if (lane == 0) counts[wave] = best.cnt;
  }
  r = join_lanes(r, c);
  if (lane == 0) sums[wave] = r;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < SC_WAVES; ++w) r = join(r, sums[w], c);
    if (k > 0) {
      // the first wave's keys are in place; the others' follow them
      best.merged = false;
      best.list = 0;
#pragma unroll
      for (int w = 1; w < SC_WAVES; ++w)
        for (int at = 0; at < counts[w]; at += 64) {
          if (best.cnt > FOUND - 64) best.merge(lane);
          best.put(found[w][min(at + lane, FOUND - 1)], at + lane < counts[w], lane);
        }
      best.merge(lane);
    }
    if (a.nsplit == 1) write_row<ET>(a, t, r, best.list, lane);
  }
  if (a.nsplit == 1) return;

  // Arrival: partials are written, and read by the last workgroup, with
  // agent-scope atomics, which are coherent across the XCDs' L2s by
  // themselves; the wave waits for its stores to be acknowledged before it
  // counts itself.  (A release / acquire of that scope would write back and
  // invalidate the whole L2 in every workgroup.)
  if (wave != 0) return;
  const int64_t p0 = t * a.nsplit;
  if (lane == 0) {
    float* const p = a.part_sums + (p0 + split) * 3;
    st_agent(p, r.m);
    st_agent(p + 1, r.s);
    st_agent(p + 2, r.w);
  }
  if (lane < k) st_agent(a.part_keys + (p0 + split) * k + lane, best.list);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  int seen = 0;
  if (lane == 0)
    seen = __hip_atomic_fetch_add(a.counters + t * SCORE_COUNTER_STEP, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (__builtin_amdgcn_readfirstlane(seen) != a.nsplit - 1) return;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  // The k-th key of any slice is a lower bound of the row's.
  uint64_t bound = 0;
  r = Sums{LOWEST, 0.f, 0.f};
  for (int i = lane; i < a.nsplit; i += 64) {
    const float* const p = a.part_sums + (p0 + i) * 3;
    r = join(r, Sums{ld_agent(p), ld_agent(p + 1), ld_agent(p + 2)}, c);
    if (k > 0) {
      const uint64_t key = ld_agent(a.part_keys + (p0 + i) * k + k - 1);
      bound = key > bound ? key : bound;
    }
  }
  r = join_lanes(r, c);
  best = Best{found[0]};
  if (k > 0) {
    bound = max_lanes<32>(bound);
    const int n = a.nsplit * k;
    for (int at = 0; at < n; at += 64) {
      if (best.cnt > FOUND - 64) best.merge(lane);
      const uint64_t key = at + lane < n ? ld_agent(a.part_keys + p0 * k + at + lane) : 0;
      best.put(key, key >= bound && key != 0, lane);
    }
    best.merge(lane);
  }
  write_row<ET>(a, t, r, best.list, lane);
  if (lane == 0) st_agent(a.counters + t * SCORE_COUNTER_STEP, 0);  // kept at zero between calls
}

template <int ET> hipError_t launch_score_t(const ScoreArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((score_kernel<ET>), dim3((unsigned)(a.T * a.nsplit)), dim3(SC_THREADS), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Slices of a row.  Few rows are cut until there is a workgroup for each CU,
// with one batch of every wave in each slice at least (48 rows of 128259 in
// 32 bits, top 20: 25 us with 256 or 512 workgroups, 27 with 1024, 34 with
// 1536, whose arrivals take longer than what they save).  Of many, 2048
// workgroups run at a time: they are cut as often as fills whole rounds, with
// four batches in each slice.
void score_plan(int64_t T, int64_t V, int elem, int* nsplit, int64_t* slice) {
  const int64_t nvec = V / (elem == 2 ? 4 : 8) + 1;
  const int64_t batch = SC_THREADS * (elem == 2 ? 4 : 2);  // 16-byte chunks
  const int64_t slots = 2048;
  int64_t ns = 1;
  if (T * 2 <= slots) {
    ns = std::min<int64_t>((256 + T - 1) / T, (nvec + batch - 1) / batch);
  } else {
    double best = 0;
    for (int64_t n = 1; n <= std::min<int64_t>(8, nvec / (4 * batch)); ++n) {
      const int64_t rounds = (T * n + slots - 1) / slots;
      const double use = (double)(T * n) / (double)(rounds * slots) - 0.03 * (double)n;
      if (use > best) { best = use; ns = n; }
    }
  }
  const int64_t most = batch * SCORE_BATCHES;  // what the kernel keeps maxima of
  ns = std::max<int64_t>(ns, (nvec + most - 1) / most);
  *slice = ((nvec + ns - 1) / ns + batch - 1) / batch * batch;
  *nsplit = (int)((nvec + *slice - 1) / *slice);
}

hipError_t launch_score(const ScoreArgs& a, int elem, hipStream_t s) {
  if (elem == 0) return launch_score_t<0>(a, s);
  if (elem == 1) return launch_score_t<1>(a, s);
  return launch_score_t<2>(a, s);
}

}  // namespace lg
