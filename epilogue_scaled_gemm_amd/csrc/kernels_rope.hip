// kernels_rope.hip -- what happens to the heads of a QKV product before
// attention: per-head norms of queries and keys, the position rotation, and
// the store of keys and values into a paged cache, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w                       (where w is given)
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)            for each pair
//
// The pairs are (i, i + rot/2) or (2i, 2i + 1) of a head's first `rot`
// values; c and s come from a table row [cos | sin] of the token's
// position, so far positions cost no precision here.  Everything is computed
// in 32 bits and rounded once, to the output's or the cache's type.
//
// Memory bound: 2 bytes in and out per value.  A head is D / 8 lanes of 16
// bytes, so its norm is a reduction by lane shuffles and the partner of a
// half-split pair is another lane of the same group; nothing goes through
// LDS.  8191 tokens of 40 heads of 128 values (bf16) take 44 us (3.9 TB/s; a
// large copy reaches 4.8), 4099 tokens of 32 query and 8 key heads with their
// values stored to pages 26 us (3.9 TB/s).  A decode step is one chain of
// latencies: 4 us in the kernel, 8 to 11 with the call around it.
#include "launch.hpp"

namespace lg {
namespace {

constexpr int RP_THREADS = 256;
constexpr int RP_WAVES = 4;

// LPH lanes hold one head (the power of two at or above D / 8), a wave 64 / LPH
// heads of one kind, so that everything that depends on the kind is scalar;
// wave jobs of a token are its queries, keys and values in turn.  NPT jobs
// per wave: their loads all go out first, and the token's cosines and sines
// are read once for them (8191 tokens: 59 us with one job per wave of mixed
// kinds, 43 with three of one kind each).
template <bool F16, int LPH, int NPT>
__global__ __launch_bounds__(RP_THREADS) void heads_kernel(HeadArgs a) {
  constexpr int HPW = 64 / LPH;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane % LPH, grp = lane / LPH;  // 16-byte chunk, head of the wave
  const int64_t t = blockIdx.x;
  const int nch = a.D >> 3;
  const int jq = (a.Hq + HPW - 1) / HPW, jk = (a.Hk + HPW - 1) / HPW, jv = (a.Hv + HPW - 1) / HPW;
  const int job0 = blockIdx.y * RP_WAVES + wave, step = gridDim.y * RP_WAVES;

  i32x4 raw[NPT];
  int kind[NPT], head[NPT];  // 0 query, 1 key, 2 value, 3 none
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int job = job0 + i * step;
    kind[i] = job < jq ? 0 : job < jq + jk ? 1 : job < jq + jk + jv ? 2 : 3;
    const int count = kind[i] == 0 ? a.Hq : a.Hk;
    head[i] = (kind[i] == 0 ? job : kind[i] == 1 ? job - jq : job - jq - jk) * HPW + grp;
    if (head[i] >= count || c >= nch) head[i] = -1;
    raw[i] = i32x4{0, 0, 0, 0};
    if (kind[i] < 3 && head[i] >= 0) {
      const HeadView& v = kind[i] == 0 ? a.q : kind[i] == 1 ? a.k : a.v;
      raw[i] = *(const i32x4*)((const uint16_t*)v.p + t * v.ts + head[i] * v.hs + c * 8);
    }
  }

  // This lane's cosines and sines, the same for every head of the token.
  float cs[8], sn[8];
  const bool turns = a.table && c < (a.rot >> 3);
  if (a.table && job0 < jq + jk) {
    const int pos = min(max(a.positions[t], 0), a.max_pos - 1);
    const float* row = a.table + (int64_t)pos * a.rot;
    const int hr = a.rot >> 1;
    if (turns) {
      if (a.interleaved) {
        const f32x4 cc = *(const f32x4*)(row + c * 4), ss = *(const f32x4*)(row + hr + c * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cs[2 * i] = cs[2 * i + 1] = cc[i];
          sn[2 * i] = sn[2 * i + 1] = ss[i];
        }
      } else {
        const int at = (c < (a.rot >> 4) ? c : c - (a.rot >> 4)) * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 cc = *(const f32x4*)(row + at + 4 * h);
          const f32x4 ss = *(const f32x4*)(row + hr + at + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            cs[4 * h + i] = cc[i];
            sn[4 * h + i] = ss[i];
          }
        }
      }
    }
  }
  int64_t page = 0, in = 0;
  bool keep = false;
  if (a.slots) {
    const int slot = a.slots[t];
    keep = slot >= 0 && slot < a.capacity;
    page = slot >> a.page_log;
    in = slot & ((1 << a.page_log) - 1);
  }

#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    if (kind[i] == 3) break;
    float y[8];
    unpack8<F16>(raw[i], y);
    if (kind[i] < 2) {
      const uint16_t* w = kind[i] == 0 ? a.q_weight : a.k_weight;
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += y[e] * y[e];
#pragma unroll
        for (int off = LPH / 2; off > 0; off >>= 1) ss += __shfl_xor(ss, off, LPH);
        const float mean = ss / (float)a.D + a.eps;
        float r = __builtin_amdgcn_rsqf(mean);
        // Squares that leave binary32's normal range (values beyond 2^60 or, with
        // next to no eps, below 2^-48): the head times a power of two that
        // brings the larger of it and the root of eps near one.
        const bool off = !(mean > 0x1p-96f && mean < 0x1p120f);
        if (__any(off)) {
          float big = sqrtf(a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(y[e]));
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, LPH));
          const bool scaled = off && big > 0.f && big < __builtin_inff();
          const int up = scaled ? -__builtin_amdgcn_frexp_expf(big) : 0;
          ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = ldexpf(y[e], up);
            ss += y[e] * y[e];
          }
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor(ss, o, LPH);
          if (scaled) r = __builtin_amdgcn_rsqf(ss / (float)a.D + ldexpf(a.eps, 2 * up));
        }
        float wf[8];
        i32x4 wr = {0, 0, 0, 0};
        if (c < nch) wr = *(const i32x4*)(w + c * 8);
        unpack8<F16>(wr, wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * r * wf[e];
      }
      if (a.table) {
        if (a.interleaved) {
          if (turns) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float p = y[e], q = y[e + 1];
              y[e] = p * cs[e] - q * sn[e];
              y[e + 1] = q * cs[e] + p * sn[e];
            }
          }
        } else {
          const int hc = a.rot >> 4;  // chunks of half the rotated part
          const bool lo = c < hc;
          const int other = !turns ? c : lo ? c + hc : c - hc;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float z = __shfl(y[e], other, LPH);
            if (turns) y[e] = lo ? y[e] * cs[e] - z * sn[e] : y[e] * cs[e] + z * sn[e];
          }
        }
      }
    }
    if (head[i] < 0) continue;
    const bool cached = kind[i] == 2 || (kind[i] == 1 && a.slots);
    if (cached && !keep) continue;
    const HeadView& d = !cached ? (kind[i] == 0 ? a.q_out : a.k_out) : kind[i] == 1 ? a.kc : a.vc;
    const int64_t at = (cached ? page * d.ps + in * d.ts : t * d.ts) + head[i] * d.hs + c * 8;
    if (!cached || !a.cache8) {
      i32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack2<F16>(y[2 * e], y[2 * e + 1]);
      *(i32x4*)((uint16_t*)d.p + at) = w;
    } else {
      const float* sp = kind[i] == 1 ? a.k_scale : a.v_scale;
      const float s = sp ? sp[head[i]] : 1.f;
      // Saturated to the type's range; a NaN passes the comparisons and
      // stays one.
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = y[e] / s;
        y[e] = z > 448.f ? 448.f : z < -448.f ? -448.f : z;
      }
      i32x2 w;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int word = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * e], y[4 * e + 1], 0, false);
        w[e] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * e + 2], y[4 * e + 3], word, true);
      }
      *(i32x2*)((uint8_t*)d.p + at) = w;
    }
  }
}

template <bool F16, int LPH> hipError_t launch_heads_l(const HeadArgs& a, int64_t T, hipStream_t s) {
  constexpr int HPW = 64 / LPH;
  const int jobs = (a.Hq + HPW - 1) / HPW + (a.Hk + HPW - 1) / HPW + (a.Hv + HPW - 1) / HPW;
  const int blocks = (jobs + RP_WAVES - 1) / RP_WAVES;  // of one job per wave
  // Few tokens: one job per wave, for the shortest chain.  Many: three.
  if (T * blocks <= 2048 || blocks < 2) {
    hipLaunchKernelGGL((heads_kernel<F16, LPH, 1>), dim3((unsigned)T, (unsigned)blocks),
                       dim3(RP_THREADS), 0, s, a);
  } else {
    hipLaunchKernelGGL((heads_kernel<F16, LPH, 3>), dim3((unsigned)T, (unsigned)((blocks + 2) / 3)),
                       dim3(RP_THREADS), 0, s, a);
  }
  return hipGetLastError();
}

template <bool F16> hipError_t launch_heads_t(const HeadArgs& a, int64_t T, hipStream_t s) {
  const int nch = a.D / 8;
  if (nch <= 2) return launch_heads_l<F16, 2>(a, T, s);
  if (nch <= 4) return launch_heads_l<F16, 4>(a, T, s);
  if (nch <= 8) return launch_heads_l<F16, 8>(a, T, s);
  if (nch <= 16) return launch_heads_l<F16, 16>(a, T, s);
  return launch_heads_l<F16, 32>(a, T, s);
}

}  // namespace

hipError_t launch_heads(const HeadArgs& a, int64_t T, bool f16, hipStream_t s) {
  return f16 ? launch_heads_t<true>(a, T, s) : launch_heads_t<false>(a, T, s);
}

}  // namespace lg
