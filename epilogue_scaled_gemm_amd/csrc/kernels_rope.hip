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
// LDS.
#include "launch.hpp"

namespace lg {
namespace {

constexpr int RP_THREADS = 256;

// LPH lanes hold one head (the power of two at or above D / 8).
template <bool F16, int LPH>
__global__ __launch_bounds__(RP_THREADS) void heads_kernel(HeadArgs a) {
  constexpr int GROUPS = RP_THREADS / LPH;
  const int c = threadIdx.x % LPH;  // 16-byte chunk of the head
  const int grp = threadIdx.x / LPH;
  const int64_t t = blockIdx.x;
  const int nch = a.D >> 3;
  const int heads = a.Hq + a.Hk + a.Hv;

  // This lane's cosines and sines, the same for every head of the token.
  float cs[8], sn[8];
  const bool turns = a.table && c < (a.rot >> 3);
  if (a.table) {
    const int64_t pos = min(max(a.positions[t], 0), a.max_pos - 1);
    const float* row = a.table + pos * a.rot;
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

  for (int hh = blockIdx.y * GROUPS + grp; hh < heads; hh += gridDim.y * GROUPS) {
    const int kind = hh < a.Hq ? 0 : hh < a.Hq + a.Hk ? 1 : 2;  // query, key, value
    const int h = kind == 0 ? hh : kind == 1 ? hh - a.Hq : hh - a.Hq - a.Hk;
    const HeadView& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    i32x4 raw = {0, 0, 0, 0};
    if (c < nch) raw = *(const i32x4*)((const uint16_t*)src.p + t * src.ts + h * src.hs + c * 8);
    float y[8];
    unpack8<F16>(raw, y);
    if (kind < 2) {
      const uint16_t* w = kind == 0 ? a.q_weight : a.k_weight;
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
#pragma unroll
        for (int off = LPH / 2; off > 0; off >>= 1) ss += __shfl_xor(ss, off, LPH);
        const float r = 1.f / sqrtf(ss / (float)a.D + a.eps);
        float wf[8];
        i32x4 wr = {0, 0, 0, 0};
        if (c < nch) wr = *(const i32x4*)(w + c * 8);
        unpack8<F16>(wr, wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * r * wf[i];
      }
      if (a.table) {
        if (a.interleaved) {
          if (turns) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float p = y[i], q = y[i + 1];
              y[i] = p * cs[i] - q * sn[i];
              y[i + 1] = q * cs[i] + p * sn[i];
            }
          }
        } else {
          const int hc = a.rot >> 4;  // chunks of half the rotated part
          const bool lo = c < hc;
          const int other = lo ? c + hc : c - hc;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float z = __shfl(y[i], turns ? other : c, LPH);
            if (turns) y[i] = lo ? y[i] * cs[i] - z * sn[i] : y[i] * cs[i] + z * sn[i];
          }
        }
      }
    }
    if (c >= nch) continue;
    const bool cached = kind == 2 || (kind == 1 && a.slots);
    if (!cached || !a.cache8) {
      uint16_t* out;
      if (cached) {
        if (!keep) continue;
        const HeadView& d = kind == 1 ? a.kc : a.vc;
        out = (uint16_t*)d.p + page * d.ps + h * d.hs + in * d.ts + c * 8;
      } else {
        const HeadView& d = kind == 0 ? a.q_out : a.k_out;
        out = (uint16_t*)d.p + t * d.ts + h * d.hs + c * 8;
      }
      i32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (int)((uint32_t)f32_to_h<F16>(y[2 * i]) | ((uint32_t)f32_to_h<F16>(y[2 * i + 1]) << 16));
      *(i32x4*)out = w;
    } else {
      if (!keep) continue;
      const HeadView& d = kind == 1 ? a.kc : a.vc;
      const float* sp = kind == 1 ? a.k_scale : a.v_scale;
      const float s = sp ? sp[h] : 1.f;
      // Saturated to the type's range; a NaN passes the comparisons and
      // stays one.
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z = y[i] / s;
        y[i] = z > 448.f ? 448.f : z < -448.f ? -448.f : z;
      }
      i32x2 w;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int word = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
        w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], word, true);
      }
      *(i32x2*)((uint8_t*)d.p + page * d.ps + h * d.hs + in * d.ts + c * 8) = w;
    }
  }
}

template <bool F16> hipError_t launch_heads_t(const HeadArgs& a, int64_t T, hipStream_t s) {
  const int nch = a.D / 8;
  const int lph = nch <= 2 ? 2 : nch <= 4 ? 4 : nch <= 8 ? 8 : nch <= 16 ? 16 : 32;
  const int groups = RP_THREADS / lph;
  const int heads = a.Hq + a.Hk + a.Hv;
  const unsigned gy = (unsigned)((heads + groups - 1) / groups);
  const dim3 grid((unsigned)T, gy);
  switch (lph) {
    case 2: hipLaunchKernelGGL((heads_kernel<F16, 2>), grid, dim3(RP_THREADS), 0, s, a); break;
    case 4: hipLaunchKernelGGL((heads_kernel<F16, 4>), grid, dim3(RP_THREADS), 0, s, a); break;
    case 8: hipLaunchKernelGGL((heads_kernel<F16, 8>), grid, dim3(RP_THREADS), 0, s, a); break;
    case 16: hipLaunchKernelGGL((heads_kernel<F16, 16>), grid, dim3(RP_THREADS), 0, s, a); break;
    default: hipLaunchKernelGGL((heads_kernel<F16, 32>), grid, dim3(RP_THREADS), 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_heads(const HeadArgs& a, int64_t T, bool f16, hipStream_t s) {
  return f16 ? launch_heads_t<true>(a, T, s) : launch_heads_t<false>(a, T, s);
}

}  // namespace lg
