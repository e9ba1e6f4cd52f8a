// kernels_norm.hip -- the root-mean-square norm of a decoder's stream with the
// addition of the residual before it and the 8-bit codes of the next layer
// behind it, in one pass:
//
//   s = x + residual,   y = s / sqrt(mean(s^2) + eps) * w,
//   codes = y / scale rounded,   scale = max|y| / QMAX of the row or 1x128 block
//
// with s, y and the scales in 32 bits, s and y rounded once where they are
// stored; the codes come from the unrounded y.
//
// Memory bound: 2 bytes in for each of x and the residual, 2 out for the sum
// and for y, 1 for the codes.  A row is one workgroup, which holds it in
// registers (up to four 16-byte chunks a lane), so everything is read once.
// For positive r = 1 / sqrt(..), max|s w| r is max|y|: the sum of squares and the
// maximum meet in one reduction and one barrier.  The maximum of a block is
// that of 16 neighbouring lanes.
//   8191 rows of 4096 values with both outputs and codes take 48 us in the kernel
// (6.3 TB/s: part of it stays in the last-level cache; a large copy reaches 5.1), one
// row 2.9 us, 24 rows of 8192 with block codes 4.5, and the calls 58, 7 and 8.
#include "launch.hpp"

namespace lg {
namespace {

enum NormKind : int { NK_NONE = -1, NK_FP8 = DQ_FP8_TOKEN, NK_INT8 = DQ_INT8_TOKEN, NK_BLOCK = DQ_FP8_BLOCK };

template <int CTRL> __device__ inline float dpp(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(x), CTRL, 0xF, 0xF, true));
}
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E;            // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140; // of 8 and of 16 lanes

// Over the 16 lanes of a DPP row, in every lane.
template <typename F> __device__ inline float row16(float x, F f) {
  x = f(x, dpp<DPP_XOR1>(x));
  x = f(x, dpp<DPP_XOR2>(x));
  x = f(x, dpp<DPP_HALF_MIRROR>(x));
  return f(x, dpp<DPP_MIRROR>(x));
}
// Over the wave, in every lane.
template <typename F> __device__ inline float wave64(float x, F f) {
  x = row16(x, f);
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

constexpr int MAX_WAVES = 16;

// C: 16-byte chunks per lane.
template <bool F16, int KIND, int C>
__global__ __launch_bounds__(64 * MAX_WAVES) void norm_kernel(NormArgs a) {
  __shared__ float2 part[2][MAX_WAVES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int nch = a.N >> 3;
  int turn = 0;

  // A sum and a maximum over the workgroup.
  auto over_row = [&](float sum, float most) {
    sum = wave64(sum, Add{});
    most = wave64(most, Max{});
    if (waves > 1) {
      if (lane == 0) part[turn][wave] = make_float2(sum, most);
      __syncthreads();
      sum = 0.f;
      most = 0.f;
      for (int w = 0; w < waves; ++w) {
        const float2 p = part[turn][w];
        sum += p.x;
        most = fmaxf(most, p.y);
      }
      turn ^= 1;  // the next use does not wait for the readers of this one
    }
    return make_float2(sum, most);
  };

  i32x4 wr[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = min(i * (int)blockDim.x + tid, nch - 1);
    wr[i] = *(const i32x4*)(a.w + (int64_t)c * 8);
  }
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    float s[C][8];
    {
      i32x4 xr[C], rr[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int64_t c = min(i * (int)blockDim.x + tid, nch - 1) * 8;
        xr[i] = *(const i32x4*)(a.x + row * a.x_s + c);
        if (a.res) rr[i] = *(const i32x4*)(a.res + row * a.res_s + c);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const bool in = i * (int)blockDim.x + tid < nch;
        unpack8<F16>(in ? xr[i] : i32x4{0, 0, 0, 0}, s[i]);
        if (a.res) {
          float r[8];
          unpack8<F16>(in ? rr[i] : i32x4{0, 0, 0, 0}, r);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[i][e] += r[e];
        }
        if (a.res_out && in)
          store_h<8, F16>(a.res_out + row * a.res_out_s + (int64_t)(i * (int)blockDim.x + tid) * 8, s[i]);
      }
    }
    float w[C][8];
    float sum = 0.f, most = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      unpack8<F16>(wr[i], w[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = fmaf(s[i][e], s[i][e], sum);
        if (KIND == NK_FP8 || KIND == NK_INT8) most = fmaxf(most, fabsf(s[i][e] * w[i][e]));
      }
    }
    float2 got = over_row(sum, most);
    const float n_inv = 1.f / (float)a.N;
    float mean = fmaf(got.x, n_inv, a.eps);
    float r = rsqrtf(mean);
    float amax = got.y * r;
    // Squares or products that leave binary32's normal range (values beyond 2^60
    // or, with next to no eps, below 2^-48; weights to match): the row times a power
    // of two that brings the larger of it and the root of eps near one, and the
    // maximum of the finished values.
    if (!(mean > 0x1p-96f && mean < 0x1p120f && (got.y == 0.f || (got.y > 0x1p-100f && got.y < 0x1p100f)))) {
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) big = fmaxf(big, amax8(s[i]));
      big = fmaxf(over_row(0.f, big).y, sqrtf(a.eps));
      const int up = big > 0.f && big < __builtin_inff() ? -__builtin_amdgcn_frexp_expf(big) : 0;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[i][e] = ldexpf(s[i][e], up);
          sum = fmaf(s[i][e], s[i][e], sum);
        }
      mean = fmaf(over_row(sum, 0.f).x, n_inv, ldexpf(ldexpf(a.eps, up), up));
      r = rsqrtf(mean);
      most = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(s[i][e] * r * w[i][e]));
      amax = over_row(0.f, most).y;
    }

    DivBy d;
    if (KIND == NK_FP8 || KIND == NK_INT8) {
      const float scale = group_scale(amax, KIND == NK_INT8 ? 127.f : 448.f);
      d = make_div(scale, amax);
      if (tid == 0) a.scales[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = i * (int)blockDim.x + tid;
      const bool in = c < nch;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = s[i][e] * r * w[i][e];
      if (a.out && in) store_h<8, F16>(a.out + row * a.out_s + (int64_t)c * 8, y);
      if constexpr (KIND == NK_FP8 || KIND == NK_INT8) {
        if (in) *(i32x2*)(a.codes + row * a.N + (int64_t)c * 8) = quant8<KIND == NK_INT8>(y, d);
      } else if constexpr (KIND == NK_BLOCK) {
        // (chunks past the row come in whole blocks)
        const float bm = row16(amax8(y), Max{});
        const float scale = group_scale(bm, 448.f);
        if (in) {
          *(i32x2*)(a.codes + row * a.N + (int64_t)c * 8) = quant8<false>(y, make_div(scale, bm));
          if ((c & 15) == 0) a.scales[row * (a.N >> 7) + (c >> 4)] = scale;
        }
      }
    }
  }
}

template <bool F16, int KIND> hipError_t launch_kind(const NormArgs& a, hipStream_t s) {
  const int nch = a.N >> 3;
  // Two chunks per lane, up to 16 waves.  (One, two and four are close: 8191 rows of
  // 4096 48, 50 and 50 us, 4000 of 8192 38, 37 and 40, 2000 of 16384 41, 42 and 38.)
  int waves = 1;
  while (waves < MAX_WAVES && waves * 128 < nch) waves *= 2;
  const int per = (nch + waves * 64 - 1) / (waves * 64);
  const dim3 grid((unsigned)std::min<int64_t>(a.T, (int64_t)1 << 20)), block(waves * 64);
  if (per <= 1) hipLaunchKernelGGL((norm_kernel<F16, KIND, 1>), grid, block, 0, s, a);
  else if (per <= 2) hipLaunchKernelGGL((norm_kernel<F16, KIND, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_kernel<F16, KIND, 4>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <bool F16> hipError_t launch_type(const NormArgs& a, int kind, hipStream_t s) {
  switch (kind) {
    case NK_FP8: return launch_kind<F16, NK_FP8>(a, s);
    case NK_INT8: return launch_kind<F16, NK_INT8>(a, s);
    case NK_BLOCK: return launch_kind<F16, NK_BLOCK>(a, s);
    default: return launch_kind<F16, NK_NONE>(a, s);
  }
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int kind, bool f16, hipStream_t s) {
  return f16 ? launch_type<true>(a, kind, s) : launch_type<false>(a, kind, s);
}

}  // namespace lg
