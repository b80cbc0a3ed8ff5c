// sq_qknorm.cuh -- norm of queries and keys for each head, rotated by
// position, in one pass (sq_qk_norm).
//
// A thread holds 8 consecutive channels of one head (one 16-byte load of a
// 16-bit type, two of fp32), so d / 8 lanes hold a head: the sum of squares
// is log2(d / 8) shuffles, and the rotation's partner channels are in the
// same thread (adjacent pairs) or a fixed number of lanes away (halves).
// Bound by HBM: every element is read once and written once. The angles of a
// row are shared by all its heads: a CTA takes `rows_per_cta` rows, forms
// their rot_dim / 2 sines and cosines once into shared memory (position times
// frequency in turns, in fp64, reduced to half a turn before the fp32 sine,
// so a position of 10^6 loses nothing), then runs over the heads.
#pragma once

#include <cuda_bf16.h>

#include "sq_kernels.cuh"

namespace sqr {

constexpr int kNormThreads = 256;
constexpr int kNormMaxRows = 8;  // rows per CTA at most

struct NormArgs {
  const void* x[2];          // q, k
  void* y[2];
  const float* w[2];         // [d] or null
  int64_t stride[2];         // elements
  int32_t heads[2];
  float scale[2];
  const int32_t* positions;
  const int32_t* n_rows;     // or null
  int32_t rows, rows_per_cta, rot, inter, rms;
  float eps;
  double turns[64];          // base^(-2 i / rot) / (2 pi)
};

// 8 channels as fp32, whatever their type.
template <typename T>
struct Pack8;
template <>
struct Pack8<float> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <>
struct Pack8<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Pack8<__half> {
  static __device__ __forceinline__ void load(const __half* p, float (&f)[8]) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
  static __device__ __forceinline__ void store(__half* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <int D, typename TI, typename TO>
__global__ void __launch_bounds__(kNormThreads) k_qk_norm(const __grid_constant__ NormArgs a) {
  constexpr int LPH = D / 8;                  // lanes per head
  __shared__ float2 cs[kNormMaxRows][D / 2];  // cosine, sine of row and pair
  const int rows = a.n_rows ? min(max(*a.n_rows, 0), a.rows) : a.rows;
  const int r0 = blockIdx.x * a.rows_per_cta;
  const int nr = min(a.rows_per_cta, rows - r0);
  if (nr <= 0) return;
  const int half = a.rot >> 1;
  if (half) {
    for (int x = threadIdx.x; x < nr * half; x += kNormThreads) {
      const int r = x / half, i = x - r * half;
      const double t = (double)a.positions[r0 + r] * a.turns[i];
      float s, c;
      sincospif(2.0f * (float)(t - rint(t)), &s, &c);
      cs[r][i] = make_float2(c, s);
    }
    __syncthreads();
  }
  const int lane = threadIdx.x & (LPH - 1);
  const int c0 = lane * 8;
  const int heads = a.heads[0] + a.heads[1];
  const int n = nr * heads;
  for (int x0 = 0; x0 < n; x0 += kNormThreads / LPH) {  // the whole warp stays for the shuffles
    const int x = x0 + threadIdx.x / LPH;
    const bool live = x < n;
    const int xx = live ? x : n - 1;
    const int r = xx / heads;
    int h = xx - r * heads;
    const int which = h >= a.heads[0];
    if (which) h -= a.heads[0];
    const int64_t row = r0 + r;
    const TI* src = static_cast<const TI*>(a.x[which]) + row * a.stride[which] + h * D;
    float f[8];
    Pack8<TI>::load(src + c0, f);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
    for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if (a.rms) ss *= 1.0f / D;
    const float inv = a.scale[which] / sqrtf(ss + a.eps);
    const float* w = a.w[which];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= w ? inv * w[c0 + e] : inv;
    if (a.inter) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if (c0 + e < a.rot) {
          const float2 t = cs[r][(c0 + e) >> 1];
          const float u = f[e], v = f[e + 1];
          f[e] = fmaf(u, t.x, -(v * t.y));
          f[e + 1] = fmaf(v, t.x, u * t.y);
        }
      }
    } else if (half) {
      // channel c < half pairs with c + half, in lane (c + half) / 8 when half
      // is a multiple of 8; any other half reads its partners' inputs again
      if ((half & 7) == 0) {
        const int dl = half >> 3;
        const bool lo = c0 < half;
        const int from = c0 < a.rot ? (lo ? lane + dl : lane - dl) : lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = __shfl_sync(0xffffffffu, f[e], from, LPH);
          if (c0 < a.rot) {
            const float2 t = cs[r][lo ? c0 + e : c0 + e - half];
            f[e] = lo ? fmaf(f[e], t.x, -(p * t.y)) : fmaf(f[e], t.x, p * t.y);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = c0 + e;
          if (c < a.rot) {
            const bool lo = c < half;
            const int pc = lo ? c + half : c - half;
            const float p = (float)src[pc] * (w ? inv * w[pc] : inv);
            const float2 t = cs[r][lo ? c : pc];
            f[e] = lo ? fmaf(f[e], t.x, -(p * t.y)) : fmaf(f[e], t.x, p * t.y);
          }
        }
      }
    }
    if (live) Pack8<TO>::store(static_cast<TO*>(a.y[which]) + (row * a.heads[which] + h) * D + c0, f);
  }
}

}  // namespace sqr
