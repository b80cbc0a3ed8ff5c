// sq_qknorm.cuh -- norm of queries and keys for each head, rotated by
// position, in one pass (sq_qk_norm).
//
// A thread holds 8 consecutive channels of one head (one 16-byte load of a
// 16-bit type, two of fp32), so d / 8 lanes hold a head: the sum of squares
// is log2(d / 8) shuffles, and the rotation's partner channels are in the
// same thread (adjacent pairs) or a fixed number of lanes away (halves).
// Every element is read once and written once: 16384 rows x 32 heads of 128
// bf16, half rotated, take 71 us, 0.58 of the measured copy rate. Bound by
// issue and latency: 186 warp instructions per 256 elements, 0.69 issued a
// cycle and scheduler, most stalls on shuffles and shared memory. The four ways
// to turn are branches of one kernel, and in the 64 registers that four CTAs per
// SM leave it spills in every instance: 20 to 32 bytes stored and 40 to 52 loaded
// a thread with 16-bit inputs, 64 to 80 and 88 to 108 with fp32. The angles of a
// row are shared by all its heads: a CTA takes groups of `rows_per_cta` rows
// and forms their rot_dim / 2 sines and cosines once into shared memory, a
// group ahead (position times frequency in turns, in fp64, reduced to half a
// turn before the fp32 sine, so a position of 10^6 loses nothing); a thread
// has the next two rows of its head on their way while it works on one.
#pragma once

#include <cuda_bf16.h>

#include "sq_kernels.cuh"

namespace sqr {

constexpr int kNormThreads = 256;
constexpr int kNormMaxRows = 8;  // rows per group at most

struct NormArgs {
  const void* x[2];          // q, k
  void* y[2];
  const float* w[2];         // [d] or null
  int64_t stride[2];         // elements
  int32_t heads[2];
  float scale[2];
  const int32_t* positions;
  const int32_t* n_rows;     // or null
  int32_t rows, rows_per_cta, head_bits, rot, inter, rms;
  float eps;
  double turns[64];          // base^(-2 i / rot) / (2 pi)
};

// 8 channels of a type, as loaded and as fp32.
template <typename T>
struct Pack8;
template <>
struct Pack8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
  }
  static __device__ __forceinline__ void store(float* p, const float2 (&f)[4]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
};
template <>
struct Pack8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].x, f[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Pack8<__half> {
  uint4 v;
  __device__ __forceinline__ void load(const __half* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    }
  }
  static __device__ __forceinline__ void store(__half* p, const float2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[i].x, f[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// How the lane's channels are turned, the same for every row.
enum { TURN_NOT, TURN_PAIRS, TURN_HALVES, TURN_AGAIN };

template <int D, typename TI, typename TO>
__global__ void __launch_bounds__(kNormThreads, 4) k_qk_norm(const __grid_constant__ NormArgs a) {
  constexpr int LPH = D / 8;                  // lanes per head
  constexpr int AT = kNormThreads / LPH;      // heads the CTA takes at once
  // cosine and sine, cosine and -sine, of row and pair: this group's and the next's
  __shared__ __align__(16) float2 cs[2][2][kNormMaxRows][D / 2];
  const int rows = a.n_rows ? min(max(*a.n_rows, 0), a.rows) : a.rows;
  const int half = a.rot >> 1;
  const int c0 = (threadIdx.x & (LPH - 1)) * 8;
  const int heads = a.heads[0] + a.heads[1];
  // the CTA's AT slots take 2^head_bits heads of AT / 2^head_bits rows at once
  const int slot = threadIdx.x / LPH, r1 = slot >> a.head_bits, rstep = AT >> a.head_bits;
  // Pairs (2i, 2i + 1) are in one lane. Channel c < half pairs with c + half, in
  // lane (c + half) / 8 if half is a multiple of 8 (the lane takes that lane's
  // channels, and the table with its sign of the sine); any other half reads
  // its partners' inputs again.
  const int how = half == 0 ? TURN_NOT : a.inter ? TURN_PAIRS : (half & 7) == 0 ? TURN_HALVES : TURN_AGAIN;
  const bool lo = c0 < half, in = c0 < a.rot;
  const int from = (c0 >> 3) + (how != TURN_HALVES || !in ? 0 : lo ? half >> 3 : -(half >> 3));
  // Where a row's table holds pair p: a lane's pairs lie apart and its
  // neighbours' beside them, so that a warp's read meets no bank twice.
  auto place = [&](int p) {
    return how == TURN_HALVES ? (((p >> 1) & 3) * (D / 16) + (p >> 3)) * 2 + (p & 1)
           : how == TURN_PAIRS ? (p & 3) * LPH + (p >> 2) : p;
  };
  const int stride = gridDim.x * a.rows_per_cta;
  auto angles = [&](int buf, int r0) {
    const int n = min(a.rows_per_cta, rows - r0) * half;
    for (int i = threadIdx.x; i < n; i += kNormThreads) {
      const int rr = i / half, p = i - rr * half;
      const double t = (double)a.positions[r0 + rr] * a.turns[p];
      float sn, c;
      sincospif(2.0f * (float)(t - rint(t)), &sn, &c);
      const int at = place(p);
      cs[buf][0][rr][at] = make_float2(c, sn);
      cs[buf][1][rr][at] = make_float2(c, -sn);
    }
  };
  int r0 = blockIdx.x * a.rows_per_cta;
  if (r0 >= rows) return;
  if (half) {
    angles(0, r0);
    __syncthreads();
  }
  const float2* table = &cs[0][lo][0][how == TURN_PAIRS ? c0 >> 3 : how == TURN_HALVES && in ? (lo ? c0 : c0 - half) >> 2 : 0];
  const float part = a.rms ? 1.0f / D : 1.0f;
#pragma unroll 1
  for (int buf = 0; r0 < rows; r0 += stride, buf ^= 1) {
    const int nr = min(a.rows_per_cta, rows - r0);
    if (half && r0 + stride < rows) angles(buf ^ 1, r0 + stride);
#pragma unroll 1
    for (int base = 0; base < heads; base += 1 << a.head_bits) {
      int h = base + (slot & ((1 << a.head_bits) - 1));
      const bool mine = h < heads;  // every lane stays for the shuffles
      h = min(h, heads - 1);
      const int which = h >= a.heads[0];
      h -= which ? a.heads[0] : 0;
      const int64_t xs = a.stride[which], ys = (int64_t)a.heads[which] * D;
      const TI* x = static_cast<const TI*>(a.x[which]) + (r0 + min(r1, nr - 1)) * xs + h * D + c0;
      TO* y = static_cast<TO*>(a.y[which]) + (r0 + r1) * ys + h * D + c0;
      Pack8<TI> now, then;
      now.load(x);
      then = now;
      if (r1 + rstep < nr) then.load(x + rstep * xs);
      const float* w = a.w[which];
      const float scale = a.scale[which];
      float2 wr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        wr[e] = w ? make_float2(scale * w[c0 + 2 * e], scale * w[c0 + 2 * e + 1]) : make_float2(scale, scale);
      const float2* t = table + (buf * 2 * kNormMaxRows + r1) * (D / 2);
#pragma unroll 1
      for (int r = r1; r - r1 < nr; r += rstep) {
        float2 f[4];
        now.get(f);
        now = then;
        if (r + 2 * rstep < nr) then.load(x + 2 * rstep * xs);
        float2 s2 = __fmul2_rn(f[0], f[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = __ffma2_rn(f[e], f[e], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        const float inv = rsqrtf(fmaf(ss, part, a.eps));
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __fmul2_rn(f[e], __fmul2_rn(make_float2(inv, inv), wr[e]));
        if (how == TURN_HALVES) {
          float2 p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[e] = make_float2(__shfl_sync(0xffffffffu, f[e].x, from, LPH), __shfl_sync(0xffffffffu, f[e].y, from, LPH));
          if (in && r < nr) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 c = reinterpret_cast<const float4*>(t)[e * (D / 16)];
              f[e] = make_float2(fmaf(f[e].x, c.x, p[e].x * c.y), fmaf(f[e].y, c.z, p[e].y * c.w));
            }
          }
        } else if (how == TURN_PAIRS) {
          if (in && r < nr) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (c0 + 2 * e < a.rot) {
                const float2 c = t[e * LPH];  // of table 0 or 1: the sign of the sine is lo's
                const float sn = lo ? -c.y : c.y;
                f[e] = make_float2(fmaf(f[e].x, c.x, -(f[e].y * sn)), fmaf(f[e].y, c.x, f[e].x * sn));
              }
            }
          }
        } else if (how == TURN_AGAIN && r < nr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = c0 + e;
            if (c < a.rot) {
              const int pc = c < half ? c + half : c - half;
              const float p = (float)x[pc - c0] * (inv * (w ? scale * w[pc] : scale));
              const float2 q = cs[buf][c < half][r][min(c, pc)];
              float& v = e & 1 ? f[e >> 1].y : f[e >> 1].x;
              v = fmaf(v, q.x, p * q.y);
            }
          }
        }
        if (mine && r < nr) Pack8<TO>::store(y, f);
        x += rstep * xs;
        y += rstep * ys;
        t += rstep * (D / 2);
      }
    }
    if (half) __syncthreads();  // the next group's angles; this one's have been used
  }
}

}  // namespace sqr
