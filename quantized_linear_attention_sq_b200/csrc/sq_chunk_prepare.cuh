// sq_chunk_prepare.cuh -- the gated delta rule in blocks of 64 rows, first
// kernel: everything of a block that does not depend on the state.
//
// With G_i the sum of log gates of the block's rows 0..i, S the state before
// the block, and for i > j (i >= j for P)
//     A_ij = beta_i e^(G_i - G_j) k_i . k_j,   P_ij = e^(G_i - G_j) q_i . k_j,
// the rows' updates u solve (1 + A) u = beta (v - e^G (k S)), so with
// T = (1 + A)^-1 diag(beta)
//     u = T r,   r_j = v_j - e^(G_j) k_j S,   o = e^G q S + (P T) r,
//     S <- e^(G_63) S + sum_i e^(G_63 - G_i) k_i u_i^T.
// This kernel forms T and P T of every block and value head, in parallel over
// blocks, for sq_chunk_scan.cuh, which walks a request's blocks in order.
// q, k are bf16: their products are exact, accumulated in fp32 by the tensor
// cores. Gates are accumulated as fp64 logarithms: a difference G_i - G_j
// keeps its precision behind a gate of zero. The inverse is formed in fp32 by
// blocks of 16: the diagonal blocks by substitution, then pairs of blocks,
// [T1 0; -T2 A21 T1, T2], to 32 and to 64.
// T and P T are stored as three bf16 terms each, whose sum is the fp32 value,
// so that the scan's products keep fp32 accuracy; only the blocks on and
// below the diagonal are stored, in the order the scan's matrix instructions
// read them.
#pragma once

#include <cuda_bf16.h>

#include "sq_recurrent.cuh"

namespace sqr {

constexpr int kTerms = 3;                                    // bf16 terms of an fp32 operand
constexpr int kTermBytes = 32 * (128 + 96 + 64 + 32);        // one term of T and P T together
constexpr int kCoefFloats = 64 + 64 + 4;                     // e^G, e^(G_63 - G), e^(G_63)
constexpr int kPrepBytes = kTerms * kTermBytes + 4 * kCoefFloats;  // per block and value head
static_assert(kPrepBytes % 16 == 0, "bulk copies move 16-byte multiples");

// One term: for each 16 columns kk = j / 16, the operand rows that are not
// all zero there: rows 16 kk .. 63 of T in order, then rows 63 .. 16 kk of
// P T backwards, so that the 128 - 32 kk result columns are contiguous
// (u_16kk .. u_63, then o_63 .. o_16kk). Rows come in groups of 8 x 16
// columns, a group as two 8 x 8 pieces of 128 contiguous bytes (the tensor
// core's unswizzled layout).
__host__ __device__ constexpr int tri_base(int kk) { return kk * 4096 - kk * (kk - 1) * 512; }
__device__ __forceinline__ int tri_offset(int i, int j, bool pt) {
  const int kk = j >> 4, li = pt ? 127 - 16 * kk - i : i - 16 * kk;
  return tri_base(kk) + (li >> 3) * 256 + ((j >> 3) & 1) * 128 + (li & 7) * 16 + (j & 7) * 2;
}

struct PrepArgs {
  RaggedArgs r;
  const int32_t* cu_blocks;  // [B + 1]
  const int32_t* block_req;  // [n_blocks]
  uint8_t* ws;               // [n_blocks][h_v] records of kPrepBytes
  int32_t n_blocks;          // entries of block_req
};

// The block's request, first row and rows; false where there is nothing to do.
__device__ __forceinline__ bool block_span(const PrepArgs& a, int c, int& first, int& n) {
  if (c >= a.cu_blocks[a.r.B]) return false;
  const int b = a.block_req[c];
  if (b < 0 || b >= a.r.B) return false;
  int r0, len;
  ragged_span(a.r, b, r0, len);
  const int at = c - a.cu_blocks[b];
  if (len < a.r.min_long || at < 0 || at >= (len + 63) / 64) return false;
  first = r0 + 64 * at;
  n = min(64, len - 64 * at);
  return true;
}

// x = hi + mid + lo exactly, each a bf16: an fp32 value's 24 significant bits
// are three times 8, cut off one after the other. Two values at a time,
// packed as (a: low half, b: high half).
__device__ __forceinline__ uint32_t pack_high(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float2 cut(float2 x) {
  return make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffff0000u), __uint_as_float(__float_as_uint(x.y) & 0xffff0000u));
}
__device__ __forceinline__ void split3(float2 x, uint32_t (&t)[kTerms]) {
  const float2 hi = cut(x);
  t[0] = pack_high(hi.x, hi.y);
  const float2 r = __ffma2_rn(hi, make_float2(-1.0f, -1.0f), x);
  const float2 mid = cut(r);
  t[1] = pack_high(mid.x, mid.y);
  const float2 lo = __ffma2_rn(mid, make_float2(-1.0f, -1.0f), r);
  t[2] = pack_high(lo.x, lo.y);
}

constexpr int kPrepThreads = 128;
constexpr int kTile = 136;   // bf16 per row of the q and k tiles (16 bytes of padding)
constexpr int kPit = 68;     // floats per row of the 64 x 64 matrices
struct PrepSmem {
  union {
    __nv_bfloat16 qk[2][64 * kTile];
    float m[2][64 * kPit];   // A (later P), T
  };
  float kk[64 * kPit], qk_dot[64 * kPit];
  double G[64];
  float beta[64];
};
static_assert(sizeof(__nv_bfloat16) * 2 * 64 * kTile == sizeof(float) * 2 * 64 * kPit, "same size");

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sqk::smem_u32(p)));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// acc += X Y for 16 x 16 blocks (rows kPit floats apart), one warp: lane owns
// rows 2 (lane / 4), + 1 and columns 4 (lane % 4) .. + 3.
__device__ __forceinline__ void block_product(float2 (&acc)[2][2], const float* X, const float* Y) {
  const int lane = threadIdx.x & 31;
  const float* x0 = X + 2 * (lane >> 2) * kPit;
  const float* y0 = Y + 4 * (lane & 3);
#pragma unroll
  for (int l = 0; l < 16; l += 4) {
    const float4 a = *reinterpret_cast<const float4*>(x0 + l), b = *reinterpret_cast<const float4*>(x0 + kPit + l);
    const float xa[4] = {a.x, a.y, a.z, a.w}, xb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float4 y = *reinterpret_cast<const float4*>(y0 + (l + m) * kPit);
      const float2 ylo = make_float2(y.x, y.y), yhi = make_float2(y.z, y.w);
      acc[0][0] = __ffma2_rn(make_float2(xa[m], xa[m]), ylo, acc[0][0]);
      acc[0][1] = __ffma2_rn(make_float2(xa[m], xa[m]), yhi, acc[0][1]);
      acc[1][0] = __ffma2_rn(make_float2(xb[m], xb[m]), ylo, acc[1][0]);
      acc[1][1] = __ffma2_rn(make_float2(xb[m], xb[m]), yhi, acc[1][1]);
    }
  }
}
__device__ __forceinline__ void block_store(float* X, const float2 (&acc)[2][2], float f) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < 2; ++r)
    *reinterpret_cast<float4*>(X + (2 * (lane >> 2) + r) * kPit + 4 * (lane & 3)) =
        make_float4(f * acc[r][0].x, f * acc[r][0].y, f * acc[r][1].x, f * acc[r][1].y);
}
__device__ __forceinline__ float* blk(float* M, int bi, int bj) { return M + 16 * bi * kPit + 16 * bj; }

// Four columns of a row of T or P T, times beta, as three terms.
__device__ __forceinline__ void emit(uint8_t* out, int i, int j, bool pt, float4 x, const float* beta) {
  const float4 f = *reinterpret_cast<const float4*>(beta + j);
  uint32_t lo[kTerms], hi[kTerms];
  split3(make_float2(x.x * f.x, x.y * f.y), lo);
  split3(make_float2(x.z * f.z, x.w * f.w), hi);
  const int at = tri_offset(i, j, pt);
#pragma unroll
  for (int s = 0; s < kTerms; ++s) *reinterpret_cast<uint2*>(out + s * kTermBytes + at) = make_uint2(lo[s], hi[s]);
}

// One CTA per block and key head; the value heads that share the key head
// share q . k and k . k.
__global__ void __launch_bounds__(kPrepThreads, 3) k_chunk_prepare(const PrepArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  PrepSmem& s = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int c = blockIdx.x / a.r.h_k, hk = blockIdx.x - c * a.r.h_k;
  int first, n;
  if (!block_span(a, c, first, n)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int x = tid; x < 2 * 64 * 16; x += kPrepThreads) {
    const int which = x >> 10, row = (x >> 4) & 63, piece = x & 15;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(which ? a.r.k : a.r.q) +
                               (int64_t)(first + min(row, n - 1)) * (which ? a.r.k_stride : a.r.q_stride) + hk * 128;
    uint4 v = reinterpret_cast<const uint4*>(src)[piece];
    if (row >= n) v = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(&s.qk[which][row * kTile + 8 * piece]) = v;
  }
  __syncthreads();
  // the ten 16 x 16 blocks on and below the diagonal of k k^T and of q k^T
  for (int item = warp; item < 20; item += 4) {
    const int t = item >> 1, which = item & 1;  // 0: q k^T, 1: k k^T
    const int bi = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    const int bj = t - bi * (bi + 1) / 2;
    float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
    const __nv_bfloat16* A = &s.qk[which][(16 * bi + (lane & 15)) * kTile + 8 * (lane >> 4)];
    const __nv_bfloat16* Bm = &s.qk[1][(16 * bj + (lane & 7) + 8 * (lane >> 4)) * kTile + 8 * ((lane >> 3) & 1)];
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t fa[4], fb[4];
      ldmatrix4(fa, A + 16 * ks);
      ldmatrix4(fb, Bm + 16 * ks);
      mma_bf16(c0, fa, fb[0], fb[1]);
      mma_bf16(c1, fa, fb[2], fb[3]);
    }
    float* D = blk(which ? s.kk : s.qk_dot, bi, bj) + (lane >> 2) * kPit + 2 * (lane & 3);
    *reinterpret_cast<float2*>(D) = make_float2(c0[0], c0[1]);
    *reinterpret_cast<float2*>(D + 8) = make_float2(c1[0], c1[1]);
    *reinterpret_cast<float2*>(D + 8 * kPit) = make_float2(c0[2], c0[3]);
    *reinterpret_cast<float2*>(D + 8 * kPit + 8) = make_float2(c1[2], c1[3]);
  }
  float *A = s.m[0], *T = s.m[1];
  const int share = a.r.h_v / a.r.h_k;
  for (int hh = 0; hh < share; ++hh) {
    const int h = hk * share + hh;
    uint8_t* rec = a.ws + ((uint64_t)c * a.r.h_v + h) * kPrepBytes;
    float* coef = reinterpret_cast<float*>(rec + kTerms * kTermBytes);
    __syncthreads();  // the dots (first head); the previous head's matrices have been read
    if (warp == 0) {
      double l[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int i = 2 * lane + x;
        const size_t at = (size_t)(first + min(i, n - 1)) * a.r.h_v + h;
        const float g = i < n ? clamp_gate(a.r.g[at]) : 1.0f;
        s.beta[i] = i < n ? a.r.beta[at] : 0.0f;
        // a gate of zero counts as 2^-126; a NaN stays one
        l[x] = log2((double)(g < 1.17549435e-38f ? 1.17549435e-38f : g));
      }
      double sum = l[0] + l[1], inc = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      const double G0 = inc - l[1], G1 = inc, G63 = __shfl_sync(0xffffffffu, inc, 31);
      s.G[2 * lane] = G0;
      s.G[2 * lane + 1] = G1;
      reinterpret_cast<float2*>(coef)[lane] = make_float2(exp2f((float)G0), exp2f((float)G1));
      reinterpret_cast<float2*>(coef + 64)[lane] = make_float2(exp2f((float)(G63 - G0)), exp2f((float)(G63 - G1)));
      if (lane < 4) coef[128 + lane] = exp2f((float)G63);
    }
    __syncthreads();
    for (int x = tid; x < 10 * 256; x += kPrepThreads) {
      const int t = x >> 8, bi = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, bj = t - bi * (bi + 1) / 2;
      const int i = 16 * bi + ((x >> 4) & 15), j = 16 * bj + (x & 15);
      A[i * kPit + j] = i > j ? s.beta[i] * (exp2f((float)(s.G[i] - s.G[j])) * s.kk[i * kPit + j]) : 0.0f;
    }
    __syncthreads();
    {  // diagonal blocks: lane owns a column of its warp's block (both half warps the same)
      const float* Ad = blk(A, warp, warp);
      float* Td = blk(T, warp, warp);
      const int col = lane & 15;
      float t[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float acc = i == col ? 1.0f : 0.0f;
#pragma unroll
        for (int l = 0; l < i; ++l) acc = fmaf(-Ad[i * kPit + l], t[l], acc);
        t[i] = acc;
      }
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) Td[i * kPit + col] = t[i];
      }
    }
    // pairs of blocks to 32 and pairs of those to 64; intermediate products go
    // to the unused blocks above the diagonal
    auto zero = [](float2 (&x)[2][2]) { x[0][0] = x[0][1] = x[1][0] = x[1][1] = make_float2(0.f, 0.f); };
    float2 acc[2][2];
    __syncthreads();
    if (warp < 2) {
      const int p = 2 * warp;
      zero(acc);
      block_product(acc, blk(A, p + 1, p), blk(T, p, p));
      block_store(blk(T, p, p + 1), acc, 1.0f);
      __syncwarp();
      zero(acc);
      block_product(acc, blk(T, p + 1, p + 1), blk(T, p, p + 1));
      block_store(blk(T, p + 1, p), acc, -1.0f);
    }
    __syncthreads();
    const int bi = warp >> 1, bj = warp & 1;
    zero(acc);
    for (int l = bj; l < 2; ++l) block_product(acc, blk(A, 2 + bi, l), blk(T, l, bj));
    block_store(blk(T, bi, 2 + bj), acc, 1.0f);
    __syncthreads();
    zero(acc);
    for (int l = 0; l <= bi; ++l) block_product(acc, blk(T, 2 + bi, 2 + l), blk(T, l, 2 + bj));
    block_store(blk(T, 2 + bi, bj), acc, -1.0f);
    // A has been used: P takes its place
    for (int x = tid; x < 10 * 256; x += kPrepThreads) {
      const int t = x >> 8, pi = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, pj = t - pi * (pi + 1) / 2;
      const int i = 16 * pi + ((x >> 4) & 15), j = 16 * pj + (x & 15);
      A[i * kPit + j] = i >= j ? exp2f((float)(s.G[i] - s.G[j])) * s.qk_dot[i * kPit + j] : 0.0f;
    }
    __syncthreads();
    // P T: five block products for each warp; T and P T leave as three terms
    const int r0 = 2 * (lane >> 2), c0 = 4 * (lane & 3);
    const int todo[4] = {0x3000, 0x2010, 0x3121, 0x32112233};  // (bi, bj) of each warp, low digits first
    const int count[4] = {2, 2, 2, 4};
    for (int x = 0; x < count[warp]; ++x) {
      const int code = (todo[warp] >> (8 * x)) & 0xff, pi = code >> 4, pj = code & 15;
      zero(acc);
      for (int l = pj; l <= pi; ++l) block_product(acc, blk(A, pi, l), blk(T, l, pj));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = 16 * pi + r0 + r, j = 16 * pj + c0;
        emit(rec, i, j, true, make_float4(acc[r][0].x, acc[r][0].y, acc[r][1].x, acc[r][1].y), s.beta);
        emit(rec, i, j, false, *reinterpret_cast<const float4*>(T + i * kPit + j), s.beta);
      }
    }
  }
}

}  // namespace sqr
