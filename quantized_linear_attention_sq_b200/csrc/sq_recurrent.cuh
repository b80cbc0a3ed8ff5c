// sq_recurrent.cuh -- the gated delta rule row by row over a ragged batch
// (sq_prefill_ragged: single tokens, short requests, gates by key channel).
//
// One CTA of 2 D threads per (request, value head); the fp32 state stays in
// registers from its load to its store: a lane owns four columns of RPT key
// rows, so a warp reads and writes whole rows of the state with 16-byte
// accesses. A row (token) costs one barrier: with S the gated state before
// the update,
//     p = S^T k,  u = beta (v - p),  o = (S + k u^T)^T q = S^T q + (k . q) u,
// so both column sums are taken of the same state, their per-warp partials
// cross the CTA through shared memory once, and every thread finishes the
// sums of its own columns and applies S += k u^T.
// One row per request is bound by HBM (the state is read and written once:
// 2 x 64 KiB per head at D = 128, two CTAs per SM keep 128 KiB in flight);
// many rows are bound by the latency of that exchange.
#pragma once

#include <cuda_bf16.h>

#include "sq_kernels.cuh"

namespace sqr {

using sqk::Geo;
using sqk::ROW_PIVOT;
using sqk::ST_NAN;
using sqk::ST_SLOT;
using sqk::Tables;

struct RaggedArgs {
  uint8_t* pool;              // packed pool, or fp32 S pool (fmt_fp32)
  const void* q;              // [rows, h_k, d] with row strides
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements
  const float* beta;          // [rows, h_v]
  const float* g;             // [rows, h_v] or [rows, h_v, d]
  void* o;                    // [rows, h_v, d]
  const int32_t* cu_seqlens;  // [B + 1]
  const int32_t* past;        // [B] or null
  const int32_t* slots;       // [B] or null
  int32_t B, rows, h_v, h_k, n_slots, fmt_fp32;
  int32_t min_long;           // requests of at least this many rows are another kernel's (0: none is)
  uint64_t slot_bytes;
  Tables t;
};

// Request b's rows, cut to the arrays.
__device__ __forceinline__ void ragged_span(const RaggedArgs& a, int b, int& first, int& n) {
  first = min(max(a.cu_seqlens[b], 0), a.rows);
  n = min(max(a.cu_seqlens[b + 1], first), a.rows) - first;
}

__device__ __forceinline__ float clamp_gate(float g) {
  return g != g ? g : fminf(fmaxf(g, 0.0f), 1.0f);  // a NaN stays one
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(__half* p, float x) { *p = __float2half_rn(x); }

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(__half* p, float4 x) {
  const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <int D>
struct RGeo {
  static constexpr int NT = 2 * D;              // threads
  static constexpr int NW = NT / 32;            // warps
  static constexpr int LPR = D / 4;             // lanes per key row (four columns each)
  static constexpr int RP = 32 / LPR;           // key rows a warp covers at once
  static constexpr int RPT = D / (NW * RP);     // key rows per thread
  static constexpr int VEC = 4 * D + 4;         // floats of a row's vectors: k q v g | beta, gate
  static constexpr int RED = 2 * NW * D;        // floats of the warps' partials: p, o
  static constexpr size_t FLOATS = 3 * VEC + 2 * RED;
  static constexpr size_t SMEM = FLOATS * 4;
  // packed pools: the fp32 state on its way between the record's thread map
  // and this kernel's, the record, the head's row tables
  static size_t packed_smem(uint32_t rec) { return SMEM + (size_t)D * D * 4 + (rec + 15) / 16 * 16 + 7 * D; }
};

// The slot's packed record, dequantized into S [D][D] in shared memory.
// `sync`: a barrier of the Geo<D>::NT threads that call it.
template <int D, typename Sync>
__device__ __forceinline__ void unpack_state(const RaggedArgs& a, int h, const uint8_t* src, uint8_t* rec, float* S,
                                             Sync sync) {
  using G = Geo<D>;
  static_assert(G::NT == RGeo<D>::NT, "one thread map");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cc = lane % G::LPR, rg = warp * G::RPW + lane / G::LPR;
  const uint32_t rb = a.t.rec_bytes[h];
  for (uint32_t x = tid * 16; x < rb; x += G::NT * 16)
    *reinterpret_cast<uint4*>(rec + x) = *reinterpret_cast<const uint4*>(src + x);
  sync();
  const float* col = a.t.col + (size_t)h * D + 16 * cc;
#pragma unroll
  for (int r = 0; r < G::RPT; ++r) {
    const int i = r * G::NG + rg;
    const uint8_t code = a.t.row_code[(size_t)h * D + i];
    const float mul = code == ROW_PIVOT ? 1.0f : __half2float(reinterpret_cast<const __half*>(rec)[i]);
    float2 T[8];
    sqk::load_row(rec + a.t.row_off[(size_t)h * D + i], code, cc, mul, T);
#pragma unroll
    for (int p = 0; p < 8; ++p)
      reinterpret_cast<float2*>(S + (size_t)i * D + 16 * cc)[p] =
          __fmul2_rn(T[p], make_float2(col[2 * p], col[2 * p + 1]));
  }
  sync();
}

// S [D][D] in shared memory, quantized into the slot's record
// (the quantization of sq_quantize_state). Returns status bits.
template <int D, typename Sync>
__device__ __forceinline__ uint32_t pack_state(const RaggedArgs& a, int h, uint8_t* dst, uint8_t* rec, const float* S,
                                               Sync sync) {
  using G = Geo<D>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cc = lane % G::LPR, rg = warp * G::RPW + lane / G::LPR;
  const uint32_t rb = a.t.rec_bytes[h];
  float* phi = reinterpret_cast<float*>(rec + (rb + 15) / 16 * 16);
  uint16_t* row_off = reinterpret_cast<uint16_t*>(phi + D);
  uint8_t* row_code = reinterpret_cast<uint8_t*>(row_off + D);
  for (int i = tid; i < D; i += G::NT) {
    row_off[i] = a.t.row_off[(size_t)h * D + i];
    row_code[i] = a.t.row_code[(size_t)h * D + i];
    phi[i] = a.t.phi[(size_t)h * D + i];
  }
  for (uint32_t x = tid * 16; x < rb; x += G::NT * 16) *reinterpret_cast<uint4*>(rec + x) = make_uint4(0, 0, 0, 0);
  sync();  // the tables, the cleared record, and S
  const float* icol = a.t.icol + (size_t)h * D + 16 * cc;
  float2 T[G::RPT][8];
#pragma unroll
  for (int r = 0; r < G::RPT; ++r)
#pragma unroll
    for (int p = 0; p < 8; ++p)
      T[r][p] = __fmul2_rn(reinterpret_cast<const float2*>(S + (size_t)(r * G::NG + rg) * D + 16 * cc)[p],
                           make_float2(icol[2 * p], icol[2 * p + 1]));
  const uint32_t st = sqk::requant_rows<D, 0>(rec, row_off, row_code, phi, rg, cc, false, T);
  sync();
  for (uint32_t x = tid * 16; x < rb; x += G::NT * 16)
    *reinterpret_cast<uint4*>(dst + x) = *reinterpret_cast<const uint4*>(rec + x);
  return st;
}

template <int D, bool KDA, bool PACKED, typename T>
__global__ void __launch_bounds__(RGeo<D>::NT, 2) k_ragged_rows(const RaggedArgs a) {
  using R = RGeo<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* vec = reinterpret_cast<float*>(smem);   // three rows' vectors
  float* red = vec + 3 * R::VEC;                 // two rows' partials
  float* Ssh = vec + R::FLOATS;                  // packed pools
  uint8_t* rec = reinterpret_cast<uint8_t*>(Ssh + D * D);
  const int b = blockIdx.x / a.h_v, h = blockIdx.x - b * a.h_v;
  int first, n;
  ragged_span(a, b, first, n);
  if (a.min_long && n >= a.min_long) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = a.slots ? a.slots[b] : b;
  T* out = static_cast<T*>(a.o) + ((size_t)first * a.h_v + h) * D;
  const size_t out_step = (size_t)a.h_v * D;
  if (slot < 0 || slot >= a.n_slots) {
    for (int t = 0; t < n; ++t)
      if (tid < D) from_f32(out + t * out_step + tid, 0.0f);
    if (tid == 0) atomicOr(a.t.status, ST_SLOT);
    return;
  }
  const bool resume = a.past && a.past[b] > 0;
  if (n == 0 && resume) return;
  const int c4 = 4 * (lane % R::LPR), rsub = lane / R::LPR;
  const int row0 = (warp * R::RP + rsub) * R::RPT;  // this thread's key rows: RPT from there
  uint8_t* record = a.pool + (uint64_t)slot * a.slot_bytes + (PACKED ? a.t.rec_off[h] : 0u);
  float* S_pool = reinterpret_cast<float*>(a.pool) + ((size_t)slot * a.h_v + h) * D * D;

  // thread tid < D brings k and v of channel tid, the others q and g
  const int hk = h / (a.h_v / a.h_k);
  const int ch = tid < D ? tid : tid - D;
  float x0 = 0.0f, x1 = 0.0f, xb = 0.0f, xg = 1.0f;
  auto fetch = [&](int t) {
    const size_t row = (size_t)first + t;
    if (tid < D) {
      x0 = to_f32(static_cast<const T*>(a.k)[row * a.k_stride + hk * D + ch]);
      x1 = to_f32(static_cast<const T*>(a.v)[row * a.v_stride + h * D + ch]);
      if (tid == 0) xb = a.beta[row * a.h_v + h];
      if (!KDA && tid == 1) xg = clamp_gate(a.g[row * a.h_v + h]);
    } else {
      x0 = to_f32(static_cast<const T*>(a.q)[row * a.q_stride + hk * D + ch]);
      if (KDA) x1 = clamp_gate(a.g[(row * a.h_v + h) * D + ch]);
    }
  };
  auto deposit = [&](float* w) {
    if (tid < D) {
      w[ch] = x0;
      w[2 * D + ch] = x1;
      if (tid == 0) w[4 * D] = xb;
      if (!KDA && tid == 1) w[4 * D + 1] = xg;
    } else {
      w[D + ch] = x0;
      if (KDA) w[3 * D + ch] = x1;
    }
  };

  float4 S[R::RPT];
  if (n > 0) fetch(0);
  if (PACKED && resume) {
    unpack_state<D>(a, h, record, rec, Ssh, [] { __syncthreads(); });
#pragma unroll
    for (int r = 0; r < R::RPT; ++r) S[r] = *reinterpret_cast<const float4*>(Ssh + (row0 + r) * D + c4);
  } else {
#pragma unroll
    for (int r = 0; r < R::RPT; ++r)
      S[r] = resume ? *reinterpret_cast<const float4*>(S_pool + (size_t)(row0 + r) * D + c4)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (n > 0) deposit(vec);
  __syncthreads();

  uint32_t st = 0;
  int cur = 0;  // t % 3
  for (int t = 0; t < n; ++t) {
    const float* w = vec + cur * R::VEC;
    const int nxt = cur == 2 ? 0 : cur + 1;
    float* rd = red + (t & 1) * R::RED;
    if (t + 1 < n) fetch(t + 1);
    const float gate = KDA ? 1.0f : w[4 * D + 1];
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f), s = p;
#pragma unroll
    for (int r4 = 0; r4 < R::RPT; r4 += 4) {
      const float4 k4 = *reinterpret_cast<const float4*>(w + row0 + r4), q4 = *reinterpret_cast<const float4*>(w + D + row0 + r4);
      const float4 g4 = KDA ? *reinterpret_cast<const float4*>(w + 3 * D + row0 + r4) : make_float4(gate, gate, gate, gate);
      const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w}, gg[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int r = r4 + y;
        S[r].x *= gg[y]; S[r].y *= gg[y]; S[r].z *= gg[y]; S[r].w *= gg[y];
        p.x = fmaf(S[r].x, kk[y], p.x); p.y = fmaf(S[r].y, kk[y], p.y);
        p.z = fmaf(S[r].z, kk[y], p.z); p.w = fmaf(S[r].w, kk[y], p.w);
        s.x = fmaf(S[r].x, qq[y], s.x); s.y = fmaf(S[r].y, qq[y], s.y);
        s.z = fmaf(S[r].z, qq[y], s.z); s.w = fmaf(S[r].w, qq[y], s.w);
      }
    }
#pragma unroll
    for (int d = R::LPR; d < 32; d <<= 1) {  // the key rows a warp covers at once
      p.x += __shfl_xor_sync(0xffffffffu, p.x, d); p.y += __shfl_xor_sync(0xffffffffu, p.y, d);
      p.z += __shfl_xor_sync(0xffffffffu, p.z, d); p.w += __shfl_xor_sync(0xffffffffu, p.w, d);
      s.x += __shfl_xor_sync(0xffffffffu, s.x, d); s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
      s.z += __shfl_xor_sync(0xffffffffu, s.z, d); s.w += __shfl_xor_sync(0xffffffffu, s.w, d);
    }
    if (rsub == 0) {
      *reinterpret_cast<float4*>(rd + warp * D + c4) = p;
      *reinterpret_cast<float4*>(rd + (R::NW + warp) * D + c4) = s;
    }
    // slot nxt was last read after the barrier of row t - 2, which every
    // thread has passed before the barrier of row t - 1
    if (t + 1 < n) deposit(vec + nxt * R::VEC);
    __syncthreads();
    float4 P = *reinterpret_cast<const float4*>(rd + c4);
#pragma unroll
    for (int x = 1; x < R::NW; ++x) {
      const float4 y = *reinterpret_cast<const float4*>(rd + x * D + c4);
      P.x += y.x; P.y += y.y; P.z += y.z; P.w += y.w;
    }
    const float beta = w[4 * D];
    const float4 v = *reinterpret_cast<const float4*>(w + 2 * D + c4);
    const float4 u = make_float4(beta * (v.x - P.x), beta * (v.y - P.y), beta * (v.z - P.z), beta * (v.w - P.w));
    if (warp == t % R::NW) {  // the warps take turns at o
      float kq = 0.0f;
#pragma unroll
      for (int x = lane; x < D; x += 32) kq = fmaf(w[x], w[D + x], kq);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) kq += __shfl_xor_sync(0xffffffffu, kq, d);
      float4 O = *reinterpret_cast<const float4*>(rd + R::NW * D + c4);
#pragma unroll
      for (int x = 1; x < R::NW; ++x) {
        const float4 y = *reinterpret_cast<const float4*>(rd + (R::NW + x) * D + c4);
        O.x += y.x; O.y += y.y; O.z += y.z; O.w += y.w;
      }
      O.x = fmaf(kq, u.x, O.x); O.y = fmaf(kq, u.y, O.y); O.z = fmaf(kq, u.z, O.z); O.w = fmaf(kq, u.w, O.w);
      if (O.x != O.x || O.y != O.y || O.z != O.z || O.w != O.w) st |= ST_NAN;
      if (rsub == 0) {
        T* op = out + t * out_step + c4;
        store4(op, O);
      }
    }
#pragma unroll
    for (int r4 = 0; r4 < R::RPT; r4 += 4) {
      const float4 k4 = *reinterpret_cast<const float4*>(w + row0 + r4);
      const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float4& t = S[r4 + y];
        t.x = fmaf(kk[y], u.x, t.x); t.y = fmaf(kk[y], u.y, t.y);
        t.z = fmaf(kk[y], u.z, t.z); t.w = fmaf(kk[y], u.w, t.w);
      }
    }
    cur = nxt;
  }

  if (PACKED) {
#pragma unroll
    for (int r = 0; r < R::RPT; ++r) *reinterpret_cast<float4*>(Ssh + (row0 + r) * D + c4) = S[r];
    st |= pack_state<D>(a, h, record, rec, Ssh, [] { __syncthreads(); });  // its first barrier orders S
  } else {
#pragma unroll
    for (int r = 0; r < R::RPT; ++r) *reinterpret_cast<float4*>(S_pool + (size_t)(row0 + r) * D + c4) = S[r];
  }
  if (st) atomicOr(a.t.status, st);
}

}  // namespace sqr
