// sq_recurrent.cuh -- the gated delta rule row by row over a ragged batch
// (sq_prefill_ragged: single tokens, short requests, gates by key channel).
//
// CTAs of 2 D threads, two per SM, walk over (request, value head) tiles; a
// tile's fp32 state stays in registers from its load to its store: a lane
// owns four columns of RPT key rows, so a warp reads and writes whole rows of
// the state with 16-byte accesses. A row (token) costs one barrier: with S
// the gated state before the update,
//     p = S^T k,  u = beta (v - p),  o = (S + k u^T)^T q = S^T q + (k . q) u,
// so both column sums are taken of the same state, their per-warp partials
// cross the CTA through shared memory once, and every thread finishes the
// sums of its own columns and applies S += k u^T.
// One row per request is bound by HBM (the state is read and written once, 2
// x 64 KiB per head at D = 128): the next tile's state (or packed record)
// comes into shared memory by bulk copy while this one is worked on, and its
// first row's vectors are fetched before this one's state is stored: 512
// single tokens with 32 heads take 365 us, 0.90 of the measured copy rate (385
// before CTAs walked over tiles with copies under way). Many rows are bound by
// the latency of the exchange: 128 requests of 1..6 rows with gates by key
// channel take 118 us, 0.71 of it. At two CTAs per SM a thread has 128 registers:
// fp32 rows at D = 128 spill (head gates: 88 bytes stored, 172 loaded, 32 and 52
// with packed states; channel gates: 28 and 40), 16-bit rows 4 and 8 bytes or none.
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
  uint32_t rec_cap;           // largest packed record
  uint64_t slot_bytes, wait_ns;
  uint64_t drain_ns;          // limit of the waits for copies under way after a wait has run out
  uint32_t test_extra_tx;     // testing only: extra bytes the first wait of tile (request 0, head 0) expects (0: none)
  Tables t;
};

// Launches that overlap (programmatic dependence): a kernel lets the next one
// of its call start as soon as all its own CTAs have, and waits for the one
// before it to be over where it needs its results, and before it ends, so
// that the end of a call is the end of all its kernels. Without effect in a
// plain launch.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Request b's rows, cut to the arrays.
__device__ __forceinline__ void ragged_span(const RaggedArgs& a, int b, int& first, int& n) {
  first = min(max(a.cu_seqlens[b], 0), a.rows);
  n = min(max(a.cu_seqlens[b + 1], first), a.rows) - first;
}

__device__ __forceinline__ float clamp_gate(float g) {  // to [0, 1]; a NaN stays one
  float r;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, 0f00000000;\n\tmin.NaN.f32 %0, t, 0f3F800000;\n\t}" : "=f"(r) : "f"(g));
  return r;
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

// x *= f, y += x f, two elements an instruction.
__device__ __forceinline__ void mul4(float4& x, float f) {
  const float2 a = __fmul2_rn(make_float2(x.x, x.y), make_float2(f, f));
  const float2 b = __fmul2_rn(make_float2(x.z, x.w), make_float2(f, f));
  x = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void fma4(float4& y, const float4& x, float f) {
  const float2 a = __ffma2_rn(make_float2(x.x, x.y), make_float2(f, f), make_float2(y.x, y.y));
  const float2 b = __ffma2_rn(make_float2(x.z, x.w), make_float2(f, f), make_float2(y.z, y.w));
  y = make_float4(a.x, a.y, b.x, b.y);
}
// Four elements as fp32.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const __half* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sqk::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all_groups() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// One row's vectors in shared memory, as they came: k, q, v, then (fp32) the
// key channels' gates, beta, the head's gate.
template <int D, typename T>
struct RowVectors {
  T k[D], q[D], v[D];
  float g[D];
  float beta, gate, pad[2];
};

template <int D>
struct RGeo {
  static constexpr int NT = 2 * D;              // threads
  static constexpr int NW = NT / 32;            // warps
  static constexpr int LPR = D / 4;             // lanes per key row (four columns each)
  static constexpr int RP = 32 / LPR;           // key rows a warp covers at once
  static constexpr int RPT = D / (NW * RP);     // key rows per thread
  static constexpr int RED = 2 * NW * D;        // floats of the warps' partials: p, o
  static constexpr int RING = 4;                // rows' vectors at hand or on their way
  static constexpr size_t FIXED = ((size_t)RING * sizeof(RowVectors<D, float>) + 2 * RED * 4 + 127) / 128 * 128;
  static constexpr size_t STATE = (size_t)D * D * 4;
  // fp32 pools: the next tile's state. Packed pools: the fp32 state on its way
  // between the record's thread map and this kernel's (and then the record
  // going out), the next tile's record, the head's row tables; at 8 bits and
  // D = 128 two CTAs fit per SM
  static size_t smem(bool packed, uint32_t rec) {
    return FIXED + STATE + (packed ? (rec + 127) / 128 * 128 + 7 * D : 0);
  }
};

// A tile of work: rows `first` .. + n of one request, one value head.
struct RowTile {
  int32_t b, h, first, n, slot;
  int32_t what;  // TILE_*
};
enum { TILE_END = 0, TILE_RUN = 1, TILE_RESUME = 2, TILE_ZERO = 4 };  // RUN: store a state; ZERO: a bad slot, o = 0

// A head's row tables and column scales as a thread of the record's thread map
// needs them to dequantize, read before the record is there.
template <int D>
struct RecordMap {
  uint32_t row[Geo<D>::RPT];  // offset of the row's codes, its width above
  float4 col[4];
};
template <int D>
__device__ __forceinline__ void map_record(const RaggedArgs& a, int h, RecordMap<D>& m) {
  using G = Geo<D>;
  static_assert(G::NT == RGeo<D>::NT, "one thread map");
  const int lane = threadIdx.x & 31, cc = lane % G::LPR, rg = (threadIdx.x >> 5) * G::RPW + lane / G::LPR;
#pragma unroll
  for (int r = 0; r < G::RPT; ++r)
    m.row[r] = a.t.row_off[(size_t)h * D + r * G::NG + rg] | (uint32_t)a.t.row_code[(size_t)h * D + r * G::NG + rg] << 16;
#pragma unroll
  for (int p = 0; p < 4; ++p) m.col[p] = *reinterpret_cast<const float4*>(a.t.col + (size_t)h * D + 16 * cc + 4 * p);
}
// A packed record in shared memory, dequantized into S [D][D] there.
template <int D>
__device__ __forceinline__ void unpack_record(const RecordMap<D>& m, const uint8_t* rec, float* S) {
  using G = Geo<D>;
  const int lane = threadIdx.x & 31, cc = lane % G::LPR, rg = (threadIdx.x >> 5) * G::RPW + lane / G::LPR;
#pragma unroll
  for (int r = 0; r < G::RPT; ++r) {
    const int i = r * G::NG + rg;
    const uint8_t code = (uint8_t)(m.row[r] >> 16);
    const float mul = code == ROW_PIVOT ? 1.0f : __half2float(reinterpret_cast<const __half*>(rec)[i]);
    float2 T[8];
    sqk::load_row(rec + (m.row[r] & 0xffffu), code, cc, mul, T);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 lo = __fmul2_rn(T[2 * p], make_float2(m.col[p].x, m.col[p].y));
      const float2 hi = __fmul2_rn(T[2 * p + 1], make_float2(m.col[p].z, m.col[p].w));
      reinterpret_cast<float4*>(S + (size_t)i * D + 16 * cc)[p] = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

// The head's tables that the quantization reads (D row impacts, row offsets,
// row widths: 7 D bytes), on their way to shared memory.
template <int D>
__device__ __forceinline__ void fetch_pack_tables(const RaggedArgs& a, int h, uint8_t* t) {
  for (int x = threadIdx.x; x < 7 * D / 4; x += Geo<D>::NT) {
    const uint8_t* src = x < D ? reinterpret_cast<const uint8_t*>(a.t.phi + (size_t)h * D + x)
                         : x < D + D / 2 ? reinterpret_cast<const uint8_t*>(a.t.row_off + (size_t)h * D) + 4 * (x - D)
                                         : a.t.row_code + (size_t)h * D + 4 * (x - D - D / 2);
    sqk::cp_async4(t + 4 * x, src);
  }
  sqk::cp_async_commit();
}
// S [D][D] in shared memory, quantized into the slot's record (the
// quantization of sq_quantize_state) with the tables of fetch_pack_tables.
// The record is built where S was. `sync`: a barrier of the Geo<D>::NT
// threads that call it; one has passed since S and the tables were complete.
// Returns status bits.
template <int D, typename Sync>
__device__ __forceinline__ uint32_t pack_state(const RaggedArgs& a, int h, uint8_t* dst, float* S, const uint8_t* tables,
                                               Sync sync) {
  using G = Geo<D>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cc = lane % G::LPR, rg = warp * G::RPW + lane / G::LPR;
  const uint32_t rb = a.t.rec_bytes[h];
  uint8_t* rec = reinterpret_cast<uint8_t*>(S);
  const float* phi = reinterpret_cast<const float*>(tables);
  const uint16_t* row_off = reinterpret_cast<const uint16_t*>(phi + D);
  const uint8_t* row_code = reinterpret_cast<const uint8_t*>(row_off + D);
  float4 icol[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) icol[p] = *reinterpret_cast<const float4*>(a.t.icol + (size_t)h * D + 16 * cc + 4 * p);
  float2 T[G::RPT][8];
#pragma unroll
  for (int r = 0; r < G::RPT; ++r)
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float4 x = reinterpret_cast<const float4*>(S + (size_t)(r * G::NG + rg) * D + 16 * cc)[p];
      T[r][2 * p] = __fmul2_rn(make_float2(x.x, x.y), make_float2(icol[p].x, icol[p].y));
      T[r][2 * p + 1] = __fmul2_rn(make_float2(x.z, x.w), make_float2(icol[p].z, icol[p].w));
    }
  sync();  // S has been read
  if (tid == 0) *reinterpret_cast<uint4*>(rec + rb - 16) = make_uint4(0, 0, 0, 0);  // the padding's bytes
  sync();
  const uint32_t st = sqk::requant_rows<D, 0>(rec, row_off, row_code, phi, rg, cc, false, T);
  sync();
  for (uint32_t x = tid * 16; x < rb; x += G::NT * 16)
    *reinterpret_cast<uint4*>(dst + x) = *reinterpret_cast<const uint4*>(rec + x);
  return st;
}

// The search for a CTA's next tile of work, by one warp: each lane looks at
// one of the next 32 tiles of the CTA. What it needs of them is on its way to
// shared memory (`ask`) while the warp does other work, then `answer` picks
// the first tile with work (asking again where none has any).
struct TileSearch {
  int32_t got[4][32];  // cu_seqlens[b], cu_seqlens[b + 1], past[b], slots[b]
};
__device__ __forceinline__ void ask(const RaggedArgs& a, TileSearch& s, uint32_t at, uint32_t step) {
  const int lane = threadIdx.x & 31;
  const uint32_t mine = at + lane * step;
  if (mine >= at && mine < (uint32_t)a.B * a.h_v) {
    const uint32_t b = mine / a.h_v;
    sqk::cp_async4(&s.got[0][lane], a.cu_seqlens + b);
    sqk::cp_async4(&s.got[1][lane], a.cu_seqlens + b + 1);
    if (a.past) sqk::cp_async4(&s.got[2][lane], a.past + b);
    if (a.slots) sqk::cp_async4(&s.got[3][lane], a.slots + b);
  }
  sqk::cp_async_commit();
}
__device__ __forceinline__ RowTile answer(const RaggedArgs& a, TileSearch& s, uint32_t& at, uint32_t step) {
  const int lane = threadIdx.x & 31;
  const uint32_t tiles = (uint32_t)a.B * a.h_v;
  while (at < tiles) {
    sqk::cp_async_wait_all();
    const uint32_t mine = at + lane * step;
    RowTile t{};
    if (mine >= at && mine < tiles) {
      t.b = mine / a.h_v;
      t.h = mine - t.b * a.h_v;
      t.first = min(max(s.got[0][lane], 0), a.rows);
      t.n = min(max(s.got[1][lane], t.first), a.rows) - t.first;
      if (!(a.min_long && t.n >= a.min_long)) {
        t.slot = a.slots ? s.got[3][lane] : t.b;
        const bool resume = a.past && s.got[2][lane] > 0;
        if (t.slot < 0 || t.slot >= a.n_slots) t.what = TILE_ZERO;
        else if (t.n > 0 || !resume) t.what = resume ? TILE_RUN | TILE_RESUME : TILE_RUN;
      }
    }
    const uint32_t found = __ballot_sync(0xffffffffu, t.what != TILE_END);
    if (found) {
      const int from = __ffs(found) - 1;
      t.b = __shfl_sync(0xffffffffu, t.b, from);
      t.h = __shfl_sync(0xffffffffu, t.h, from);
      t.first = __shfl_sync(0xffffffffu, t.first, from);
      t.n = __shfl_sync(0xffffffffu, t.n, from);
      t.slot = __shfl_sync(0xffffffffu, t.slot, from);
      t.what = __shfl_sync(0xffffffffu, t.what, from);
      at += (from + 1) * step;
      return t;
    }
    if (at + 32ull * step >= tiles) break;
    at += 32 * step;
    ask(a, s, at, step);
  }
  at = tiles;
  return RowTile{};
}

template <int D, bool KDA, bool PACKED, typename T>
__global__ void __launch_bounds__(RGeo<D>::NT, 2) k_ragged_rows(const RaggedArgs a) {
  using R = RGeo<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  using Row = RowVectors<D, T>;
  Row* ring = reinterpret_cast<Row*>(smem);
  float* red = reinterpret_cast<float*>(smem + R::RING * sizeof(RowVectors<D, float>));  // two rows' partials
  float* Ssh = reinterpret_cast<float*>(smem + R::FIXED);  // fp32 pools: the incoming state; packed: see RGeo
  uint8_t* rec_in = smem + R::FIXED + R::STATE;
  uint8_t* tables = rec_in + (a.rec_cap + 127) / 128 * 128;
  __shared__ RowTile tiles[3];                   // this one, the next, the one behind it
  __shared__ TileSearch search;
  __shared__ __align__(8) uint64_t arrived;      // the incoming state or record
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c4 = 4 * (lane % R::LPR), rsub = lane / R::LPR;
  const int row0 = (warp * R::RP + rsub) * R::RPT;  // this thread's key rows: RPT from there

  auto state_of = [&](const RowTile& t) { return reinterpret_cast<float*>(a.pool) + ((size_t)t.slot * a.h_v + t.h) * D * D; };
  auto record_of = [&](const RowTile& t) { return a.pool + (uint64_t)t.slot * a.slot_bytes + a.t.rec_off[t.h]; };
  auto bring = [&](const RowTile& t) {  // by one thread
    if (!(t.what & TILE_RESUME)) return;
    const uint32_t bytes = PACKED ? a.t.rec_bytes[t.h] : (uint32_t)R::STATE;
    sqk::mbar_arrive_expect_tx(&arrived, bytes + (t.b == 0 && t.h == 0 ? a.test_extra_tx : 0u));
    if (PACKED) sqk::bulk_g2s(rec_in, record_of(t), bytes, &arrived);
    else sqk::bulk_g2s(Ssh, state_of(t), bytes, &arrived);
  };
  // Row t of tile c on its way to a ring slot, one group of copies (an empty one if there is no such row).
  auto fetch = [&](const RowTile& c, int t, uint32_t slot) {
    if (t < c.n && (c.what & TILE_RUN)) {
      Row& w = ring[slot % R::RING];
      const size_t row = (size_t)c.first + t;
      constexpr int P = D * (int)sizeof(T) / 16;  // pieces of 16 bytes of k, q and v
      static_assert(3 * P + 2 <= R::NT && D / 4 + 2 <= R::NT, "one piece per thread");
      const int hk = c.h / (a.h_v / a.h_k);
      const int which = tid / P, x = tid % P * (16 / (int)sizeof(T));
      if (which == 0) cp_async16(w.k + x, static_cast<const T*>(a.k) + row * a.k_stride + hk * D + x);
      else if (which == 1) cp_async16(w.q + x, static_cast<const T*>(a.q) + row * a.q_stride + hk * D + x);
      else if (which == 2) cp_async16(w.v + x, static_cast<const T*>(a.v) + row * a.v_stride + c.h * D + x);
      else if (tid == 3 * P) sqk::cp_async4(&w.beta, a.beta + row * a.h_v + c.h);
      else if (!KDA && tid == 3 * P + 1) sqk::cp_async4(&w.gate, a.g + row * a.h_v + c.h);
      if (KDA && tid >= R::NT - D / 4) {
        const int y = 4 * (tid - (R::NT - D / 4));
        cp_async16(w.g + y, a.g + (row * a.h_v + c.h) * D + y);
      }
    }
    sqk::cp_async_commit();
  };

  let_next_start();
  if (tid == 0) {
    sqk::mbar_init(&arrived, 1);
    sqk::fence_mbar_init();
  }
  uint32_t at = blockIdx.x;  // warp 0: the search goes on here
  if (warp == 0) {
    for (int x = 0; x < 2; ++x) {
      ask(a, search, at, gridDim.x);
      const RowTile t = answer(a, search, at, gridDim.x);
      if (lane == 0) {
        tiles[x] = t;
        if (x == 0) bring(t);
      }
    }
  }
  __syncthreads();
  uint32_t phase = 0, st = 0, base = 0;  // base: ring slot of the tile's first row
  fetch(tiles[0], 0, 0);
  fetch(tiles[0], 1, 1);
  for (int turn = 0; tiles[turn].what != TILE_END; turn = turn == 2 ? 0 : turn + 1) {
    const RowTile& c = tiles[turn];
    const RowTile& nx = tiles[turn == 2 ? 0 : turn + 1];
    const int n = c.n;
    T* out = static_cast<T*>(a.o) + ((size_t)c.first * a.h_v + c.h) * D;
    const size_t out_step = (size_t)a.h_v * D;
    const bool resume = c.what & TILE_RESUME;
    float4 S[R::RPT];
    bool ok = true;
    if (PACKED) {
      if (resume) {
        RecordMap<D> m;
        map_record<D>(a, c.h, m);
        ok = sqk::mbar_wait_bounded(&arrived, phase & 1, a.wait_ns);
        if (ok) unpack_record<D>(m, rec_in, Ssh);
      }
      if (c.what & TILE_RUN) fetch_pack_tables<D>(a, c.h, tables);
      __syncthreads();
    } else if (resume) {
      ok = sqk::mbar_wait_bounded(&arrived, phase & 1, a.wait_ns);
    }
    if (resume) ++phase;
#pragma unroll
    for (int r = 0; r < R::RPT; ++r)
      S[r] = resume && ok ? *reinterpret_cast<const float4*>(Ssh + (row0 + r) * D + c4) : make_float4(0.f, 0.f, 0.f, 0.f);
    cp_async_wait_but_one();  // the first row
    if (!__syncthreads_and(ok)) {  // the state did not come: the CTA's tiles from this one on stay as they are
      st |= sqk::ST_TIMEOUT;
      // no copy is under way when the CTA ends
      if (tid == 0) (void)sqk::mbar_wait_bounded(&arrived, (phase - 1) & 1, a.drain_ns);
      cp_async_wait_all_groups();
      break;
    }
    if (tid == 0) bring(nx);  // every thread has taken this tile's state
    if (warp == 0) ask(a, search, at, gridDim.x);
    if (c.what == TILE_ZERO) {
      for (int t = 0; t < n; ++t)
        if (tid < D) from_f32(out + t * out_step + tid, 0.0f);
      st |= ST_SLOT;
    }
#pragma unroll 1
    for (int t = 0; t < n && c.what != TILE_ZERO; ++t) {
      const Row& w = ring[(base + t) % R::RING];
      float* rd = red + (t & 1) * R::RED;
      // the slot of row t + 2 was last read after the barrier of row t - 2, which every thread has left
      fetch(c, t + 2, base + t + 2);
      const float gate = KDA ? 1.0f : clamp_gate(w.gate);
      float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r4 = 0; r4 < R::RPT; r4 += 4) {
        const float4 k4 = load4(w.k + row0 + r4);
        float4 g4 = make_float4(gate, gate, gate, gate);
        if (KDA) {
          g4 = load4(w.g + row0 + r4);
          g4 = make_float4(clamp_gate(g4.x), clamp_gate(g4.y), clamp_gate(g4.z), clamp_gate(g4.w));
        }
        const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, gg[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          float4& x = S[r4 + y];
          mul4(x, gg[y]);
          fma4(p, x, kk[y]);
        }
      }
      auto deposit = [&](float4 x, float* to) {
#pragma unroll
        for (int d = R::LPR; d < 32; d <<= 1) {  // the key rows a warp covers at once
          x.x += __shfl_xor_sync(0xffffffffu, x.x, d); x.y += __shfl_xor_sync(0xffffffffu, x.y, d);
          x.z += __shfl_xor_sync(0xffffffffu, x.z, d); x.w += __shfl_xor_sync(0xffffffffu, x.w, d);
        }
        if (rsub == 0) *reinterpret_cast<float4*>(to + c4) = x;
      };
      deposit(p, rd + warp * D);
      p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r4 = 0; r4 < R::RPT; r4 += 4) {
        const float4 q4 = load4(w.q + row0 + r4);
        const float qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          fma4(p, S[r4 + y], qq[y]);
        }
      }
      deposit(p, rd + (R::NW + warp) * D);
      cp_async_wait_but_one();  // the next row
      __syncthreads();
      auto collect = [&](const float* from) {
        float4 x = *reinterpret_cast<const float4*>(from + c4);
#pragma unroll
        for (int y = 1; y < R::NW; ++y) {
          const float4 z = *reinterpret_cast<const float4*>(from + y * D + c4);
          x.x += z.x; x.y += z.y; x.z += z.z; x.w += z.w;
        }
        return x;
      };
      const float4 P = collect(rd), v = load4(w.v + c4);
      const float beta = w.beta;
      const float4 u = make_float4(beta * (v.x - P.x), beta * (v.y - P.y), beta * (v.z - P.z), beta * (v.w - P.w));
      if (warp == t % R::NW) {  // the warps take turns at o
        float kq = 0.0f;
#pragma unroll
        for (int x = lane; x < D; x += 32) kq = fmaf(to_f32(w.k[x]), to_f32(w.q[x]), kq);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) kq += __shfl_xor_sync(0xffffffffu, kq, d);
        float4 O = collect(rd + R::NW * D);
        O.x = fmaf(kq, u.x, O.x); O.y = fmaf(kq, u.y, O.y); O.z = fmaf(kq, u.z, O.z); O.w = fmaf(kq, u.w, O.w);
        if (O.x != O.x || O.y != O.y || O.z != O.z || O.w != O.w) st |= ST_NAN;
        if (rsub == 0) store4(out + t * out_step + c4, O);
      }
#pragma unroll
      for (int r4 = 0; r4 < R::RPT; r4 += 4) {
        const float4 k4 = load4(w.k + row0 + r4);
        const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          fma4(S[r4 + y], u, kk[y]);
        }
      }
    }

    if (warp == 0) {
      const RowTile t = answer(a, search, at, gridDim.x);
      if (lane == 0) tiles[turn == 0 ? 2 : turn - 1] = t;
    }
    base += n;
    fetch(nx, 0, base);
    fetch(nx, 1, base + 1);
    if (c.what & TILE_RUN) {
      if (PACKED) {
#pragma unroll
        for (int r = 0; r < R::RPT; ++r) *reinterpret_cast<float4*>(Ssh + (row0 + r) * D + c4) = S[r];
        cp_async_wait_all_groups();  // the tables (and the next rows)
        __syncthreads();
        st |= pack_state<D>(a, c.h, record_of(c), Ssh, tables, [] { __syncthreads(); });
      } else {
        float* S_pool = state_of(c);
#pragma unroll
        for (int r = 0; r < R::RPT; ++r) *reinterpret_cast<float4*>(S_pool + (size_t)(row0 + r) * D + c4) = S[r];
      }
    }
    __syncthreads();  // the rows' vectors and the staged state have been read
  }
  if (st) atomicOr(a.t.status, st);
  wait_for_previous();
}

}  // namespace sqr
