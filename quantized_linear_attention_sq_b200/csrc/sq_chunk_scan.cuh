// sq_chunk_scan.cuh -- the gated delta rule in blocks of 64 rows, second
// kernel: the walk over a request's blocks (see sq_chunk_prepare.cuh for the
// formulas and for T and P T).
//
// One CTA per (request, value head), one per SM. The transposed state S^T
// [128 value columns][128 key rows] lives in registers in fp32 (a thread owns
// one value column and a quarter of the key rows) and all four products of a block
// run on the tensor cores with a transposed left operand out of tensor
// memory, so no operand that a thread computes ever goes through shared
// memory:
//     D1 = S^T [q; k]^T         (A: S^T,  B: the q and k tiles as TMA left them)
//     D2 = r^T [T; P T]^T       (A: r^T,  B: the prepared block)
//     D3 = (e^(G63 - G) u)^T k  (A: u^T,  B: the k tile again, read the other way)
// with r = beta (v - e^G D1k), u = D2u, o = e^G D1q + D2o, S <- e^(G63) S + D3 in
// fp32 by the threads. S, r and u are split into three bf16 terms (T and P T
// are stored so), k and q are bf16 already: D1 and D3 take three products,
// D2 the six largest of nine, so that the state, and o before its rounding to
// bf16, are fp32-accurate. The state adds one fresh accumulator per block in fp32:
// the tensor core never accumulates across blocks.
//
// Eighteen warps: sixteen compute (four per 32 lanes of tensor memory, sharing
// the columns), one moves (TMA loads of the next block, stores of o), one
// issues the matrix products. The chain of a block is D1k -> r -> D2 -> u ->
// D3 -> S; D3 and S go by halves of the key rows, so that the second half of
// D3 and the first of the next D1k run under S. The q product runs under r, o
// is finished and leaves under D3, and the next block's rows are taken in under
// the next D1k; v and o pass between rows and tensor memory by ldmatrix and
// stmatrix.
// Bound by the latency of that chain: about 5.25 k cycles a block (32 requests
// of 2048 rows with 32 heads: 755 us; one request of 32768 rows: 1420 us); in
// 24 requests of 0..1900 rows the tensor pipe is active 47 % of the time and a
// scheduler issues 0.47 instructions a cycle. With two terms for S the 32
// requests took 756 us where three took 822, but the state's error against 64
// bits rose from 2.4e-7 to 1.0e-6: three stay. Two terms for what only reaches
// o took 710 us where three take 755, but values some 1000 times smaller than
// those they overwrote came back 1 to 2 % off: three there too.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "sq_chunk_prepare.cuh"

namespace sqr {

constexpr int kScanCompute = 512;             // threads that own a part of the state
constexpr int kScanThreads = kScanCompute + 64;
constexpr int kMoveWarp = kScanCompute / 32, kProductWarp = kMoveWarp + 1;
constexpr int kScanStages = 2;
constexpr uint32_t kTileBytes = 64 * 128 * 2;  // q, k, v or o rows of a block
// A stage: channels 0..63 of the q rows, then of the k rows, the same for
// channels 64..127, channels 0..63 and 64..127 of the v rows (all 128-byte
// swizzled: 16-byte piece x of row r is at x ^ (r & 7)), the prepared block.
constexpr uint32_t kStageV = 2 * kTileBytes, kStagePrep = 3 * kTileBytes;
constexpr uint32_t kStageBytes = kStagePrep + (kPrepBytes + 1023) / 1024 * 1024;
constexpr uint32_t kStageTx = kStagePrep + kPrepBytes;
constexpr uint32_t kOutAt = kScanStages * kStageBytes;  // o rows on their way out

constexpr int kRanked = 256;  // most requests that are taken by length, see request_of
struct ScanCtl {
  uint64_t full[kScanStages], empty[kScanStages];
  uint64_t s_ready[2], d3[2];
  uint64_t r_ready, u_ready, d1, d2, d2o, o_ready, o_free, drain;
  uint32_t tmem;
  int32_t abort, request;
  alignas(16) int32_t length[kRanked];  // of request_of: not where TMA writes, which ordinary stores are not ordered with
};
constexpr size_t kScanSmem = 1024 + kOutAt + kTileBytes + sizeof(ScanCtl) + 16;

// Byte offset of 16-byte piece x of row r in a tile of v or o rows.
__device__ __forceinline__ int tile_piece(int r, int x) {
  return (x >> 3) * (kTileBytes / 2) + r * 128 + (((x & 7) ^ (r & 7)) << 4);
}

struct ScanArgs {
  PrepArgs p;
};

// Columns of tensor memory (all 512).
constexpr uint32_t TM_S = 0;      // S^T terms hi and mid, over D3: 16 columns for each 16 key rows; lo from 128 on
constexpr uint32_t TM_R = 192;    // r^T terms
constexpr uint32_t TM_D1Q = 288;  // S^T q^T
constexpr uint32_t TM_D1K = 352;  // S^T k^T
constexpr uint32_t TM_D2 = 352;   // u^T (over S^T k^T), then the P T part of o
// u^T terms: two over the lo terms of S^T, which D1 has read, one behind the rest.
__host__ __device__ constexpr uint32_t u_col(int s) { return s == 2 ? 480u : 128u + 32u * s; }

// Column of term s of S^T for key rows 16 ks .. 16 ks + 15.
__host__ __device__ constexpr uint32_t s_col(int s, int ks) {
  return s == 2 ? 128u + 8u * ks : 16u * ks + 8u * s;
}

// ---------------------------------------------------------- instructions
__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          sqk::smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(sqk::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, int z, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(sqk::smem_u32(src))
               : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The barrier gets one arrival when every product issued so far is done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sqk::smem_u32(bar))
               : "memory");
}
// D (+)= A B, A [128 x 16] bf16 in tensor memory, B in shared memory.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
#define SQ_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define SQ_W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
__device__ __forceinline__ void tc_ld16(uint32_t (&x)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : SQ_R8(x, 0), SQ_R8(x, 8)
      : "r"(addr)
      : "memory");
}
// Waits for the loads; the values pass through it, so no use of them moves above.
#define SQ_RW8(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]), "+r"(x[i + 4]), "+r"(x[i + 5]), "+r"(x[i + 6]), "+r"(x[i + 7])
__device__ __forceinline__ void tc_wait_ld(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SQ_RW8(x, 0), SQ_RW8(x, 8)::"memory");
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const uint32_t (&x)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), SQ_W8(x, 0)
               : "memory");
}

// The same by fragments, as the warp-wide matrix instructions lay out a
// result: 16 lanes from `addr`'s on, 16 columns; this lane gets rows lane / 4
// (x[4 g], x[4 g + 1]) and + 8 (x[4 g + 2], x[4 g + 3]), columns 8 g + 2
// (lane % 4), + 1.
__device__ __forceinline__ void tc_ld_frag(uint32_t (&x)[8], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : SQ_R8(x, 0) : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&x)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SQ_RW8(x, 0)::"memory");
}
// 8 columns of 32 bits: rows lane / 4 (x[2 g]) and + 8 (x[2 g + 1]), column 4 g + lane % 4.
__device__ __forceinline__ void tc_st_frag(uint32_t addr, const uint32_t (&x)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3])
               : "memory");
}
__device__ __forceinline__ void stmatrix4t(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(sqk::smem_u32(p)), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

// fp32 accumulators, bf16 operands, M = 128, N columns; `mn`: B has N
// contiguous; `a_term`: term of A, of which the second is stored negated.
__host__ __device__ constexpr uint32_t mma_desc(uint32_t N, bool mn, int a_term) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_term == 1 ? 1u << 13 : 0u) | (mn ? 1u << 16 : 0u) | ((N >> 3) << 17) |
         ((128u >> 4) << 24);
}
// x = t[0] - t[1] + t[2] for two values at a time, each term rounded to
// nearest (8 bits each: the sum is x). A bf16 is subtracted as it is, so the
// differences come with alternating sign: 7 instructions, a fifth less time
// than cutting and packing.
__device__ __forceinline__ void bf16_minus(uint32_t t, float a, float b, float& x, float& y) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tsub.rn.f32.bf16 %0, l, %3;\n\tsub.rn.f32.bf16 %1, h, %4;\n\t}"
      : "=f"(x), "=f"(y)
      : "r"(t), "f"(a), "f"(b));
}
__device__ __forceinline__ void split_a(float a, float b, uint32_t (&t)[kTerms]) {
  float x, y, z, w;
  t[0] = bf16x2(a, b);
  bf16_minus(t[0], a, b, x, y);
  t[1] = bf16x2(x, y);
  bf16_minus(t[1], x, y, z, w);
  t[2] = bf16x2(z, w);
}
// Shared memory operand: address, leading and stride offsets in bytes, swizzle mode (0 none, 2: 128 bytes).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride, uint64_t swizzle) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         (1ull << 46) | (swizzle << 61);
}

// A warp's 32 value columns x 16 rows of r or u, as fragments (x[h][...] the
// 16 lanes 16 h on), to tensor memory as three terms.
__device__ __forceinline__ void put_frag(const float (&x)[2][8], uint32_t hi, uint32_t mid, uint32_t lo) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t t[kTerms][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[kTerms];
      split_a(x[h][2 * i], x[h][2 * i + 1], w);
#pragma unroll
      for (int s = 0; s < kTerms; ++s) t[s][i] = w[s];
    }
    const uint32_t lanes = (uint32_t)(16 * h) << 16;
    tc_st_frag(hi + lanes, t[0]);
    tc_st_frag(mid + lanes, t[1]);
    tc_st_frag(lo + lanes, t[2]);
  }
}

// A warp's arrival on a barrier once its tensor memory stores are done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  tc_wait_st();
  tc_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) sqk::mbar_arrive(bar);
}

// Wait of a whole warp; false: it ran out, in any lane.
__device__ __forceinline__ bool warp_wait(ScanCtl& c, uint64_t* bar, uint32_t parity, uint64_t ns) {
  const bool ok = sqk::mbar_wait_bounded(bar, parity, ns);
  if (__all_sync(0xffffffffu, ok)) return true;
  c.abort = 1;
  return false;
}

// The 256 threads of the record's thread map.
__device__ __forceinline__ void record_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The request whose turn it is as the `rank`-th: of up to kRanked requests the
// longest start first, so that no long one is left to run alone (24 requests
// of 0..1900 rows: 146 us in their own order, 113 by length). Each CTA sorts for
// itself, which would take long with more: those run in their own order, and a
// long request behind many short ones starts only after the short ones' CTAs,
// which leave at once, have had their turns.
__device__ __forceinline__ int request_of(const RaggedArgs& a, int rank, ScanCtl& ctl) {
  if (a.B > kRanked || a.B == 1) return rank;
  const int tid = threadIdx.x, padded = (a.B + 3) & ~3;
  int n = -1;
  if (tid < a.B) {
    int first;
    ragged_span(a, tid, first, n);
  }
  if (tid < padded) ctl.length[tid] = n;
  __syncthreads();
  if (tid < a.B) {
    int before = 0;
    for (int j = 0; j < padded; j += 4) {
      const int4 l = *reinterpret_cast<const int4*>(ctl.length + j);
      before += (l.x > n || (l.x == n && j < tid)) + (l.y > n || (l.y == n && j + 1 < tid)) +
                (l.z > n || (l.z == n && j + 2 < tid)) + (l.w > n || (l.w == n && j + 3 < tid));
    }
    if (before == rank) ctl.request = tid;
  }
  __syncthreads();
  return ctl.request;
}

template <bool PACKED>
__global__ void __launch_bounds__(kScanThreads, 1)
    k_chunk_scan(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap o_map,
                 const ScanArgs args) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ScanCtl& ctl = *reinterpret_cast<ScanCtl*>(smem + kOutAt + kTileBytes);
  const RaggedArgs& a = args.p.r;
  const int rank = blockIdx.x / a.h_v, h = blockIdx.x - rank * a.h_v, hk = h / (a.h_v / a.h_k);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = request_of(a, rank, ctl);
  // everything about the request at once: its loads wait on none of each other
  const int slot = a.slots ? a.slots[b] : b, c0 = args.p.cu_blocks[b];
  const bool resume = a.past && a.past[b] > 0;
  int first, n;
  ragged_span(a, b, first, n);
  if (n < a.min_long) {
    wait_for_previous();
    return;
  }
  const int blocks = (n + 63) >> 6;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o);
  if (slot < 0 || slot >= a.n_slots || !blocks_within(c0, blocks, args.p.n_blocks)) {
    const int64_t pieces = row_pieces(n);
    for (int64_t x = tid; x < pieces; x += kScanThreads)
      reinterpret_cast<uint4*>(out + ((size_t)(first + (x >> 4)) * a.h_v + h) * 128)[x & 15] = make_uint4(0, 0, 0, 0);
    if (tid == 0) atomicOr(a.t.status, ST_SLOT);
    wait_for_previous();
    return;
  }
  uint8_t* record = a.pool + (uint64_t)slot * a.slot_bytes + (PACKED ? a.t.rec_off[h] : 0u);
  float* S_pool = reinterpret_cast<float*>(a.pool) + ((size_t)slot * a.h_v + h) * 128 * 128;

  if (tid == 0) {
    constexpr uint32_t warps = kScanCompute / 32;
    for (int x = 0; x < 2; ++x) {
      sqk::mbar_init(&ctl.full[x], 1);
      sqk::mbar_init(&ctl.empty[x], warps);
      sqk::mbar_init(&ctl.s_ready[x], warps);
      sqk::mbar_init(&ctl.d3[x], 1);
    }
    sqk::mbar_init(&ctl.r_ready, warps);
    sqk::mbar_init(&ctl.u_ready, warps);
    sqk::mbar_init(&ctl.o_ready, warps);
    sqk::mbar_init(&ctl.o_free, 1);
    sqk::mbar_init(&ctl.d1, 1);
    sqk::mbar_init(&ctl.d2, 1);
    sqk::mbar_init(&ctl.d2o, 1);
    sqk::mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    sqk::fence_mbar_init();
  }
  if (warp == kProductWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sqk::smem_u32(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // S^T: value column of this thread's lane; S[y][j] is key row 64 y + 16 part + j
  const int part = warp >> 2, col = (warp & 3) * 32 + lane;  // compute warps
  float S[2][16];
  if (PACKED && resume) {
    uint8_t* rec = smem + 128 * 128 * 4;
    if (warp < 8) {
      for (uint32_t x = tid * 16; x < a.t.rec_bytes[h]; x += 256 * 16) cp_async16(rec + x, record + x);
      sqk::cp_async_commit();
      RecordMap<128> m;
      map_record<128>(a, h, m);
      cp_async_wait_all_groups();
      record_sync();
      unpack_record<128>(m, rec, reinterpret_cast<float*>(smem));
    }
    __syncthreads();
  }
  if (warp < kMoveWarp) {
    const float* src = (PACKED ? reinterpret_cast<const float*>(smem) : S_pool) + (size_t)(16 * part) * 128 + col;
#pragma unroll
    for (int x = 0; x < 32; ++x) S[x >> 4][x & 15] = resume ? src[(64 * (x >> 4) + (x & 15)) * 128] : 0.0f;
    if (PACKED && resume) sqk::fence_proxy_async_smem();  // before TMA writes where S was read
  }
  wait_for_previous();  // the prepared blocks; before the first wait with a limit
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = ctl.tmem;
  const uint64_t ns = a.wait_ns;
  uint32_t st = 0;

  if (warp == kMoveWarp) {  // ------------------------------- loads and stores
    int issued = 0;
    auto load = [&](int i) {
      const int sg = i & 1;
      uint8_t* stage = smem + sg * kStageBytes;
      const int row = first + 64 * i;
      if (lane == 0) {
        sqk::mbar_arrive_expect_tx(&ctl.full[sg], kStageTx + (b == 0 && h == 0 && i == 0 ? a.test_extra_tx : 0u));
        tma_tile(stage + kTileBytes / 2, &k_map, 0, hk, row, &ctl.full[sg]);
        tma_tile(stage + 3 * kTileBytes / 2, &k_map, 64, hk, row, &ctl.full[sg]);
        tma_tile(stage, &q_map, 0, hk, row, &ctl.full[sg]);
        tma_tile(stage + kTileBytes, &q_map, 64, hk, row, &ctl.full[sg]);
        tma_tile(stage + kStageV, &v_map, 0, h, row, &ctl.full[sg]);
        tma_tile(stage + kStageV + kTileBytes / 2, &v_map, 64, h, row, &ctl.full[sg]);
        sqk::bulk_g2s(stage + kStagePrep, args.p.ws + ((uint64_t)(c0 + i) * a.h_v + h) * kPrepBytes, kPrepBytes,
                      &ctl.full[sg]);
      }
      issued = i + 1;
    };
    load(0);
    if (blocks > 1) load(1);
    for (int i = 0; i < blocks; ++i) {
      // block i's stage is free when its D3 is done; its o follows
      if (i + kScanStages < blocks) {
        if (!warp_wait(ctl, &ctl.empty[i & 1], (i >> 1) & 1, ns)) break;
        load(i + kScanStages);
      }
      if (!warp_wait(ctl, &ctl.o_ready, i & 1, ns)) break;
      const int live = n - 64 * i;
      if (live >= 64) {
        if (lane == 0) {
          tma_store(&o_map, 0, h, first + 64 * i, smem + kOutAt);
          tma_store(&o_map, 64, h, first + 64 * i, smem + kOutAt + kTileBytes / 2);
          sqk::bulk_commit();
          sqk::bulk_wait_read_all();
        }
      } else {  // the last block: its live rows only
        for (int y = lane; y < live * 16; y += 32) {
          const int row = y >> 4, piece = y & 15;
          reinterpret_cast<uint4*>(out + ((size_t)(first + 64 * i + row) * a.h_v + h) * 128)[piece] =
              *reinterpret_cast<const uint4*>(smem + kOutAt + tile_piece(row, piece));
        }
      }
      __syncwarp();
      if (lane == 0) sqk::mbar_arrive(&ctl.o_free);
    }
    // no copy is in flight when the CTA ends
    for (int i = max(0, issued - kScanStages); i < issued; ++i)
      sqk::mbar_wait_bounded(&ctl.full[i & 1], (i >> 1) & 1, a.drain_ns);
    if (lane == 0) sqk::bulk_wait_all();
  } else if (warp == kProductWarp) {  // ------------------------------------- products
    const uint32_t base = sqk::smem_u32(smem);
    for (int i = 0; i < blocks; ++i) {
      const uint32_t ph = i & 1;
      const uint32_t stage = base + (i & 1) * kStageBytes;
      const uint64_t qt = smem_desc(stage, 16, 1024, 2), kt = qt + kTileBytes / 32;
      if (!warp_wait(ctl, &ctl.full[i & 1], (i >> 1) & 1, ns)) break;
      bool ok = true;
#pragma unroll
      for (int y = 0; y < 2; ++y) {  // k: the key rows 64 y .. 64 y + 63
        ok = ok && warp_wait(ctl, &ctl.s_ready[y], ph, ns);
        tc_after();
        if (ok && elect_one()) {
#pragma unroll
          for (int s = kTerms - 1; s >= 0; --s)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma(tm + TM_D1K, tm + TM_S + s_col(s, ks) + (s == 2 ? 32 : 64) * y, kt + y * kTileBytes / 16 + ks * 2,
                     mma_desc(64, false, s), s < kTerms - 1 || ks > 0 || y > 0);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) {
        tc_commit(&ctl.d1);
#pragma unroll
        for (int s = kTerms - 1; s >= 0; --s)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc_mma(tm + TM_D1Q, tm + TM_S + s_col(s, ks), qt + ((ks >> 2) * kTileBytes + (ks & 3) * 32) / 16,
                   mma_desc(64, false, s), s < kTerms - 1 || ks > 0);
      }
      __syncwarp();
      // rows 16 kk .. 63 of T see columns 16 kk .. 16 kk + 15: the six largest products of terms of r and of T, the
      // largest last; then the same for P T
      if (!warp_wait(ctl, &ctl.r_ready, ph, ns)) break;
      tc_after();
      if (elect_one()) {
        const uint64_t prep = smem_desc(stage + kStagePrep, 128, 256, 0);
        constexpr int pr[6] = {2, 0, 1, 1, 0, 0}, pt[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
        for (int x = 0; x < 6; ++x)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma(tm + TM_D2 + 16 * kk, tm + TM_R + 32 * pr[x] + 8 * kk,
                   prep + (term_base(pt[x]) + pair_base(kk)) / 16,
                   mma_desc(64 - 16 * kk, false, pr[x]), x > 0 || kk > 0);
        tc_commit(&ctl.d2);
#pragma unroll
        for (int x = 0; x < 6; ++x)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // P T follows T's 64 - 16 kk rows, 32 bytes each
            tc_mma(tm + TM_D2 + 64 + 16 * kk, tm + TM_R + 32 * pr[x] + 8 * kk,
                   prep + (term_base(pt[x]) + pair_base(kk) + 32 * (64 - 16 * kk)) / 16,
                   mma_desc(64 - 16 * kk, false, pr[x]), x > 0 || kk > 0);
        tc_commit(&ctl.d2o);
      }
      __syncwarp();
      if (!warp_wait(ctl, &ctl.u_ready, ph, ns)) break;
      tc_after();
      if (elect_one()) {
        const uint64_t km = smem_desc(stage + kTileBytes / 2, kTileBytes, 1024, 2);
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // key rows 64 x .. 64 x + 63
#pragma unroll
          for (int s = kTerms - 1; s >= 0; --s)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma(tm + TM_S + 64 * x, tm + u_col(s) + 8 * kk, km + (x * kTileBytes + kk * 2048) / 16,
                     mma_desc(64, true, s), s < kTerms - 1 || kk > 0);
          tc_commit(&ctl.d3[x]);
        }
      }
      __syncwarp();
    }
    // no product is in flight when the tensor memory is given back
    if (elect_one()) tc_commit(&ctl.drain);
    __syncwarp();
    warp_wait(ctl, &ctl.drain, 0, a.drain_ns);
  } else {  // -------------------------------------------------- the rest
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    auto split_state = [&](int y, uint32_t (&t)[kTerms][8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t z[kTerms];
        split_a(S[y][2 * j], S[y][2 * j + 1], z);
#pragma unroll
        for (int s = 0; s < kTerms; ++s) t[s][j] = z[s];
      }
    };
    auto put_state = [&](int y, const uint32_t (&t)[kTerms][8]) {
      const uint32_t to = tl + TM_S + 16 * part;
      tc_st8(to + 64 * y, t[0]);
      tc_st8(to + 64 * y + 8, t[1]);
      tc_st8(tl + TM_S + 128 + 32 * y + 8 * part, t[2]);
      warp_arrive(&ctl.s_ready[y]);
    };
    // r, u and o go by fragments: rows j = 16 part + 8 g + 2 (lane % 4), + 1 of value columns lane / 4 + 8 m of the warp's
    const uint32_t rt = tl + TM_R + 8 * part, ut = tl + 8 * part;
    constexpr uint32_t upper = 16u << 16;                         // the warp's lanes 16..31
    const int j2 = 16 * part + 2 * (lane & 3);                    // first of this lane's rows
    const int at = tile_piece(16 * part + (lane & 7), 4 * (warp & 3) + (lane >> 3));  // of v or o: a matrix's row; g: + 1024
    for (int y = 0; y < 2; ++y) {
      uint32_t t[kTerms][8];
      split_state(y, t);
      put_state(y, t);
    }
    float x[2][8];
    // block i's rows: beta v into x; false where the wait ran out
    auto take_rows = [&](int i) {
      if (!warp_wait(ctl, &ctl.full[i & 1], (i >> 1) & 1, ns)) return false;
      uint8_t* stage = smem + (i & 1) * kStageBytes;
      const int live = n - 64 * i;
      if (live < 64) {
        // rows of the k tile behind the request's last: another request's, or none's
        for (int y = tid; y < (64 - live) * 16; y += kScanCompute)
          *reinterpret_cast<uint4*>(stage + kTileBytes / 2 + ((y >> 3) & 1) * kTileBytes + (live + (y >> 4)) * 128 +
                                    (y & 7) * 16) = make_uint4(0, 0, 0, 0);
        sqk::fence_proxy_async_smem();
      }
      const float* beta = reinterpret_cast<const float*>(stage + kStagePrep + kTermsBytes) + 64 + j2;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t v[4];
        ldmatrix4t(v, stage + kStageV + at + 1024 * g);
        const float2 e = *reinterpret_cast<const float2*>(beta + 8 * g);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          x[m >> 1][4 * g + 2 * (m & 1)] = e.x * __uint_as_float(v[m] << 16);
          x[m >> 1][4 * g + 2 * (m & 1) + 1] = e.y * __uint_as_float(v[m] & 0xffff0000u);
        }
      }
      return true;
    };
    bool ok = take_rows(0);
    for (int i = 0; i < blocks && ok; ++i) {
      const uint32_t ph = i & 1;
      const int live = min(64, n - 64 * i);
      const float* coef = reinterpret_cast<const float*>(smem + (i & 1) * kStageBytes + kStagePrep + kTermsBytes);
      uint32_t w[2][8];
      auto factors = [&](float2 (&e)[2], int from) {  // of this lane's rows, read before a wait
        e[0] = *reinterpret_cast<const float2*>(coef + from + j2);
        e[1] = *reinterpret_cast<const float2*>(coef + from + j2 + 8);
      };
      float2 e[2];
      factors(e, 128);
      if (!warp_wait(ctl, &ctl.d1, ph, ns)) break;
      tc_after();
      tc_ld_frag(w[0], tl + TM_D1K + 16 * part);
      tc_ld_frag(w[1], tl + upper + TM_D1K + 16 * part);
      tc_wait_ld(w[0]);
      tc_wait_ld(w[1]);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          float* y = &x[m >> 1][4 * g + 2 * (m & 1)];
          y[0] = fmaf(-e[g].x, __uint_as_float(w[m >> 1][4 * g + 2 * (m & 1)]), y[0]);
          y[1] = fmaf(-e[g].y, __uint_as_float(w[m >> 1][4 * g + 2 * (m & 1) + 1]), y[1]);
        }
      }
      if (live < 64) {  // whatever the rows behind the last held
#pragma unroll
        for (int z = 0; z < 16; ++z)
          if (j2 + 8 * ((z >> 2) & 1) + (z & 1) >= live) x[z >> 3][z & 7] = 0.0f;
      }
      put_frag(x, rt, rt + 32, rt + 64);
      warp_arrive(&ctl.r_ready);

      factors(e, 192);
      if (!warp_wait(ctl, &ctl.d2, ph, ns)) break;
      tc_after();
      tc_ld_frag(w[0], tl + TM_D2 + 16 * part);
      tc_ld_frag(w[1], tl + upper + TM_D2 + 16 * part);
      tc_wait_ld(w[0]);
      tc_wait_ld(w[1]);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          x[m >> 1][4 * g + 2 * (m & 1)] = e[g].x * __uint_as_float(w[m >> 1][4 * g + 2 * (m & 1)]);
          x[m >> 1][4 * g + 2 * (m & 1) + 1] = e[g].y * __uint_as_float(w[m >> 1][4 * g + 2 * (m & 1) + 1]);
        }
      }
      put_frag(x, ut + u_col(0), ut + u_col(1), ut + u_col(2));
      warp_arrive(&ctl.u_ready);

      // o, under the state's product
      factors(e, 0);
      if (!warp_wait(ctl, &ctl.d2o, ph, ns)) break;
      if (i > 0 && !warp_wait(ctl, &ctl.o_free, (i - 1) & 1, ns)) break;
      {
        uint32_t y[2][8];
        tc_after();
        tc_ld_frag(w[0], tl + TM_D1Q + 16 * part);
        tc_ld_frag(w[1], tl + upper + TM_D1Q + 16 * part);
        tc_ld_frag(y[0], tl + TM_D2 + 64 + 16 * part);
        tc_ld_frag(y[1], tl + upper + TM_D2 + 64 + 16 * part);
        tc_wait_ld(w[0]);
        tc_wait_ld(w[1]);
        tc_wait_ld(y[0]);
        tc_wait_ld(y[1]);
        uint32_t o[2][4];
        __nv_bfloat162 bad = __float2bfloat162_rn(0.0f);  // stays 0 while every o is finite
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int z = 4 * g + 2 * (m & 1);
            o[g][m] = bf16x2(fmaf(e[g].x, __uint_as_float(w[m >> 1][z]), __uint_as_float(y[m >> 1][z])),
                             fmaf(e[g].y, __uint_as_float(w[m >> 1][z + 1]), __uint_as_float(y[m >> 1][z + 1])));
            bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&o[g][m]), __float2bfloat162_rn(0.0f), bad);
          }
          stmatrix4t(smem + kOutAt + at + 1024 * g, o[g][0], o[g][1], o[g][2], o[g][3]);
        }
        if (*reinterpret_cast<const uint32_t*>(&bad) != 0) {  // an infinity or a NaN: a NaN in a live row is reported
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int m = 0; m < 4; ++m)
              if (((o[g][m] & 0x7fffu) > 0x7f80u && j2 + 8 * g < live) ||
                  ((o[g][m] & 0x7fffffffu) > 0x7f80ffffu && j2 + 8 * g + 1 < live))
                st |= ST_NAN;
        }
      }
      sqk::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) sqk::mbar_arrive(&ctl.o_ready);
      const float g63 = coef[256];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        ok = ok && warp_wait(ctl, &ctl.d3[y], ph, ns);
        if (!ok) break;
        tc_after();
        uint32_t d[16];
        tc_ld16(d, tl + TM_S + 64 * y + 16 * part);
        tc_wait_ld(d);
#pragma unroll
        for (int j = 0; j < 16; ++j) S[y][j] = fmaf(g63, S[y][j], __uint_as_float(d[j]));
        if (i + 1 < blocks) {
          uint32_t t[kTerms][8];
          split_state(y, t);
          // the lo terms go where the second half of D3 still reads u
          if (y == 0) ok = warp_wait(ctl, &ctl.d3[1], ph, ns);
          if (!ok) break;
          put_state(y, t);
        }
      }
      // under the next block's first product: its rows
      if (lane == 0) sqk::mbar_arrive(&ctl.empty[i & 1]);  // this warp's reads of the stage came before
      if (ok && i + 1 < blocks) ok = take_rows(i + 1);
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kProductWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  if (ctl.abort) {  // the state in the pool stays as it was
    if (tid == 0) atomicOr(a.t.status, sqk::ST_TIMEOUT);
    return;
  }
  if (warp < kMoveWarp) {
    float* dst = (PACKED ? reinterpret_cast<float*>(smem) : S_pool) + (size_t)(16 * part) * 128 + col;
#pragma unroll
    for (int x = 0; x < 32; ++x) dst[(64 * (x >> 4) + (x & 15)) * 128] = S[x >> 4][x & 15];
  }
  if (PACKED) {
    if (warp < 8) {
      fetch_pack_tables<128>(a, h, smem + 128 * 128 * 4);
      cp_async_wait_all_groups();
    }
    __syncthreads();
    if (warp < 8) st |= pack_state<128>(a, h, record, reinterpret_cast<float*>(smem), smem + 128 * 128 * 4, record_sync);
  }
  if (st) atomicOr(a.t.status, st);
}

}  // namespace sqr
