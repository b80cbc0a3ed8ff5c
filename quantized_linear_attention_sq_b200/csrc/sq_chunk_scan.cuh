// sq_chunk_scan.cuh -- the gated delta rule in blocks of 64 rows, second
// kernel: the walk over a request's blocks (see sq_chunk_prepare.cuh for the
// formulas and for T and P T).
//
// One CTA per (request, value head), one per SM. The transposed state S^T
// [128 value columns][128 key rows] lives in registers in fp32 (a thread owns
// one value column and half of the key rows) and all four products of a block
// run on the tensor cores with a transposed left operand out of tensor
// memory, so no operand that a thread computes ever goes through shared
// memory:
//     D1 = S^T [q; k]^T         (A: S^T,  B: the q and k tiles as TMA left them)
//     D2 = r^T [T; P T]^T       (A: r^T,  B: the prepared block)
//     D3 = (e^(G63 - G) u)^T k  (A: u^T,  B: the k tile again, read the other way)
// with r = beta (v - e^G D1k), u = D2u, o = e^G D1q + D2o, S <- e^(G63) S + D3 in
// fp32 by the threads. S, r and u are split into three bf16 terms (T and P T
// are stored so), k and q are bf16 already: D1k and D3 take three products,
// D2 the six largest of nine, so that the state is fp32-accurate; what only
// reaches o, which is bf16, takes two terms (D1q) and three products (the P T
// half of D2): 2^-16. The state adds one fresh accumulator per block in fp32:
// the tensor core never accumulates across blocks.
//
// Ten warps: eight compute (two per 32 lanes of tensor memory, sharing the
// columns), one moves (TMA loads of the next block, stores of o), one issues
// the matrix products. The chain of a block is D1k -> r -> D2 -> u -> D3 ->
// S; its links overlap by halves: the products over the first half of a
// thread's S, r or u start while it splits the second, and D3 is handed over
// in two halves of the key rows. The q product runs under r, o is finished
// under D3 and leaves under the next D1.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "sq_chunk_prepare.cuh"

namespace sqr {

constexpr int kScanCompute = 256;             // threads that own a part of the state
constexpr int kScanThreads = kScanCompute + 64;
constexpr int kScanStages = 2;
constexpr uint32_t kTileBytes = 64 * 128 * 2;  // q, k, v or o rows of a block
// A stage: channels 0..63 of the q rows, then of the k rows, the same for
// channels 64..127 (128-byte swizzled), the v rows, the prepared block.
constexpr uint32_t kStageV = 2 * kTileBytes, kStagePrep = 3 * kTileBytes;
constexpr uint32_t kStageBytes = kStagePrep + (kPrepBytes + 1023) / 1024 * 1024;
constexpr uint32_t kStageTx = kStagePrep + kPrepBytes;
constexpr uint32_t kOutAt = kScanStages * kStageBytes;  // o rows on their way out

struct ScanCtl {
  uint64_t full[kScanStages], empty[kScanStages];
  uint64_t s_ready[2], r_ready[2], u_ready[2], d3[2];
  uint64_t d1, d2, o_ready, o_free, drain;
  uint32_t tmem;
  int32_t abort;
};
constexpr size_t kScanSmem = 1024 + kOutAt + kTileBytes + sizeof(ScanCtl) + 16;

struct ScanArgs {
  PrepArgs p;
  uint64_t wait_ns;
};

// Columns of tensor memory (480 of 512).
constexpr uint32_t TM_S = 0;      // S^T terms hi and mid, over D3: 32 columns for each 32 key rows; lo from 128 on
constexpr uint32_t TM_RU = 192;   // r^T terms, then u^T terms
constexpr uint32_t TM_D1Q = 288;  // S^T q^T
constexpr uint32_t TM_D1K = 352;  // S^T k^T
constexpr uint32_t TM_D2 = 352;   // u^T (over S^T k^T), then the P T part of o, rows backwards

// Column of term s of S^T for key rows 16 ks .. 16 ks + 15.
__host__ __device__ constexpr uint32_t s_col(int s, int ks) {
  return s == 2 ? 128u + 8u * ks : 32u * (ks >> 1) + 16u * s + 8u * (ks & 1);
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
__device__ __forceinline__ void tc_ld32(uint32_t (&x)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SQ_R8(x, 0), SQ_R8(x, 8), SQ_R8(x, 16), SQ_R8(x, 24)
      : "r"(addr)
      : "memory");
}
// Waits for the loads; the values pass through it, so no use of them moves above.
#define SQ_RW8(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]), "+r"(x[i + 4]), "+r"(x[i + 5]), "+r"(x[i + 6]), "+r"(x[i + 7])
__device__ __forceinline__ void tc_wait_ld(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SQ_RW8(x, 0), SQ_RW8(x, 8), SQ_RW8(x, 16), SQ_RW8(x, 24)::"memory");
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const uint32_t (&x)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), SQ_W8(x, 0)
               : "memory");
}

// fp32 accumulators, bf16 operands, M = 128, N columns; `mn`: B has N contiguous.
__host__ __device__ constexpr uint32_t mma_desc(uint32_t N, bool mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}
// Shared memory operand: address, leading and stride offsets in bytes, swizzle mode (0 none, 2: 128 bytes).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride, uint64_t swizzle) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         (1ull << 46) | (swizzle << 61);
}

// 16 fp32 values of a lane (k index 0..15 of an A operand) to tensor memory as three terms.
__device__ __forceinline__ void put_terms(const float* x, uint32_t hi, uint32_t mid, uint32_t lo) {
  uint32_t t[kTerms][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t w[kTerms];
    split3(make_float2(x[2 * i], x[2 * i + 1]), w);
#pragma unroll
    for (int s = 0; s < kTerms; ++s) t[s][i] = w[s];
  }
  tc_st8(hi, t[0]);
  tc_st8(mid, t[1]);
  tc_st8(lo, t[2]);
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

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kScanCompute) : "memory"); }

template <bool PACKED>
__global__ void __launch_bounds__(kScanThreads, 1)
    k_chunk_scan(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap o_map,
                 const ScanArgs args) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ScanCtl& ctl = *reinterpret_cast<ScanCtl*>(smem + kOutAt + kTileBytes);
  const RaggedArgs& a = args.p.r;
  const int b = blockIdx.x / a.h_v, h = blockIdx.x - b * a.h_v, hk = h / (a.h_v / a.h_k);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int first, n;
  ragged_span(a, b, first, n);
  if (n < a.min_long) return;
  const int slot = a.slots ? a.slots[b] : b;
  const int blocks = (n + 63) >> 6, c0 = args.p.cu_blocks[b];
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o);
  if (slot < 0 || slot >= a.n_slots || c0 < 0 || c0 + blocks > args.p.n_blocks) {
    for (int x = tid; x < n * 16; x += kScanThreads)
      reinterpret_cast<uint4*>(out + ((size_t)(first + (x >> 4)) * a.h_v + h) * 128)[x & 15] = make_uint4(0, 0, 0, 0);
    if (tid == 0) atomicOr(a.t.status, ST_SLOT);
    return;
  }
  const bool resume = a.past && a.past[b] > 0;
  uint8_t* record = a.pool + (uint64_t)slot * a.slot_bytes + (PACKED ? a.t.rec_off[h] : 0u);
  float* S_pool = reinterpret_cast<float*>(a.pool) + ((size_t)slot * a.h_v + h) * 128 * 128;

  if (tid == 0) {
    constexpr uint32_t warps = kScanCompute / 32;
    for (int x = 0; x < 2; ++x) {
      sqk::mbar_init(&ctl.full[x], 1);
      sqk::mbar_init(&ctl.empty[x], warps);
      sqk::mbar_init(&ctl.s_ready[x], warps);
      sqk::mbar_init(&ctl.r_ready[x], warps);
      sqk::mbar_init(&ctl.u_ready[x], warps);
      sqk::mbar_init(&ctl.d3[x], 1);
    }
    sqk::mbar_init(&ctl.o_ready, warps);
    sqk::mbar_init(&ctl.o_free, 1);
    sqk::mbar_init(&ctl.d1, 1);
    sqk::mbar_init(&ctl.d2, 1);
    sqk::mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    sqk::fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sqk::smem_u32(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // S^T: value column of this thread's lane; S[y][j] is key row 64 y + 32 half + j
  const int half = warp >> 2, col = (warp & 3) * 32 + lane;  // compute warps
  float S[2][32];
  if (warp < 8) {
    const float* src = S_pool + (size_t)(32 * half) * 128 + col;
    if (PACKED && resume) {
      float* Ssh = reinterpret_cast<float*>(smem);
      unpack_state<128>(a, h, record, smem + 128 * 128 * 4, Ssh, compute_sync);
      src = Ssh + (32 * half) * 128 + col;
    }
#pragma unroll
    for (int x = 0; x < 64; ++x) S[x >> 5][x & 31] = resume ? src[(64 * (x >> 5) + (x & 31)) * 128] : 0.0f;
    if (PACKED && resume) sqk::fence_proxy_async_smem();  // before TMA writes where S was read
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = ctl.tmem;
  const uint64_t ns = args.wait_ns;
  uint32_t st = 0;

  if (warp == 8) {  // ------------------------------------- loads and stores
    if (lane == 0) {
      int issued = 0;
      auto load = [&](int i) {
        const int sg = i & 1;
        uint8_t* stage = smem + sg * kStageBytes;
        sqk::mbar_arrive_expect_tx(&ctl.full[sg], kStageTx);
        const int row = first + 64 * i;
        tma_tile(stage + kTileBytes / 2, &k_map, 0, hk, row, &ctl.full[sg]);
        tma_tile(stage + 3 * kTileBytes / 2, &k_map, 64, hk, row, &ctl.full[sg]);
        tma_tile(stage, &q_map, 0, hk, row, &ctl.full[sg]);
        tma_tile(stage + kTileBytes, &q_map, 64, hk, row, &ctl.full[sg]);
        tma_tile(stage + kStageV, &v_map, 0, h, row, &ctl.full[sg]);
        sqk::bulk_g2s(stage + kStagePrep, args.p.ws + ((uint64_t)(c0 + i) * a.h_v + h) * kPrepBytes, kPrepBytes,
                      &ctl.full[sg]);
        issued = i + 1;
      };
      load(0);
      if (blocks > 1) load(1);
      for (int i = 0; i < blocks; ++i) {
        // block i's stage is free when its D3 is done; its o follows
        if (i + kScanStages < blocks) {
          if (!sqk::mbar_wait_bounded(&ctl.empty[i & 1], (i >> 1) & 1, ns)) {
            ctl.abort = 1;
            break;
          }
          load(i + kScanStages);
        }
        if (!sqk::mbar_wait_bounded(&ctl.o_ready, i & 1, ns)) {
          ctl.abort = 1;
          break;
        }
        const int live = n - 64 * i;
        if (live >= 64) {
          tma_store(&o_map, 0, h, first + 64 * i, smem + kOutAt);
          sqk::bulk_commit();
          sqk::bulk_wait_read_all();
        } else {  // the last block: its live rows only
          for (int y = 0; y < live; ++y)
            sqk::bulk_s2g(out + ((size_t)(first + 64 * i + y) * a.h_v + h) * 128, smem + kOutAt + 256 * y, 256);
          sqk::bulk_commit();
        }
        sqk::mbar_arrive(&ctl.o_free);
      }
      // no copy is in flight when the CTA ends
      for (int i = max(0, issued - kScanStages); i < issued; ++i)
        sqk::mbar_wait_bounded(&ctl.full[i & 1], (i >> 1) & 1, ns);
      sqk::bulk_wait_all();
    }
  } else if (warp == 9) {  // ------------------------------------- products
    const uint32_t base = sqk::smem_u32(smem);
    for (int i = 0; i < blocks; ++i) {
      const uint32_t ph = i & 1;
      const uint32_t stage = base + (i & 1) * kStageBytes;
      const uint64_t qt = smem_desc(stage, 16, 1024, 2), kt = qt + kTileBytes / 32;
      if (!warp_wait(ctl, &ctl.full[i & 1], (i >> 1) & 1, ns)) break;
      bool ok = true;
#pragma unroll 1
      for (int y = 0; y < 2 && ok; ++y) {  // k: the key rows 64 y .. 64 y + 63
        ok = warp_wait(ctl, &ctl.s_ready[y], ph, ns);
        tc_after();
        if (ok && elect_one()) {
#pragma unroll
          for (int s = kTerms - 1; s >= 0; --s)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma(tm + TM_D1K, tm + TM_S + s_col(s, ks) + (s == 2 ? 32 : 64) * y, kt + y * kTileBytes / 16 + ks * 2,
                     mma_desc(64, false), s < kTerms - 1 || ks > 0 || y > 0);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) {
        tc_commit(&ctl.d1);
#pragma unroll
        for (int s = 1; s >= 0; --s)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc_mma(tm + TM_D1Q, tm + TM_S + s_col(s, ks), qt + ((ks >> 2) * kTileBytes + (ks & 3) * 32) / 16,
                   mma_desc(64, false), s < 1 || ks > 0);
      }
      __syncwarp();
      // rows 16 kk .. 63 of T and P T see columns 16 kk .. 16 kk + 15. Terms of r and of T: the six largest products
      // for T, the largest last; P T joins three of them, the first of which sets the accumulators
#pragma unroll 1
      for (int y = 0; y < 2 && ok; ++y) {  // kk = y and y + 2
        ok = warp_wait(ctl, &ctl.r_ready[y], ph, ns);
        tc_after();
        if (ok && elect_one()) {
          const uint64_t prep = smem_desc(stage + kStagePrep, 128, 256, 0);
          constexpr int pr[6] = {1, 2, 0, 1, 0, 0}, pt[6] = {0, 0, 2, 1, 1, 0};
#pragma unroll
          for (int x = 0; x < 6; ++x)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int kk = 2 * z + y;
              const uint64_t b = prep + (term_base(pt[x]) + (pt[x] == 2 ? tri_base(kk) : pair_base(kk))) / 16;
              tc_mma(tm + TM_D2 + 16 * kk, tm + TM_RU + 32 * pr[x] + 8 * kk, b,
                     mma_desc(x >= 1 && x <= 3 ? 64 - 16 * kk : 128 - 32 * kk, false), x > 0 || z > 0 || y > 0);
            }
          if (y == 1) tc_commit(&ctl.d2);
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int y = 0; y < 2 && ok; ++y) {  // rows 16 y .. + 15 and 16 (y + 2) .. + 15 of u and k
        ok = warp_wait(ctl, &ctl.u_ready[y], ph, ns);
        tc_after();
        if (ok && elect_one()) {
          const uint64_t km = smem_desc(stage + kTileBytes / 2, kTileBytes, 1024, 2) + y * 128;
#pragma unroll
          for (int x = 0; x < 2; ++x) {  // key rows 64 x .. 64 x + 63
#pragma unroll
            for (int s = kTerms - 1; s >= 0; --s)
#pragma unroll
              for (int z = 0; z < 2; ++z)
                tc_mma(tm + TM_S + 64 * x, tm + TM_RU + 32 * s + 16 * z + 8 * y, km + (x * kTileBytes + z * 4096) / 16,
                       mma_desc(64, true), s < kTerms - 1 || z > 0 || y > 0);
            if (y == 1) tc_commit(&ctl.d3[x]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    // no product is in flight when the tensor memory is given back
    if (elect_one()) tc_commit(&ctl.drain);
    __syncwarp();
    warp_wait(ctl, &ctl.drain, 0, ns);
  } else {  // -------------------------------------------------- the rest
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    auto put_state = [&](int y) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t hi = tl + TM_S + 64 * y + 32 * half + 8 * z;
        put_terms(S[y] + 16 * z, hi, hi + 16, tl + TM_S + 128 + 32 * y + 16 * half + 8 * z);
      }
      warp_arrive(&ctl.s_ready[y]);
    };
    put_state(0);
    put_state(1);
    for (int i = 0; i < blocks; ++i) {
      const int sg = i & 1;
      const uint32_t ph = i & 1;
      uint8_t* stage = smem + sg * kStageBytes;
      if (!warp_wait(ctl, &ctl.full[sg], (i >> 1) & 1, ns)) break;
      const int live = min(64, n - 64 * i);
      if (live < 64) {
        // rows of the k tile behind the request's last: another request's, or none's
        for (int x = tid; x < (64 - live) * 16; x += kScanCompute)
          *reinterpret_cast<uint4*>(stage + kTileBytes / 2 + ((x >> 3) & 1) * kTileBytes + (live + (x >> 4)) * 128 +
                                    (x & 7) * 16) = make_uint4(0, 0, 0, 0);
        sqk::fence_proxy_async_smem();
      }
      const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(stage + kStageV) + 32 * half * 128 + col;
      const float* coef = reinterpret_cast<const float*>(stage + kStagePrep + kTermsBytes);
      const float4* eg = reinterpret_cast<const float4*>(coef + 32 * half);
      const float4* eb = reinterpret_cast<const float4*>(coef + 64 + 32 * half);
      const float4* ebg = reinterpret_cast<const float4*>(coef + 128 + 32 * half);
      const float4* ed = reinterpret_cast<const float4*>(coef + 192 + 32 * half);
      const int mine = live - 32 * half;  // live rows of this half
      float x[32];
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 e = eb[j >> 2];
        x[j] = j < mine ? e.x * __bfloat162float(v[j * 128]) : 0.0f;
        x[j + 1] = j + 1 < mine ? e.y * __bfloat162float(v[(j + 1) * 128]) : 0.0f;
        x[j + 2] = j + 2 < mine ? e.z * __bfloat162float(v[(j + 2) * 128]) : 0.0f;
        x[j + 3] = j + 3 < mine ? e.w * __bfloat162float(v[(j + 3) * 128]) : 0.0f;
      }
      if (!warp_wait(ctl, &ctl.d1, ph, ns)) break;
      tc_after();
      tc_ld32(w, tl + TM_D1K + 32 * half);
      tc_wait_ld(w);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int j = 16 * y; j < 16 * y + 16; j += 4) {
          const float4 e = ebg[j >> 2];
          x[j] = j < mine ? fmaf(-e.x, __uint_as_float(w[j]), x[j]) : 0.0f;
          x[j + 1] = j + 1 < mine ? fmaf(-e.y, __uint_as_float(w[j + 1]), x[j + 1]) : 0.0f;
          x[j + 2] = j + 2 < mine ? fmaf(-e.z, __uint_as_float(w[j + 2]), x[j + 2]) : 0.0f;
          x[j + 3] = j + 3 < mine ? fmaf(-e.w, __uint_as_float(w[j + 3]), x[j + 3]) : 0.0f;
        }
        const uint32_t to = tl + TM_RU + 16 * half + 8 * y;
        put_terms(x + 16 * y, to, to + 32, to + 64);
        warp_arrive(&ctl.r_ready[y]);
      }

      if (!warp_wait(ctl, &ctl.d2, ph, ns)) break;
      tc_after();
      tc_ld32(w, tl + TM_D2 + 32 * half);
      tc_wait_ld(w);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int j = 16 * y; j < 16 * y + 16; j += 4) {
          const float4 e = ed[j >> 2];
          x[j] = e.x * __uint_as_float(w[j]);
          x[j + 1] = e.y * __uint_as_float(w[j + 1]);
          x[j + 2] = e.z * __uint_as_float(w[j + 2]);
          x[j + 3] = e.w * __uint_as_float(w[j + 3]);
        }
        const uint32_t to = tl + TM_RU + 16 * half + 8 * y;
        put_terms(x + 16 * y, to, to + 32, to + 64);
        warp_arrive(&ctl.u_ready[y]);
      }

      // o, under the state's product
      uint32_t o2[16];
      {
        uint32_t y[32];
        tc_ld32(w, tl + TM_D1Q + 32 * half);
        tc_ld32(y, tl + TM_D2 + 96 - 32 * half);
        tc_wait_ld(w);
        tc_wait_ld(y);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 e = eg[j >> 2];
          const float p0 = fmaf(e.x, __uint_as_float(w[j]), __uint_as_float(y[31 - j]));
          const float p1 = fmaf(e.y, __uint_as_float(w[j + 1]), __uint_as_float(y[30 - j]));
          const float p2 = fmaf(e.z, __uint_as_float(w[j + 2]), __uint_as_float(y[29 - j]));
          const float p3 = fmaf(e.w, __uint_as_float(w[j + 3]), __uint_as_float(y[28 - j]));
          o2[j >> 1] = bf16x2(p0, p1);
          o2[(j >> 1) + 1] = bf16x2(p2, p3);
        }
      }
      const float g63 = coef[256];
      bool ok = true;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        ok = ok && warp_wait(ctl, &ctl.d3[y], ph, ns);
        if (!ok) break;
        tc_after();
        if (y == 1 && lane == 0) sqk::mbar_arrive(&ctl.empty[sg]);  // this warp's reads of the stage came before
        tc_ld32(w, tl + TM_S + 64 * y + 32 * half);
        tc_wait_ld(w);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 t = __ffma2_rn(make_float2(g63, g63), make_float2(S[y][j], S[y][j + 1]),
                                      make_float2(__uint_as_float(w[j]), __uint_as_float(w[j + 1])));
          S[y][j] = t.x;
          S[y][j + 1] = t.y;
        }
        if (i + 1 < blocks) put_state(y);
      }
      if (!ok) break;
      // o's rows go out while the next block's first product runs
      if (i > 0 && !warp_wait(ctl, &ctl.o_free, (i - 1) & 1, ns)) break;
      uint16_t* op = reinterpret_cast<uint16_t*>(smem + kOutAt) + 32 * half * 128 + col;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const uint32_t t = o2[j >> 1];
        op[j * 128] = (uint16_t)t;
        op[(j + 1) * 128] = (uint16_t)(t >> 16);
        if (((t & 0x7fffu) > 0x7f80u && j < mine) || ((t & 0x7fffffffu) > 0x7f80ffffu && j + 1 < mine)) st |= ST_NAN;
      }
      sqk::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) sqk::mbar_arrive(&ctl.o_ready);
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  if (ctl.abort) {  // the state in the pool stays as it was
    if (tid == 0) atomicOr(a.t.status, sqk::ST_TIMEOUT);
    return;
  }
  if (warp < 8) {
    if (PACKED) {
      float* Ssh = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int x = 0; x < 64; ++x) Ssh[(64 * (x >> 5) + 32 * half + (x & 31)) * 128 + col] = S[x >> 5][x & 31];
      st |= pack_state<128>(a, h, record, smem + 128 * 128 * 4, Ssh, compute_sync);
    } else {
      float* dst = S_pool + (size_t)(32 * half) * 128 + col;
#pragma unroll
      for (int x = 0; x < 64; ++x) dst[(64 * (x >> 5) + (x & 31)) * 128] = S[x >> 5][x & 31];
    }
    if (st) atomicOr(a.t.status, st);
  }
}

}  // namespace sqr
