// sq_tables.cuh -- offsets, blocks, positions and pool slots of a ragged
// batch from its lengths (sq_batch_tables).
//
// One launch, no exchange between CTAs: every CTA walks the lengths in tiles
// of 1024 requests with a running prefix and writes the part of the outputs
// that is its own, so a CTA needs nothing from another one. The lengths are
// read once per CTA from L2 (at most 64 KB); the outputs are written once.
// One more CTA hands out the slots. Latency: 5.0 us for 512 requests and 2561
// slots, 7.4 us for 1000 requests and 262144 rows.
#pragma once

#include "sq_kernels.cuh"

namespace sqr {

constexpr int kTabThreads = 256;
constexpr int kTabPer = 4;                        // requests per thread and tile
constexpr int kTabTile = kTabThreads * kTabPer;   // requests per tile
constexpr uint32_t ST_TRUNCATED = 32u;
constexpr uint32_t ST_NO_SLOT = 64u;
constexpr int kBlock = 64;                        // rows of one block

struct TableArgs {
  const int32_t* lengths;   // [B]
  const int32_t* past;      // [B] or null
  int32_t* cu_seqlens;      // [B + 1]
  int32_t* cu_blocks;       // [B + 1]
  int32_t* positions;       // [max_rows] or null
  int32_t* block_req;       // [max_rows / 64 + B]
  const int32_t* slot_ids;  // [B] or null
  const uint8_t* used;      // [n_slots]
  int32_t* slot_out;        // [B]
  uint8_t* used_out;        // [n_slots]
  uint32_t* status;         // or null
  int32_t B, max_rows, n_slots, row_ctas;
};

// Exclusive prefix of x over the CTA, and the total. `tmp`: one value per warp.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* tmp, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();  // tmp of the previous scan has been read
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w < warp) before += tmp[w];
    total += tmp[w];
  }
  return before + s - x;
}

// Last index i of [0, n) with first[i] <= x (first is non-decreasing, first[0] <= x).
__device__ __forceinline__ int last_not_above(const int32_t* first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The r-th request that needs a slot takes the r-th free one: the requests'
// numbers go to a list in shared memory in order, then the flags are scanned
// in order and each free slot looks up the request of its rank.
__device__ __forceinline__ void assign_slots(const TableArgs& a, uint16_t* list, int64_t* tmp) {
  int64_t need = 0, total;
  for (int b0 = 0; b0 < a.B; b0 += kTabThreads) {
    const int b = b0 + threadIdx.x;
    const int32_t s = b < a.B ? a.slot_ids[b] : 0;
    const int64_t r = need + block_scan(s < 0 ? 1 : 0, tmp, total);
    if (b < a.B) {
      if (s < 0) list[r] = (uint16_t)b;
      a.slot_out[b] = s < 0 ? -1 : s;
    }
    need += total;
  }
  int64_t given = 0;
  constexpr int PER = 16;
  for (int s0 = 0; s0 < a.n_slots; s0 += kTabThreads * PER) {
    const int s = s0 + threadIdx.x * PER;
    alignas(16) uint8_t f[PER];
    int free_here = 0;
    if (s + PER <= a.n_slots && (reinterpret_cast<uintptr_t>(a.used) & 15u) == 0) {
      *reinterpret_cast<uint4*>(f) = *reinterpret_cast<const uint4*>(a.used + s);
    } else {
#pragma unroll
      for (int x = 0; x < PER; ++x) f[x] = s + x < a.n_slots ? a.used[s + x] : 1;
    }
#pragma unroll
    for (int x = 0; x < PER; ++x) free_here += f[x] == 0;
    int64_t r = given + block_scan(free_here, tmp, total);  // its barriers also order the list before its reads
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      if (s + x < a.n_slots) {
        if (f[x] == 0) {
          if (r < need) {
            a.slot_out[list[r]] = s + x;
            f[x] = 1;
          }
          ++r;
        }
        a.used_out[s + x] = f[x];
      }
    }
    given += total;
  }
  if (given < need && threadIdx.x == 0 && a.status) atomicOr(a.status, ST_NO_SLOT);
}

__global__ void __launch_bounds__(kTabThreads) k_batch_tables(const TableArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];  // the slot CTA's list
  __shared__ int64_t tmp[kTabThreads / 32];
  __shared__ int32_t row0[kTabTile + 1], blk0[kTabTile + 1], shift[kTabTile];
  if ((int)blockIdx.x == a.row_ctas) {
    assign_slots(a, reinterpret_cast<uint16_t*>(dyn), tmp);
    return;
  }
  // this CTA's share of the rows and of the blocks (int64: row_ctas * rows may pass 2^31)
  const int64_t n_blk = (int64_t)a.max_rows / kBlock + a.B;
  const int64_t me = blockIdx.x, ctas = a.row_ctas;
  const int r_lo = (int)(a.max_rows * me / ctas), r_hi = (int)(a.max_rows * (me + 1) / ctas);
  const int k_lo = (int)(n_blk * me / ctas), k_hi = (int)(n_blk * (me + 1) / ctas);
  int64_t rows = 0, blocks = 0;  // before this tile, not cut
  if (me == 0 && threadIdx.x == 0) a.cu_seqlens[0] = a.cu_blocks[0] = 0;
  for (int b0 = 0, tile = 0; b0 < a.B; b0 += kTabTile, ++tile) {
    const int n = min(kTabTile, a.B - b0);
    const int at = threadIdx.x * kTabPer;
    int64_t len[kTabPer], sum = 0, total;
#pragma unroll
    for (int x = 0; x < kTabPer; ++x) {
      len[x] = at + x < n ? (int64_t)max(a.lengths[b0 + at + x], 0) : 0;
      sum += len[x];
    }
    int64_t first = rows + block_scan(sum, tmp, total);
    rows += total;
    int32_t cut[kTabPer];
    sum = 0;
    __syncthreads();  // the previous tile's tables have been read
#pragma unroll
    for (int x = 0; x < kTabPer; ++x) {
      const int32_t lo = (int32_t)min(first, (int64_t)a.max_rows);
      first += len[x];
      cut[x] = (int32_t)min(first, (int64_t)a.max_rows) - lo;
      row0[at + x] = lo;
      if (at + x < n) shift[at + x] = (a.past ? a.past[b0 + at + x] : 0) - lo;
      sum += (cut[x] + kBlock - 1) / kBlock;
    }
    int64_t kfirst = blocks + block_scan(sum, tmp, total);
    blocks += total;
#pragma unroll
    for (int x = 0; x < kTabPer; ++x) {
      blk0[at + x] = (int32_t)kfirst;
      kfirst += (cut[x] + kBlock - 1) / kBlock;
    }
    const int32_t row_end = (int32_t)min(rows, (int64_t)a.max_rows), blk_end = (int32_t)blocks;
    __syncthreads();
    if (tile % a.row_ctas == (int)me) {
      for (int x = threadIdx.x; x < n; x += kTabThreads) {
        a.cu_seqlens[b0 + x + 1] = x + 1 < n ? row0[x + 1] : row_end;
        a.cu_blocks[b0 + x + 1] = x + 1 < n ? blk0[x + 1] : blk_end;
      }
    }
    if (a.positions) {
      const int hi = min(r_hi, row_end);
      for (int r = max(r_lo, row0[0]) + threadIdx.x; r < hi; r += kTabThreads)
        a.positions[r] = r + shift[last_not_above(row0, n, r)];
    }
    const int hi = min(k_hi, blk_end);
    for (int k = max(k_lo, blk0[0]) + threadIdx.x; k < hi; k += kTabThreads)
      a.block_req[k] = b0 + last_not_above(blk0, n, k);
  }
  if (me == 0 && threadIdx.x == 0 && rows > a.max_rows && a.status) atomicOr(a.status, ST_TRUNCATED);
}

}  // namespace sqr
