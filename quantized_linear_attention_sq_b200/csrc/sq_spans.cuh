// sq_spans.cuh -- index arithmetic of ragged batches whose products or sums pass
// 32 bits at the largest sizes (2^30 rows), for host and device.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SQ_HD __host__ __device__ __forceinline__
#else
#define SQ_HD inline
#endif

namespace sqr {

// 16-byte pieces of n rows of 128 16-bit elements.
SQ_HD int64_t row_pieces(int32_t n) { return (int64_t)n * 16; }

// Most blocks of 64 rows that B requests with `rows` rows in all can have.
SQ_HD int64_t most_blocks(int32_t rows, int32_t B) { return (int64_t)(rows / 64) + B; }

// The `blocks` records from c0 on lie among n_blocks of them; c0 is what a
// table holds, any number.
SQ_HD bool blocks_within(int32_t c0, int32_t blocks, int32_t n_blocks) { return c0 >= 0 && blocks <= n_blocks - c0; }
// Number of block c among those from c0 on, negative where it is not one.
SQ_HD int32_t block_after(int32_t c, int32_t c0) { return c0 < 0 || c0 > c ? -1 : c - c0; }

}  // namespace sqr
