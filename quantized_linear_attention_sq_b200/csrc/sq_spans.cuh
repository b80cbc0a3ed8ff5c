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

}  // namespace sqr
