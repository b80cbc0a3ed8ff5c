/*
 * sq_ragged.h -- C ABI of the ragged-batch operators that feed the state
 * pool of sq.h, B200 (sm_100a): a serving loop packs the rows (tokens) of
 * its requests one request after the other, without padding, and runs
 *   sq_batch_tables     offsets, blocks, positions and pool slots of the batch
 *   sq_qk_norm          norm of q and k per head, rotated by position
 *   sq_prefill_ragged   the gated delta rule over every request's rows,
 *                       from and into the requests' pool slots
 * before its decode steps (sq_decode_step).
 *
 * Conventions as in sq.h: calls are asynchronous on `stream`, bad arguments
 * are rejected on the host before any launch, sq_last_error() holds the
 * message, and bad data found on the device never traps: defined values are
 * written and a bit is set in a status word. Nothing here allocates. The
 * calls may be captured into CUDA graphs.
 */
#ifndef SQ_RAGGED_H
#define SQ_RAGGED_H

#include <stdint.h>

#include "sq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of activations. */
typedef enum { SQ_F32 = 0, SQ_BF16 = 1, SQ_F16 = 2 } sq_dtype;

/* Rows of one block of the block tables. */
#define SQ_RAGGED_BLOCK 64

/* Most requests of one ragged batch (and at most 2^30 rows or slots):
 * SQ_ERR_UNSUPPORTED beyond. */
#define SQ_RAGGED_MAX_REQUESTS 16384

/* Further bits of the status word. */
#define SQ_STATUS_TRUNCATED 32u /* sq_batch_tables: the lengths add up to more than max_rows; the rows past it were cut */
#define SQ_STATUS_NO_SLOT 64u   /* sq_batch_tables: fewer free slots than requests that need one; theirs are -1 */

/* Tables of a ragged batch from its lengths, in one launch. With
 * n_b = max(lengths[b], 0), and everything cut at max_rows rows:
 *   cu_seqlens [B + 1]  first row of request b: min(sum of n_a over a < b, max_rows)
 *   cu_blocks  [B + 1]  first block of request b: sum over a < b of
 *                       ceil(rows of request a / SQ_RAGGED_BLOCK)
 *   positions  [max_rows]  position of row r of request b in its sequence:
 *                       r - cu_seqlens[b] + past[b]
 *   block_req  [max_rows / SQ_RAGGED_BLOCK + B]  request of each block
 * Rows and blocks behind the last request's are left as they were.
 * Slots: every request with slot_ids[b] < 0 takes a free slot of the pool,
 * in order (the r-th such request takes the r-th slot whose `used` flag is
 * zero); slot_out is slot_ids with those filled in (-1 where no slot was
 * left), used_out is `used` with the taken slots set to 1. slot_out may be
 * slot_ids and used_out may be used (in place); other outputs must not
 * overlap each other or an input.
 *   lengths  device int32 [B]
 *   past     device int32 [B], rows a request's state has already seen, or NULL for 0
 *   cu_seqlens, cu_blocks, positions, block_req  device int32; positions may be NULL
 *   slot_ids, slot_out  device int32 [B], used, used_out  device uint8
 *            [n_slots]: all four, or all NULL with n_slots = 0
 *   status   device uint32 the SQ_STATUS_* bits are ORed into, or NULL
 * B == 0 writes cu_seqlens[0] = cu_blocks[0] = 0. B may be at most
 * SQ_RAGGED_MAX_REQUESTS (SQ_ERR_UNSUPPORTED beyond). */
sq_status sq_batch_tables(const int32_t* lengths, const int32_t* past, int32_t B, int32_t max_rows,
                          int32_t* cu_seqlens, int32_t* cu_blocks, int32_t* positions, int32_t* block_req,
                          const int32_t* slot_ids, const uint8_t* used, int32_t n_slots, int32_t* slot_out,
                          uint8_t* used_out, uint32_t* status, void* stream);

typedef enum { SQ_NORM_L2 = 0, SQ_NORM_RMS = 1 } sq_norm_mode;

/* What sq_qk_norm does to each head of a row. */
typedef struct {
  int32_t mode;          /* sq_norm_mode */
  float eps;             /* finite, >= 0 */
  float q_scale;         /* factor of q after its norm (and weight) */
  int32_t rot_dim;       /* leading channels that are rotated: even, 0 .. d (0: none) */
  int32_t interleaved;   /* pairs (2i, 2i + 1), else (i, i + rot_dim / 2) */
  double base;           /* > 0: pair i turns by position * base^(-2 i / rot_dim) */
} sq_norm_desc;

/* Norm of queries and keys for each head, and their rotation by position, in
 * one pass. For every row r and head, over its d channels,
 *     y = x / sqrt(sum x^2 + eps)      (SQ_NORM_L2)
 *     y = x / sqrt(mean x^2 + eps)     (SQ_NORM_RMS)
 * times the weight of the channel (where given), times q_scale for q, then
 * the first rot_dim channels turned by positions[r]. Sums are fp32; the
 * angle is formed in fp64, so far positions keep their precision; the result
 * is rounded once to the output type.
 *   q, k     device, element type `in`; row r, head h starts at element
 *            r * row_stride + h * d (rows of a wider matrix are fine); 16-byte
 *            aligned, row strides a multiple of 16 bytes and at least h * d
 *   q_weight, k_weight  device fp32 [d], or NULL for 1
 *   positions  device int32 [rows], needed where rot_dim > 0
 *   q_out, k_out  device, element type `out`, contiguous [rows, h, d],
 *            16-byte aligned; must not overlap the inputs
 *   n_rows   device int32: only rows below it are computed, the others are
 *            left as they were (for instance &cu_seqlens[B]), or NULL for all
 * h_q or h_k may be 0 (its pointers are then ignored). d in {32, 64, 128}. */
sq_status sq_qk_norm(const sq_norm_desc* desc, const void* q, const void* k, int64_t q_row_stride,
                     int64_t k_row_stride, int32_t in, const float* q_weight, const float* k_weight,
                     const int32_t* positions, void* q_out, void* k_out, int32_t out, int32_t rows,
                     const int32_t* n_rows, int32_t h_q, int32_t h_k, int32_t d, void* stream);

/* Tables of a ragged batch as sq_batch_tables writes them (device pointers). */
typedef struct {
  const int32_t* cu_seqlens;  /* [B + 1] */
  const int32_t* cu_blocks;   /* [B + 1] */
  const int32_t* block_req;   /* [rows / SQ_RAGGED_BLOCK + B] */
  const int32_t* past;        /* [B], or NULL for 0 */
} sq_ragged_tables;

/* The gated delta rule over a ragged batch ("STEPQuant review (e-cogni)",
 * "Contexto"): request b's rows cu_seqlens[b] .. cu_seqlens[b+1] - 1, in
 * order, from its state:
 *     S <- diag(g) S ;  u = beta (v - S^T k) ;  S <- S + k u^T ;  o = S^T q
 * A request with past[b] > 0 goes on from the state in its pool slot
 * (dequantized for packed pools), one with past[b] <= 0 from zeros; the
 * state after its last row is stored in the slot once (quantized as
 * sq_quantize_state does). A request without rows keeps its slot's state if
 * past[b] > 0 and stores zeros otherwise.
 *   q, k     device, type `dtype`, row r, key head h at r * row_stride + h * d
 *   v        device, type `dtype`, row r, value head h at r * v_row_stride + h * d
 *            (all 16-byte aligned, row strides a multiple of 16 bytes)
 *   beta     device fp32 [rows, h_v]
 *   g        device fp32 [rows, h_v] (SQ_GATE_HEAD) or [rows, h_v, d]
 *            (SQ_GATE_KEY_CHANNEL, then 16-byte aligned), in [0, 1]; values
 *            outside are taken as the nearer bound
 *   o        device, type `dtype`, contiguous [rows, h_v, d]; rows of no
 *            request are left as they were; must not overlap an input
 *   slot_ids device int32 [B] (distinct), or NULL for slots 0..B-1; a
 *            request whose slot is out of range, or whose first block (where
 *            it runs in blocks) no table of these sizes can hold, gets o = 0
 *            and SQ_STATUS_BAD_SLOT, and no state
 *   rows     rows of q, k, v, beta, g and o; table entries are cut to it
 *   max_len  the longest request's rows as far as the host knows (rows if it
 *            does not): it chooses the kernels, longer requests stay correct
 *   workspace  device, 16-byte aligned, sq_ragged_workspace_bytes() bytes,
 *            used by this call's kernels only while they run: calls that may
 *            overlap (two streams, two graphs in flight) need one each
 * SQ_BF16 requests of SQ_GATE_HEAD pools with d = 128 that are not very short
 * run in blocks of 64 rows on the tensor cores: the state, and o before it is
 * rounded, stay accurate to fp32 (operands are split into three bf16 terms),
 * so they differ from a row by row run in their last bits only. All others
 * run row by row in fp32. A NaN or an infinity in a row reaches the state and
 * o from its block of 64 rows on, and no other request.
 * A wait that runs out (sq_set_wait_limit) sets SQ_STATUS_TIMEOUT: the CTA
 * leaves once its copies under way have landed. The state of the (request,
 * value head) it was at keeps its slot's bytes; row by row its o is untouched
 * and the further (request, value head)s of that CTA are left out the same
 * way, in blocks o of blocks before the wait is already written. */
sq_status sq_prefill_ragged(sq_handle* h, void* pool, const void* q, const void* k, const void* v, int64_t q_row_stride,
                            int64_t k_row_stride, int64_t v_row_stride, int32_t dtype, const float* beta,
                            const float* g, void* o, const sq_ragged_tables* tables, const int32_t* slot_ids, int32_t B,
                            int32_t rows, int32_t max_len, void* workspace, uint64_t workspace_bytes, void* stream);

/* Bytes of workspace sq_prefill_ragged needs for these sizes (0 where it
 * needs none: workspace may then be NULL). Where max_len lets requests run in
 * blocks it is 31760 bytes for each of rows / 64 + B blocks and each value
 * head, whether the blocks are used or not: with 32 value heads 1.1 GB for 32
 * requests of 2048 rows, 4.2 GB for one of 262144, and 0.5 GB for 512 requests
 * of one row if max_len does not say that they are short (it is 0 if it does).
 * B may be at most SQ_RAGGED_MAX_REQUESTS (SQ_ERR_UNSUPPORTED beyond). Host only. */
sq_status sq_ragged_workspace_bytes(const sq_handle* h, int32_t dtype, int32_t B, int32_t rows, int32_t max_len,
                                    uint64_t* bytes);

#ifdef __cplusplus
}
#endif
#endif /* SQ_RAGGED_H */
