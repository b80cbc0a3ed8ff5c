// sq_ragged.cu -- host side of the ragged-batch operators declared in
// include/sq_ragged.h: argument checks, launch rules and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "sq.h"
#include "sq_chunk_prepare.cuh"
#include "sq_chunk_scan.cuh"
#include "sq_handle.h"
#include "sq_host.h"
#include "sq_qknorm.cuh"
#include "sq_ragged.h"
#include "sq_recurrent.cuh"
#include "sq_spans.cuh"
#include "sq_tables.cuh"

using sqi::cuda_fail;
using sqi::fail;

namespace {

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Most rows of a call: row numbers and their steps stay within 32 bits.
constexpr int32_t kMaxRows = 1 << 30;
inline int elt_bytes(int dtype) { return dtype == SQ_F32 ? 4 : 2; }

#define SQ_NEED(p, n)                                                                       \
  do {                                                                                      \
    if (!(p)) return fail(SQ_ERR_INVALID_ARG, #p " is NULL");                               \
    if (!aligned(p, n)) return fail(SQ_ERR_INVALID_ARG, #p " is not %d-byte aligned", (n)); \
  } while (0)

sq_status check_rows_of(const char* name, const void* p, int64_t stride, int64_t width, int bytes, int32_t rows) {
  if (!p) return fail(SQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 16)) return fail(SQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (stride < width && rows > 1)
    return fail(SQ_ERR_INVALID_ARG, "%s: row stride %lld is below a row's %lld elements", name, (long long)stride,
                (long long)width);
  if (stride * bytes % 16 != 0 && rows > 1)
    return fail(SQ_ERR_INVALID_ARG, "%s: row stride %lld is not a multiple of 16 bytes", name, (long long)stride);
  if (stride > ((int64_t)1 << 38)) return fail(SQ_ERR_INVALID_ARG, "%s: row stride too large", name);
  return SQ_OK;
}

// Allows a kernel all the shared memory of a CTA, once per device (`seen`: a
// bit for each device that has it).
template <typename K>
cudaError_t allow_smem(K kernel, int device, std::atomic<uint64_t>& seen) {
  const uint64_t bit = 1ull << (device & 63);
  if (device < 64 && (seen.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  int optin = 0;
  cudaFuncAttributes fa;
  cudaError_t e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - (int)fa.sharedSizeBytes);
  // all of the unified storage as shared memory, so that as many CTAs fit as the kernel is laid out for
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e == cudaSuccess) seen.fetch_or(bit, std::memory_order_release);
  return e;
}

// A launch that may overlap the end of the one before it on the stream (the
// kernel itself waits where it must).
template <typename... A>
cudaError_t launch(void (*kernel)(A...), bool overlap, int64_t grid, int threads, size_t smem, cudaStream_t st,
                   const A&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// ------------------------------------------------------------------- norms
template <int D, typename TI, typename TO>
void launch_norm(const sqr::NormArgs& a, int grid, cudaStream_t st) {
  sqr::k_qk_norm<D, TI, TO><<<grid, sqr::kNormThreads, 0, st>>>(a);
}
template <int D, typename TI>
void launch_norm_to(int out, const sqr::NormArgs& a, int grid, cudaStream_t st) {
  if (out == SQ_F32) launch_norm<D, TI, float>(a, grid, st);
  else if (out == SQ_BF16) launch_norm<D, TI, __nv_bfloat16>(a, grid, st);
  else launch_norm<D, TI, __half>(a, grid, st);
}
template <int D>
void launch_norm_from(int in, int out, const sqr::NormArgs& a, int grid, cudaStream_t st) {
  if (in == SQ_F32) launch_norm_to<D, float>(out, a, grid, st);
  else if (in == SQ_BF16) launch_norm_to<D, __nv_bfloat16>(out, a, grid, st);
  else launch_norm_to<D, __half>(out, a, grid, st);
}

// --------------------------------------------------------------- recurrent
struct RowsLaunch {
  int device, sms;
  cudaStream_t st;
};
template <int D, bool KDA, bool PACKED, typename T>
cudaError_t launch_rows(const sqr::RaggedArgs& a, const RowsLaunch& l) {
  static std::atomic<uint64_t> seen{0};
  auto kern = sqr::k_ragged_rows<D, KDA, PACKED, T>;
  const cudaError_t e = allow_smem(kern, l.device, seen);
  if (e != cudaSuccess) return e;
  const size_t smem = sqr::RGeo<D>::smem(PACKED, a.rec_cap);
  const int64_t tiles = (int64_t)a.B * a.h_v, most = 2ll * l.sms * (128 / D) * (128 / D);
  // beside blocks (min_long), the launch before is the blocks' preparation
  return launch(kern, a.min_long > 0, tiles < most ? tiles : most, sqr::RGeo<D>::NT, smem, l.st, a);
}
template <int D, bool KDA, typename T>
cudaError_t launch_rows_pool(const sqr::RaggedArgs& a, const RowsLaunch& l) {
  return a.fmt_fp32 ? launch_rows<D, KDA, false, T>(a, l) : launch_rows<D, KDA, true, T>(a, l);
}
template <int D, bool KDA>
cudaError_t launch_rows_type(int dtype, const sqr::RaggedArgs& a, const RowsLaunch& l) {
  if (dtype == SQ_F32) return launch_rows_pool<D, KDA, float>(a, l);
  if (dtype == SQ_BF16) return launch_rows_pool<D, KDA, __nv_bfloat16>(a, l);
  return launch_rows_pool<D, KDA, __half>(a, l);
}
template <int D>
cudaError_t launch_rows_gate(bool kda, int dtype, const sqr::RaggedArgs& a, const RowsLaunch& l) {
  return kda ? launch_rows_type<D, true>(dtype, a, l) : launch_rows_type<D, false>(dtype, a, l);
}

// ------------------------------------------------------------------ blocks
// Requests of at least this many rows run in blocks on the tensor cores,
// shorter ones row by row. Measured on 48 requests of 1..420 rows into 8-bit
// states and on 24 of 0..1900 (the whole call, us): from 6 rows 276, 182; from
// 10 rows 275, 180; from 16 rows 271, 190; from 24 rows 304, 212. Both have 32
// value heads and were measured with two terms for o's operands; with few
// heads, or with many requests of just over 10 rows, it was not measured.
constexpr int kMinLong = 10;

bool in_blocks(const sq_handle* h, int dtype, int32_t max_len) {
  return dtype == SQ_BF16 && h->desc.gate == SQ_GATE_HEAD && h->d == 128 && max_len >= kMinLong;
}

// Tensor map of a [rows, heads, 128] bf16 matrix: boxes of 64 rows and 64
// channels of one head, rows behind the last read as zeros.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}
sq_status row_map(CUtensorMap* m, const char* name, const void* p, int64_t stride, int heads, int32_t rows) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return fail(SQ_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  if (rows == 1) stride = (int64_t)heads * 128;  // never used, but must be valid
  const cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {256, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, 64}, one[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SQ_OK : fail(SQ_ERR_CUDA, "tensor map of %s: driver error %d", name, (int)r);
}

struct Blocks {
  sqr::ScanArgs a{};
  CUtensorMap q, k, v, o;
};

// Sets up the blocks' arguments and launches their preparation.
sq_status start_blocks(const sq_handle* h, const sqr::RaggedArgs& r, const sq_ragged_tables& t, void* workspace,
                       cudaStream_t st, Blocks& b) {
  b.a.p.r = r;
  b.a.p.cu_blocks = t.cu_blocks;
  b.a.p.block_req = t.block_req;
  b.a.p.ws = static_cast<uint8_t*>(workspace);
  b.a.p.n_blocks = (int32_t)sqr::most_blocks(r.rows, r.B);
  sq_status s = row_map(&b.q, "q", r.q, r.q_stride, r.h_k, r.rows);
  if (s == SQ_OK) s = row_map(&b.k, "k", r.k, r.k_stride, r.h_k, r.rows);
  if (s == SQ_OK) s = row_map(&b.v, "v", r.v, r.v_stride, r.h_v, r.rows);
  if (s == SQ_OK) s = row_map(&b.o, "o", r.o, (int64_t)r.h_v * 128, r.h_v, r.rows);
  if (s != SQ_OK) return s;
  static std::atomic<uint64_t> seen{0};
  cudaError_t e = allow_smem(sqr::k_chunk_prepare, h->device, seen);
  if (e == cudaSuccess)
    e = launch(sqr::k_chunk_prepare, false, (int64_t)b.a.p.n_blocks * r.h_k, sqr::kPrepThreads, sizeof(sqr::PrepSmem),
               st, b.a.p);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, "launching the blocks' preparation");
}

template <bool PACKED>
sq_status finish_blocks(const sq_handle* h, const Blocks& b, cudaStream_t st) {
  static std::atomic<uint64_t> seen{0};
  cudaError_t e = allow_smem(sqr::k_chunk_scan<PACKED>, h->device, seen);
  if (e == cudaSuccess)
    e = launch(sqr::k_chunk_scan<PACKED>, true, (int64_t)b.a.p.r.B * b.a.p.r.h_v, sqr::kScanThreads, sqr::kScanSmem, st,
               b.q, b.k, b.v, b.o, b.a);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, "launching the blocks' scan");
}

}  // namespace

extern "C" {

sq_status sq_batch_tables(const int32_t* lengths, const int32_t* past, int32_t B, int32_t max_rows,
                          int32_t* cu_seqlens, int32_t* cu_blocks, int32_t* positions, int32_t* block_req,
                          const int32_t* slot_ids, const uint8_t* used, int32_t n_slots, int32_t* slot_out,
                          uint8_t* used_out, uint32_t* status, void* stream) {
  sqi::g_last_error.clear();
  if (B < 0 || max_rows < 0 || n_slots < 0)
    return fail(SQ_ERR_INVALID_ARG, "B, max_rows and n_slots must be >= 0 (got %d, %d, %d)", B, max_rows, n_slots);
  if (B > SQ_RAGGED_MAX_REQUESTS)
    return fail(SQ_ERR_UNSUPPORTED, "B = %d is above %d requests", B, SQ_RAGGED_MAX_REQUESTS);
  if (max_rows > kMaxRows || n_slots > kMaxRows)
    return fail(SQ_ERR_UNSUPPORTED, "max_rows = %d or n_slots = %d is above %d", max_rows, n_slots, kMaxRows);
  SQ_NEED(cu_seqlens, 4);
  SQ_NEED(cu_blocks, 4);
  if (B > 0) {
    SQ_NEED(lengths, 4);
    SQ_NEED(block_req, 4);
  }
  if (!aligned(past, 4) || !aligned(positions, 4) || !aligned(status, 4))
    return fail(SQ_ERR_INVALID_ARG, "past, positions or status is not 4-byte aligned");
  const bool slots = slot_ids || used || slot_out || used_out || n_slots;
  if (slots) {
    if (B > 0) {
      SQ_NEED(slot_ids, 4);
      SQ_NEED(slot_out, 4);
    }
    if (n_slots > 0 && (!used || !used_out)) return fail(SQ_ERR_INVALID_ARG, "used or used_out is NULL");
  }
  sqr::TableArgs a{};
  a.lengths = lengths; a.past = past;
  a.cu_seqlens = cu_seqlens; a.cu_blocks = cu_blocks; a.positions = positions; a.block_req = block_req;
  a.slot_ids = slot_ids; a.used = used; a.slot_out = slot_out; a.used_out = used_out;
  a.status = status;
  a.B = B; a.max_rows = max_rows; a.n_slots = n_slots;
  // a CTA for every 2048 rows, up to 256 of them
  const int64_t want = ((int64_t)max_rows + 2047) / 2048;
  a.row_ctas = want < 1 ? 1 : want > 256 ? 256 : (int)want;
  sqr::k_batch_tables<<<a.row_ctas + (slots ? 1 : 0), sqr::kTabThreads, slots ? (size_t)B * 2 : 0, as_stream(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, "launching the batch tables");
}

sq_status sq_qk_norm(const sq_norm_desc* desc, const void* q, const void* k, int64_t q_row_stride,
                     int64_t k_row_stride, int32_t in, const float* q_weight, const float* k_weight,
                     const int32_t* positions, void* q_out, void* k_out, int32_t out, int32_t rows,
                     const int32_t* n_rows, int32_t h_q, int32_t h_k, int32_t d, void* stream) {
  sqi::g_last_error.clear();
  if (!desc) return fail(SQ_ERR_INVALID_ARG, "desc is NULL");
  if (desc->mode != SQ_NORM_L2 && desc->mode != SQ_NORM_RMS) return fail(SQ_ERR_INVALID_ARG, "bad mode %d", desc->mode);
  if (!(desc->eps >= 0.0f) || !std::isfinite(desc->eps))
    return fail(SQ_ERR_INVALID_ARG, "eps = %g is not finite >= 0", (double)desc->eps);
  if (!std::isfinite(desc->q_scale)) return fail(SQ_ERR_INVALID_ARG, "q_scale is not finite");
  if (in < SQ_F32 || in > SQ_F16 || out < SQ_F32 || out > SQ_F16)
    return fail(SQ_ERR_INVALID_ARG, "bad element type (in %d, out %d)", in, out);
  if (d != 32 && d != 64 && d != 128) return fail(SQ_ERR_UNSUPPORTED, "d must be 32, 64 or 128 (got %d)", d);
  if (rows < 0 || h_q < 0 || h_k < 0)
    return fail(SQ_ERR_INVALID_ARG, "rows, h_q and h_k must be >= 0 (got %d, %d, %d)", rows, h_q, h_k);
  if (rows > kMaxRows) return fail(SQ_ERR_UNSUPPORTED, "rows = %d is above %d", rows, kMaxRows);
  if ((int64_t)h_q + h_k > 65536) return fail(SQ_ERR_INVALID_ARG, "too many heads (%d + %d)", h_q, h_k);
  if (desc->rot_dim < 0 || desc->rot_dim > d || desc->rot_dim % 2 != 0)
    return fail(SQ_ERR_INVALID_ARG, "rot_dim = %d is not even in [0, %d]", desc->rot_dim, d);
  if (desc->rot_dim > 0 && (!(desc->base > 0.0) || !std::isfinite(desc->base)))
    return fail(SQ_ERR_INVALID_ARG, "base = %g is not finite > 0", desc->base);
  if (rows == 0 || h_q + h_k == 0) return SQ_OK;
  if (desc->rot_dim > 0) SQ_NEED(positions, 4);
  if (!aligned(n_rows, 4) || !aligned(q_weight, 4) || !aligned(k_weight, 4))
    return fail(SQ_ERR_INVALID_ARG, "n_rows or a weight is not 4-byte aligned");
  sq_status s = SQ_OK;
  if (h_q) {
    s = check_rows_of("q", q, q_row_stride, (int64_t)h_q * d, elt_bytes(in), rows);
    if (s != SQ_OK) return s;
    SQ_NEED(q_out, 16);
    if (q_out == q) return fail(SQ_ERR_INVALID_ARG, "q_out overlaps q");
  }
  if (h_k) {
    s = check_rows_of("k", k, k_row_stride, (int64_t)h_k * d, elt_bytes(in), rows);
    if (s != SQ_OK) return s;
    SQ_NEED(k_out, 16);
    if (k_out == k) return fail(SQ_ERR_INVALID_ARG, "k_out overlaps k");
  }
  sqr::NormArgs a{};
  a.x[0] = q; a.x[1] = k; a.y[0] = q_out; a.y[1] = k_out;
  a.w[0] = q_weight; a.w[1] = k_weight;
  a.stride[0] = q_row_stride; a.stride[1] = k_row_stride;
  a.heads[0] = h_q; a.heads[1] = h_k;
  a.scale[0] = desc->q_scale; a.scale[1] = 1.0f;
  a.positions = positions; a.n_rows = n_rows;
  a.rows = rows; a.rot = desc->rot_dim; a.inter = desc->interleaved != 0; a.rms = desc->mode == SQ_NORM_RMS;
  a.eps = desc->eps;
  for (int i = 0; i < desc->rot_dim / 2; ++i)
    a.turns[i] = std::pow(desc->base, -2.0 * i / desc->rot_dim) / (2.0 * 3.14159265358979323846);
  // as many rows per CTA as leave every SM two of them
  int per = sqr::kNormMaxRows;
  while (per > 1 && (rows + per - 1) / per < 2 * 148) per >>= 1;
  a.rows_per_cta = per;
  const int slots = sqr::kNormThreads * 8 / d;
  while ((1 << a.head_bits) < slots && (1 << a.head_bits) < h_q + h_k) a.head_bits++;
  const int groups = (rows + per - 1) / per, grid = groups < 4 * 148 ? groups : 4 * 148;  // four CTAs per SM
  cudaStream_t st = as_stream(stream);
  if (d == 128) launch_norm_from<128>(in, out, a, grid, st);
  else if (d == 64) launch_norm_from<64>(in, out, a, grid, st);
  else launch_norm_from<32>(in, out, a, grid, st);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, "launching the query and key norm");
}

sq_status sq_ragged_workspace_bytes(const sq_handle* h, int32_t dtype, int32_t B, int32_t rows, int32_t max_len,
                                    uint64_t* bytes) {
  sqi::g_last_error.clear();
  if (!h || !bytes) return fail(SQ_ERR_INVALID_ARG, "NULL argument");
  if (dtype < SQ_F32 || dtype > SQ_F16) return fail(SQ_ERR_INVALID_ARG, "bad element type %d", dtype);
  if (B < 0 || rows < 0 || max_len < 0)
    return fail(SQ_ERR_INVALID_ARG, "B, rows and max_len must be >= 0 (got %d, %d, %d)", B, rows, max_len);
  if (B > SQ_RAGGED_MAX_REQUESTS)
    return fail(SQ_ERR_UNSUPPORTED, "B = %d is above %d requests", B, SQ_RAGGED_MAX_REQUESTS);
  if (rows > kMaxRows) return fail(SQ_ERR_UNSUPPORTED, "rows = %d is above %d", rows, kMaxRows);
  *bytes = in_blocks(h, dtype, max_len)
               ? (uint64_t)sqr::most_blocks(rows, B) * (uint64_t)h->desc.h_v * sqr::kPrepBytes : 0;
  return SQ_OK;
}

sq_status sq_prefill_ragged(sq_handle* h, void* pool, const void* q, const void* k, const void* v, int64_t q_row_stride,
                            int64_t k_row_stride, int64_t v_row_stride, int32_t dtype, const float* beta,
                            const float* g, void* o, const sq_ragged_tables* tables, const int32_t* slot_ids, int32_t B,
                            int32_t rows, int32_t max_len, void* workspace, uint64_t workspace_bytes, void* stream) {
  sqi::g_last_error.clear();
  if (!h) return fail(SQ_ERR_INVALID_ARG, "NULL handle");
  uint64_t need = 0;
  sq_status s = sq_ragged_workspace_bytes(h, dtype, B, rows, max_len, &need);
  if (s != SQ_OK) return s;
  if ((int64_t)B * h->desc.h_v > (int64_t)INT32_MAX / 2) return fail(SQ_ERR_INVALID_ARG, "B too large");
  if (B == 0) return SQ_OK;
  SQ_NEED(pool, 16);
  if (!tables) return fail(SQ_ERR_INVALID_ARG, "tables is NULL");
  const int32_t *cu_seqlens = tables->cu_seqlens, *cu_blocks = tables->cu_blocks, *block_req = tables->block_req;
  SQ_NEED(cu_seqlens, 4);
  SQ_NEED(cu_blocks, 4);
  SQ_NEED(block_req, 4);
  if (!aligned(tables->past, 4) || !aligned(slot_ids, 4))
    return fail(SQ_ERR_INVALID_ARG, "past or slot_ids is not 4-byte aligned");
  const int d = h->d, eb = elt_bytes(dtype);
  const bool kda = h->desc.gate == SQ_GATE_KEY_CHANNEL;
  if (rows > 0) {
    s = check_rows_of("q", q, q_row_stride, (int64_t)h->desc.h_k * d, eb, rows);
    if (s == SQ_OK) s = check_rows_of("k", k, k_row_stride, (int64_t)h->desc.h_k * d, eb, rows);
    if (s == SQ_OK) s = check_rows_of("v", v, v_row_stride, (int64_t)h->desc.h_v * d, eb, rows);
    if (s != SQ_OK) return s;
    SQ_NEED(beta, 4);
    SQ_NEED(g, kda ? 16 : 4);
    SQ_NEED(o, 16);
  }
  if (workspace_bytes < need)
    return fail(SQ_ERR_INVALID_ARG, "workspace has %llu bytes, %llu are needed", (unsigned long long)workspace_bytes,
                (unsigned long long)need);
  if (need) SQ_NEED(workspace, 16);
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != h->device) return fail(SQ_ERR_INVALID_ARG, "device %d is current, the handle's is %d", dev, h->device);
  sqr::RaggedArgs a{};
  a.pool = static_cast<uint8_t*>(pool);
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_row_stride; a.k_stride = k_row_stride; a.v_stride = v_row_stride;
  a.beta = beta; a.g = g; a.o = o;
  a.cu_seqlens = cu_seqlens; a.past = tables->past; a.slots = slot_ids;
  a.B = B; a.rows = rows; a.h_v = h->desc.h_v; a.h_k = h->desc.h_k; a.n_slots = h->desc.n_slots;
  a.fmt_fp32 = h->desc.fmt == SQ_FMT_FP32;
  a.rec_cap = a.fmt_fp32 ? 0u : (uint32_t)h->max_rec;
  a.slot_bytes = h->slot_bytes;
  a.wait_ns = h->wait_ns;
  a.drain_ns = h->wait_ns > sqi::kWaitNs ? h->wait_ns : sqi::kWaitNs;  // a short limit is no limit for these
  a.test_extra_tx = h->test_extra_tx;
  a.t = h->tables;
  cudaStream_t st = as_stream(stream);
  const bool blocks = rows > 0 && in_blocks(h, dtype, max_len);
  Blocks bl;
  if (blocks) {
    if (sqr::most_blocks(rows, B) * h->desc.h_k > (int64_t)INT32_MAX)
      return fail(SQ_ERR_UNSUPPORTED, "too many blocks of rows");
    a.min_long = kMinLong;
    s = start_blocks(h, a, *tables, workspace, st, bl);
    if (s != SQ_OK) return s;
    h->launches++;
  }
  // the short requests run beside the preparation of the long ones
  const RowsLaunch l{h->device, h->num_sms, st};
  if (d == 128) e = launch_rows_gate<128>(kda, dtype, a, l);
  else if (d == 64) e = launch_rows_gate<64>(kda, dtype, a, l);
  else e = launch_rows_gate<32>(kda, dtype, a, l);
  if (e != cudaSuccess) return cuda_fail(e, "launching the ragged rows");
  h->launches++;
  if (blocks) {
    s = a.fmt_fp32 ? finish_blocks<false>(h, bl, st) : finish_blocks<true>(h, bl, st);
    if (s != SQ_OK) return s;
    h->launches++;
  }
  return SQ_OK;
}

}  // extern "C"
