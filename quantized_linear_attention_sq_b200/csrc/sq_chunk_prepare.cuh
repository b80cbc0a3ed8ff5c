// sq_chunk_prepare.cuh -- the gated delta rule in blocks of 64 rows, first
// kernel: everything of a block that does not depend on the state.
//
// With G_i the sum of log gates of the block's rows 0..i, S the state before
// the block, and for i > j (i >= j for P)
//     A_ij = beta_i e^(G_i - G_j) k_i . k_j,   P_ij = e^(G_i - G_j) q_i . k_j,
// the rows' updates u solve (1 + A) u = r, so with T = (1 + A)^-1
//     u = T r,   r_j = beta_j (v_j - e^(G_j) k_j S),   o = e^G q S + (P T) r,
//     S <- e^(G_63) S + sum_i e^(G_63 - G_i) k_i u_i^T.
// This kernel forms T and P T of every block and value head, in parallel over
// blocks, for sq_chunk_scan.cuh, which walks a request's blocks in order.
// q, k are bf16: their products are exact, accumulated in fp32 by the tensor
// cores, and stay in registers for the value heads that share them. Logs of
// gates are summed as pairs of fp32: a difference G_i - G_j keeps its
// precision behind a gate of zero. Decays are products of factors that are
// all at most one (token to the end of its 16, from the start of its 16,
// between 16s; inside a 16 the quotient of two of them), so a block needs a
// few hundred exponentials, not one for each pair. The inverse goes by blocks
// of 16: those on the diagonal by substitution in fp32, then pairs of blocks,
// [T1 0; -T2 A21 T1, T2], to 32 and to 64 on the tensor cores, every operand
// as three bf16 terms whose sum is the fp32 value (the six largest of nine
// products: fp32 accuracy). T and P T leave as such terms: o may be a small
// difference of large sums (an old value overwritten by a smaller one), so what
// reaches it is held like the state's. Only the blocks on and below the diagonal
// are stored, in the order the scan's matrix instructions read them.
// Bound by latency: a value head is a chain of six short phases with a
// barrier between them, and five CTAs per SM run theirs against each other: 534
// us for 32 requests of 2048 rows with 32 value heads (485 us with two terms for
// P T; from 594 to 521 when five fitted an SM). In 24 requests of 0..1900 rows a
// scheduler issues 0.46 instructions a cycle.
#pragma once

#include <cuda_bf16.h>

#include "sq_recurrent.cuh"
#include "sq_spans.cuh"

namespace sqr {

constexpr int kTerms = 3;                                    // bf16 terms of an fp32 operand
constexpr int kTriBytes = 32 * (64 + 48 + 32 + 16);          // one term of one matrix
constexpr int kTermsBytes = kTerms * 2 * kTriBytes;
constexpr int kCoefFloats = 4 * 64 + 4;                      // e^G, beta, beta e^G, e^(G_63 - G), e^(G_63)
constexpr int kPrepBytes = kTermsBytes + 4 * kCoefFloats;    // per block and value head
static_assert(kPrepBytes % 16 == 0, "bulk copies move 16-byte multiples");

// A term holds T and P T: for each 16 columns kk = j / 16, the operand
// rows that are not all zero there, rows 16 kk .. 63 of T, then the same rows
// of P T. Rows come in groups of 8 x 16 columns, a group as two 8 x 8 pieces
// of 128 contiguous bytes (the tensor core's unswizzled layout).
__host__ __device__ constexpr int term_base(int s) { return s * 2 * kTriBytes; }
__host__ __device__ constexpr int pair_base(int kk) { return kk * 4096 - kk * (kk - 1) * 512; }  // within a term
__device__ __forceinline__ int row_piece(int li, int j) {
  return (li >> 3) * 256 + ((j >> 3) & 1) * 128 + (li & 7) * 16 + (j & 7) * 2;
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
  const int blocks = a.cu_blocks[a.r.B], b = a.block_req[c];  // two loads at once, then three
  if (c >= blocks || b < 0 || b >= a.r.B) return false;
  const int at = block_after(c, a.cu_blocks[b]);
  int r0, len;
  ragged_span(a.r, b, r0, len);
  if (len < a.r.min_long || at < 0 || at >= (len + 63) / 64) return false;
  first = r0 + 64 * at;
  n = min(64, len - 64 * at);
  return true;
}

// x = hi + mid + lo, each a bf16 rounded to nearest: an fp32 value's 24
// significant bits are three times 8. Two values at a time, packed as (a: low
// half, b: high half). The remainders are fused multiply-adds with a bf16
// operand as it is: 7 instructions, where cutting and packing takes 11.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t take_bf16x2(float& a, float& b) {  // leaves the remainders
  const uint32_t t = bf16x2(a, b);
  asm("{\n\t.reg .b16 l, h, m;\n\tmov.b16 m, 0xBF80;\n\tmov.b32 {l, h}, %2;\n\t"
      "fma.rn.f32.bf16 %0, l, m, %0;\n\tfma.rn.f32.bf16 %1, h, m, %1;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(t));
  return t;
}
__device__ __forceinline__ void split3(float a, float b, uint32_t (&t)[kTerms]) {
  t[0] = take_bf16x2(a, b);
  t[1] = take_bf16x2(a, b);
  t[2] = bf16x2(a, b);
}

constexpr int kPrepThreads = 128;
constexpr int kTile = 136;   // bf16 per row of the q and k tiles (16 bytes of padding)
constexpr int kBlk = 512;    // bytes of one 16 x 16 bf16 block

// 16 bytes (columns 8 half .. + 7) of row r of such a block: swapped in every
// other four rows, so that the eight rows of a matrix load lie in different banks.
__device__ __forceinline__ int blk_piece(int r, int half) { return r * 32 + ((half ^ ((r >> 2) & 1)) << 4); }

// Factors of the rows of one value head; R_b is G at the end of 16 number b.
struct PrepGate {
  float2 G[64];      // log2, high and low part
  float beta[64];
  float from[64];    // e^(G_i - R_(b-1))  from its 16's start
  float to[64];      // e^(R_b - G_j)      to its 16's end
  float inv[64];     // 1 / from
  float hop[4][4];   // e^(R_(bi-1) - R_bj), bj < bi
  int32_t steep[4];  // the 16's decay is below 2^-100: its inverses may overflow, its pairs are formed one by one
};
constexpr int kAd = 20;      // floats per row of a block of A on the diagonal
static_assert(16 * kAd * 4 <= kTerms * kBlk, "one fits where a block of T will be");
struct PrepSmem {
  union {
    __nv_bfloat16 qk[2][64 * kTile];
    struct {
      uint8_t A[6][kTerms][kBlk];       // blocks below the diagonal
      uint8_t P[10][kTerms][kBlk];      // blocks on and below it
      uint8_t T[10][kTerms][kBlk];
    } m;
  };
  // A's blocks on the diagonal, 16 rows of kAd floats each: where the last row
  // of T's blocks (number 3: the one at (2, 0)) is written once they have been read
  __device__ __forceinline__ float* Ad(int b) { return reinterpret_cast<float*>(m.T[b < 3 ? 6 + b : 3][0]); }
  PrepGate gate[2];  // two value heads at a time
  float2 part[4];    // log gates summed by each warp
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sqk::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sqk::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A 16 x 16 fp32 block in the instruction's result layout: lane owns rows
// lane / 4 (elements 0, 1) and + 8 (2, 3), columns 8 x + 2 (lane % 4), + 1.
struct Acc {
  float c[2][4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int y = 0; y < 4; ++y) c[0][y] = c[1][y] = 0.0f;
  }
  __device__ __forceinline__ void add(const uint32_t (&a)[4], const uint32_t (&b)[4]) {  // += A B, b read transposed
    mma_bf16(c[0], a, b[0], b[1]);
    mma_bf16(c[1], a, b[2], b[3]);
  }
};
using Terms = uint32_t[kTerms][4];
__device__ __forceinline__ void add6(Acc& acc, const Terms& a, const Terms& b) {  // smallest products first
  acc.add(a[2], b[0]);
  acc.add(a[0], b[2]);
  acc.add(a[1], b[1]);
  acc.add(a[1], b[0]);
  acc.add(a[0], b[1]);
  acc.add(a[0], b[0]);
}
// The result layout is the left operand's.
__device__ __forceinline__ void acc_terms(const Acc& acc, Terms& t) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint32_t w[kTerms];
    split3(acc.c[x >> 1][2 * (x & 1)], acc.c[x >> 1][2 * (x & 1) + 1], w);
#pragma unroll
    for (int s = 0; s < kTerms; ++s) t[s][x] = w[s];
  }
}
// A left operand's registers to a block: `block` is at this lane's place in it
// (row lane / 4, columns 2 (lane % 4)), `turn` (16 or -16) leads to columns + 8.
__device__ __forceinline__ void put_left(uint8_t* block, int turn, const uint32_t (&t)[4]) {
  *reinterpret_cast<uint32_t*>(block) = t[0];
  *reinterpret_cast<uint32_t*>(block + 256) = t[1];
  *reinterpret_cast<uint32_t*>(block + turn) = t[2];
  *reinterpret_cast<uint32_t*>(block + turn + 256) = t[3];
}

// Number of a block on or below the diagonal, and of one below it.
__device__ __forceinline__ int tri(int bi, int bj) { return bi * (bi + 1) / 2 + bj; }
__device__ __forceinline__ int below(int bi, int bj) { return bi * (bi - 1) / 2 + bj; }

// 2^x to 2 ulp, 0 for results below 2^-126.
__device__ __forceinline__ float pow2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// a + b as an unevaluated pair (the rounding error of the high parts is kept).
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
  const float s = __fadd_rn(a.x, b.x), t = __fsub_rn(s, a.x);
  const float e = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t));
  return make_float2(s, __fadd_rn(e, __fadd_rn(a.y, b.y)));
}
__device__ __forceinline__ float pair_diff(float2 a, float2 b) {
  return __fadd_rn(__fsub_rn(a.x, b.x), __fsub_rn(a.y, b.y));
}

// Gates and betas of value heads h and h + 1 (`heads` of them), a thread for
// each row of each.
__device__ __forceinline__ float2 load_gates(const PrepArgs& a, int first, int n, int h, int heads) {
  const int which = threadIdx.x >> 6, i = threadIdx.x & 63;
  const size_t at = (size_t)(first + min(i, n - 1)) * a.r.h_v + h + (which < heads ? which : 0);
  return i < n ? make_float2(a.r.g[at], a.r.beta[at]) : make_float2(1.0f, 0.0f);
}
// Their decay factors; `rec`: their records, whose factors are written here.
__device__ __forceinline__ void prepare_gates(PrepSmem& sm, uint8_t* rec, float2 gb, int heads) {
  const int tid = threadIdx.x, lane = tid & 31, which = tid >> 6, i = tid & 63;
  const bool on = which < heads;
  PrepGate& s = sm.gate[which];
  const float g = clamp_gate(gb.x), beta = gb.y;
  // a gate of zero counts as 2^-128: pow2 makes 0 of every decay over it, as of
  // those over a gate below 2^-126; a NaN stays one. log2f is good to an
  // ulp: over decays that matter the sum of those errors is below 2^-22.
  float2 G = make_float2(g == 0.0f ? -128.0f : log2f(g), 0.0f);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float2 y = make_float2(__shfl_up_sync(0xffffffffu, G.x, d), __shfl_up_sync(0xffffffffu, G.y, d));
    if (lane >= d) G = pair_add(G, y);
  }
  if (lane == 31) sm.part[tid >> 5] = G;
  __syncthreads();
  if (i >= 32) G = pair_add(G, sm.part[2 * which]);
  s.G[i] = G;
  __syncthreads();
  const float2 zero = make_float2(0.0f, 0.0f), end = s.G[63], mine = s.G[i | 15], prev = i < 16 ? zero : s.G[(i & ~15) - 1];
  s.beta[i] = beta;
  s.from[i] = pow2(pair_diff(G, prev));
  s.to[i] = pow2(pair_diff(mine, G));
  s.inv[i] = pow2(pair_diff(prev, G));
  if ((i & 15) == 0) s.steep[i >> 4] = !(pair_diff(mine, prev) >= -100.0f);
  const int bi = (i >> 2) & 3, bj = i & 3;
  if (i < 16 && bj < bi) s.hop[bi][bj] = pow2(pair_diff(s.G[16 * bi - 1], s.G[16 * bj + 15]));
  if (on) {
    float* coef = reinterpret_cast<float*>(rec + (size_t)which * kPrepBytes + kTermsBytes);
    const float e = pow2(pair_diff(G, zero));
    coef[i] = e;
    coef[64 + i] = beta;
    coef[128 + i] = beta * e;
    coef[192 + i] = pow2(pair_diff(end, G));
    if (i < 4) coef[256 + i] = pow2(pair_diff(end, zero));
  }
}

// One CTA per block and key head; the value heads that share the key head
// share q . k and k . k.
__global__ void __launch_bounds__(kPrepThreads, 5) k_chunk_prepare(const PrepArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  PrepSmem& s = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int c = blockIdx.x / a.r.h_k, hk = blockIdx.x - c * a.r.h_k;
  let_next_start();
  int first, n;
  if (!block_span(a, c, first, n)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int share = a.r.h_v / a.r.h_k;
  float2 gb = load_gates(a, first, n, hk * share, min(2, share));  // with the tiles
#pragma unroll 8
  for (int x = tid; x < 2 * 64 * 16; x += kPrepThreads) {
    const int which = x >> 10, row = (x >> 4) & 63, piece = x & 15;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(which ? a.r.k : a.r.q) +
                               (int64_t)(first + min(row, n - 1)) * (which ? a.r.k_stride : a.r.q_stride) + hk * 128;
    uint4 v = reinterpret_cast<const uint4*>(src)[piece];
    if (row >= n) v = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(&s.qk[which][row * kTile + 8 * piece]) = v;
  }
  __syncthreads();
  // the ten blocks on and below the diagonal, of q k^T (even warps) and of
  // k k^T (odd ones), five for each warp: every other one of the list
  // 00 10 11 20 21 22 30 31 32 33
  const int which = warp & 1, odd = warp >> 1;
  constexpr int rows0[5] = {0, 1, 2, 3, 3}, cols0[5] = {0, 1, 1, 0, 2};
  constexpr int rows1[5] = {1, 2, 2, 3, 3}, cols1[5] = {0, 0, 2, 1, 3};
  Acc dot[5];
#pragma unroll
  for (int x = 0; x < 5; ++x) {
    const int bi = odd ? rows1[x] : rows0[x], bj = odd ? cols1[x] : cols0[x];
    dot[x].zero();
    const __nv_bfloat16* A = &s.qk[which][(16 * bi + (lane & 15)) * kTile + 8 * (lane >> 4)];
    const __nv_bfloat16* Bm = &s.qk[1][(16 * bj + (lane & 7) + 8 * (lane >> 4)) * kTile + 8 * ((lane >> 3) & 1)];
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t fa[4], fb[4];
      ldmatrix4(fa, A + 16 * ks);
      ldmatrix4(fb, Bm + 16 * ks);
      dot[x].add(fa, fb);
    }
  }
  const int j2 = 2 * (lane & 3), r4 = lane >> 2;
  const int piece = blk_piece(lane & 15, lane >> 4);  // this lane's row of a matrix load
  const int left = blk_piece(r4, 0) + 2 * j2, turn = blk_piece(0, 1) - 2 * (blk_piece(r4, 0) & 16);  // see put_left
#pragma unroll 1
  for (int hh = 0; hh < share; ++hh) {
    const int h = hk * share + hh;
    uint8_t* rec = a.ws + ((uint64_t)c * a.r.h_v + h) * kPrepBytes;
    if ((hh & 1) == 0) {
      prepare_gates(s, rec, gb, min(2, share - hh));
      if (hh + 2 < share) gb = load_gates(a, first, n, h + 2, min(2, share - hh - 2));
    }
    const PrepGate& gt = s.gate[hh & 1];
    __syncthreads();  // the factors; the tiles (first head) or the previous head's matrices have been read
#pragma unroll
    for (int x = 0; x < 5; ++x) {
      const int bi = odd ? rows1[x] : rows0[x], bj = odd ? cols1[x] : cols0[x];
      const bool diag = bi == bj;
      const float* col = (diag ? gt.inv : gt.to) + 16 * bj + j2;
      float2 c0 = *reinterpret_cast<const float2*>(col), c1 = *reinterpret_cast<const float2*>(col + 8);
      const float hop = diag ? 1.0f : gt.hop[bi][bj];
      Acc m;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = 16 * bi + r4 + 8 * y;
        const float f = gt.from[i] * hop * (which ? gt.beta[i] : 1.0f);
        m.c[0][2 * y] = f * c0.x * dot[x].c[0][2 * y];
        m.c[0][2 * y + 1] = f * c0.y * dot[x].c[0][2 * y + 1];
        m.c[1][2 * y] = f * c1.x * dot[x].c[1][2 * y];
        m.c[1][2 * y + 1] = f * c1.y * dot[x].c[1][2 * y + 1];
      }
      if ((x == 0 || x == 1 || x == 2 || x == 4) && diag) {  // the others never are
        if (gt.steep[bi]) {
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const int li = r4 + 8 * ((z >> 1) & 1), lj = j2 + (z & 1) + 8 * (z >> 2);
            const float e = lj <= li ? pow2(pair_diff(gt.G[16 * bi + li], gt.G[16 * bi + lj])) : 0.0f;
            m.c[z >> 2][z & 3] = (which ? gt.beta[16 * bi + li] : 1.0f) * e * dot[x].c[z >> 2][z & 3];
          }
        }
#pragma unroll
        for (int z = 0; z < 8; ++z)  // above the diagonal: nothing, whatever the dots hold
          if (j2 + (z & 1) + 8 * (z >> 2) > r4 + 8 * ((z >> 1) & 1)) m.c[z >> 2][z & 3] = 0.0f;
        if (which) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int z = 0; z < 2; ++z)
              *reinterpret_cast<float2*>(s.Ad(bi) + (r4 + 8 * y) * kAd + j2 + 8 * z) =
                  make_float2(m.c[z][2 * y], m.c[z][2 * y + 1]);
          continue;
        }
      }
      Terms t;
      acc_terms(m, t);
      uint8_t* dst = (which ? s.m.A[below(bi, bj)][0] : s.m.P[tri(bi, bj)][0]) + left;
#pragma unroll
      for (int u = 0; u < kTerms; ++u) put_left(dst + u * kBlk, turn, t[u]);
    }
    __syncthreads();
    {  // the block on the diagonal: lane owns a column of its warp's (both half warps the same)
      const float* Ad = s.Ad(warp);
      const int col = lane & 15, half = lane >> 4;
      float t[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float acc = i == col ? 1.0f : 0.0f;
#pragma unroll
        for (int l = 0; l < i; l += 4) {  // A is 0 on its diagonal block's diagonal and above
          const float4 c = *reinterpret_cast<const float4*>(Ad + i * kAd + l);
          acc = fmaf(-c.x, t[l], acc);
          if (l + 1 < i) acc = fmaf(-c.y, t[l + 1], acc);
          if (l + 2 < i) acc = fmaf(-c.z, t[l + 2], acc);
          if (l + 3 < i) acc = fmaf(-c.w, t[l + 3], acc);
        }
        t[i] = acc;
      }
      uint8_t* dst = s.m.T[tri(warp, warp)][0] + 2 * (col & 7);
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // each half warp stores eight rows
        float v = half ? t[8 + i] : t[i];
        uint8_t* p = dst + blk_piece(8 * half + i, col >> 3);
#pragma unroll
        for (int u = 0; u < kTerms; ++u) {
          const uint32_t w = __float_as_uint(v);
          *reinterpret_cast<uint16_t*>(p + u * kBlk) = (uint16_t)(w >> 16);
          v -= __uint_as_float(w & 0xffff0000u);
        }
      }
    }
    // the other blocks, T(R, C) = -sum_l (sum_m T(R, m) A(m, l)) T(l, C): of
    // the pairs of blocks (stage 0: two warps), then of the pairs of those
#pragma unroll 1
    for (int stage = 0; stage < 2; ++stage) {
      __syncthreads();
      if (stage == 0 && warp >= 2) continue;
      const int R = stage ? 2 + (warp >> 1) : 2 * warp + 1, C = stage ? warp & 1 : 2 * warp;
      const int m0 = stage ? 2 : R, l1 = stage ? 1 : C;
      Acc acc, y;
      Terms ta, tb;
      acc.zero();
#pragma unroll 1
      for (int l = C; l <= l1; ++l) {
        y.zero();
#pragma unroll 1
        for (int m = m0; m <= R; ++m) {
#pragma unroll
          for (int u = 0; u < kTerms; ++u) {
            ldmatrix4(ta[u], s.m.T[tri(R, m)][u] + piece);
            ldmatrix4t(tb[u], s.m.A[below(m, l)][u] + piece);
          }
          add6(y, ta, tb);
        }
        acc_terms(y, ta);
#pragma unroll
        for (int u = 0; u < kTerms; ++u) ldmatrix4t(tb[u], s.m.T[tri(l, C)][u] + piece);
        add6(acc, ta, tb);
      }
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        acc.c[0][z] = -acc.c[0][z];
        acc.c[1][z] = -acc.c[1][z];
      }
      acc_terms(acc, ta);
#pragma unroll
      for (int u = 0; u < kTerms; ++u) put_left(s.m.T[tri(R, C)][u] + left, turn, ta[u]);
    }
    __syncthreads();
    // P T: five block products for each warp; T and P T leave
    const uint32_t todo = warp == 0 ? 0x3000u : warp == 1 ? 0x2010u : warp == 2 ? 0x3121u : 0x32112233u;  // (bi, bj)
    const int count = warp < 3 ? 2 : 4;
#pragma unroll 1
    for (int x = 0; x < count; ++x) {
      const int pi = (todo >> (8 * x + 4)) & 15, pj = (todo >> (8 * x)) & 15;
      Acc acc;
      acc.zero();
#pragma unroll 1
      for (int l = pj; l <= pi; ++l) {
        Terms pa, tb;
#pragma unroll
        for (int u = 0; u < kTerms; ++u) {
          ldmatrix4(pa[u], s.m.P[tri(pi, l)][u] + piece);
          ldmatrix4t(tb[u], s.m.T[tri(l, pj)][u] + piece);
        }
        add6(acc, pa, tb);
      }
      // T: the warp's 32 pieces of a term are 512 contiguous bytes of the record
      uint8_t* out = rec + row_piece(lane & 15, 8 * (lane >> 4)) + 512 * (pi - pj);
#pragma unroll
      for (int u = 0; u < kTerms; ++u)
        *reinterpret_cast<uint4*>(out + term_base(u) + pair_base(pj)) =
            *reinterpret_cast<const uint4*>(s.m.T[tri(pi, pj)][u] + piece);
      // P T: rows 64 - 16 pj of the operand on, row 16 (pi - pj) + ... of them
      uint8_t* o_at = rec + pair_base(pj) + 512 * (4 + pi - 2 * pj) + row_piece(r4, j2);
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        uint32_t t[kTerms];
        split3(acc.c[z >> 1][2 * (z & 1)], acc.c[z >> 1][2 * (z & 1) + 1], t);
        uint8_t* o2 = o_at + row_piece(8 * (z & 1), 8 * (z >> 1));
#pragma unroll
        for (int u = 0; u < kTerms; ++u) *reinterpret_cast<uint32_t*>(o2 + term_base(u)) = t[u];
      }
    }
  }
}

}  // namespace sqr
