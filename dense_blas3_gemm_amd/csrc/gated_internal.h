// Internal interfaces of the gated feed-forward operators: both projections of a gated block
// with the activation and the product of the two behind them, the product that runs back
// through that, and products of 8-bit integers with a scale for each row of A and column of B.
#pragma once

#include "mlp_internal.h"

namespace dbgemm {

// What a product's results go through, element (m, n); w is alpha * (A op(B)), or for 8-bit
// integers (the exact sum * sa[m]) * sb[n] (or the factors the other way round, kFarFactor), w2 the
// same of the second B:
//   GT_LINEAR: C <- act(w + bias) + beta * R
//   GT_GATED:  g = w + bias, u = w2 + bias2; G <- g, U <- u (where kept); C <- act(g) * u
//   GT_GRAD:   C <- w * U * act'(G); D2 <- w * act(G); H <- act(G) * U; the column sums of the
//              first two in fp32, before their rounding
enum { GT_LINEAR = 0, GT_GATED = 1, GT_GRAD = 2 };
// operands: bf16, E4M3 bytes, 8-bit integers
enum { GT_BF16 = 0, GT_E4M3 = 1, GT_I8 = 2 };

struct GatedEp {
  int act;
  int bias_f32;
  const void* bias;  // N values or null
  const void* bias2;
  const float* sa;  // 8-bit integers: one factor for each row of A and each column of B (and of B2)
  const float* sb;
  const float* sb2;
  const void* R;  // C's element type, or null
  int64_t ldr;
  float beta;
  void* G;  // bf16; written and null unless kept (GT_GATED), or read (GT_GRAD)
  int64_t ldg;
  void* U;
  int64_t ldu;
  void* D2;  // C's element type
  int64_t ldd2;
  void* H;  // bf16, or null
  int64_t ldh;
  // What the epilogue reads, the residual or G and U, would fill half of the caches (128 of 256 MB) or
  // more: the 256 x 256 tiles read it past them.  us through them and past, three sets of buffers in
  // turn: 8-bit integers with a bf16 residual, K = 1024, 2048 x 8192 (32 MB) 28.5 and 31.7, 4096 x 8192
  // (64) 56.6 and 61.0, 4096 x 12288 (96) 81.9 and 81.1, 8192 x 8192 (128) 129 and 113, 8192 x 12288 (192)
  // 167 and 153; with K = 4096 62 and 64.5, 135 and 127, 194 and 183, 269 and 244, 382 and 359; a gradient,
  // K = 1024, 64 MB of G and U 48.6 and 53.2, 128 106 and 102, 256 210 and 196.  So past them is the faster
  // from 128 MB on throughout, and from 64 to 96 by K; a smaller one may still be there from whoever wrote
  // it (1078 x 7888 x 2240 with an fp32 residual, 34 MB, 39 us, past the caches 52).
  int past;
  float* colsum;  // fp32 partial sums, [part][2][whole8(N)], or null
  float* sum1;    // the kernels of a few rows: the sums themselves, each or null
  float* sum2;
};

// Past this magnitude of a row's factor its columns' factors come first: sum * sa[m] could leave fp32's
// range (a row that holds bf16's lowest value has a factor of 2.7e36) where sum * sa[m] * sb[n] does
// not.  A sum is a whole number of at most 2^31, so neither order loses anything else: up to here its
// product with sa[m] is at most 2^95; past here one with sb[n] overflows from |sb[n]| = 2^97 on only,
// where the result does too; and times a subnormal factor it is a whole number of 2^-149, exact.
constexpr float kFarFactor = 0x1p64f;

// (B2 and ldb2 of GemmArgs hold the second B.)
struct GatedArgs : GemmArgs {
  int op;
  int in_kind;
  GatedEp ep;
};

// The MFMA kernels of an operand kind: the input mode of the policies that serve it, of its own
// configurations, and their K tile for a policy's.  8-bit integers run on the bf16 tiles: as many
// bytes of K, twice the elements.
constexpr int gt_policy_in(int kind) { return kind == GT_E4M3 ? 5 : 0; }
constexpr int gt_in(int kind) { return kind == GT_E4M3 ? 5 : kind == GT_I8 ? 7 : 0; }
constexpr int gt_bk(int kind, int bk) { return kind == GT_I8 ? 2 * bk : bk; }

// a, whose grid fields are set, on policy p (has_epilogue); N in whole eights, operands as the MFMA
// kernels take them.  With ep.colsum set, *parts receives the partial rows it writes.
hipError_t launch_mfma_gated(const Policy& p, const GatedArgs& a, int* parts, hipStream_t s);
// one per kernel family, operand kind and transB, each in its own object
#define DBGEMM_GT_DECL(in, b)                                                                           \
  hipError_t launch_mfma_pp_gt_##in##b(const Policy& p, const GatedArgs& a, int* parts, hipStream_t s); \
  hipError_t launch_mfma_dma_gt_##in##b(const Policy& p, const GatedArgs& a, int* parts, hipStream_t s);
DBGEMM_GT_DECL(0, 0)
DBGEMM_GT_DECL(0, 1)
DBGEMM_GT_DECL(1, 0)
DBGEMM_GT_DECL(1, 1)
DBGEMM_GT_DECL(2, 0)
DBGEMM_GT_DECL(2, 1)
#undef DBGEMM_GT_DECL

// Products of up to kFewRows rows, `cols` columns of each B to a workgroup, the rest as for
// launch_mfma_gated; ep.sum1 and ep.sum2 receive the column sums.
constexpr int64_t kFewRows = 64;
hipError_t launch_gated_skinny(const GatedArgs& a, int cols, hipStream_t s);
// The columns that take the least time by a model, and that time in us.
double few_rows_us(int op, int in_kind, int transB, int64_t M, int64_t N, int64_t K, int cu_count, int* cols);

// Any sizes, strides and alignment (op(A) = A).  With ep.colsum set, *parts receives the number
// of partial rows written (at most max_parts >= 1).
hipError_t launch_gated_simt(const GatedArgs& a, int max_parts, int* parts, hipStream_t s);
bool gated_simt_thin(const GatedArgs& a);  // whether on the kernel for few elements

// Rows of bf16 or fp32 -> 8-bit integers and a factor each.
hipError_t launch_quantize_i8(int64_t rows, int64_t cols, const void* src, int64_t ld_src, int src_kind, int8_t* dst,
                              int64_t ld_dst, float* scales, hipStream_t s);

}  // namespace dbgemm

// For tests: the launches of a call on a device of cu_count CUs, by the code that makes them, as
// "kernel[+sk<splits>] rowsxcolumns; ..." in their order (without the launches that add up splits and
// partial column sums).  op and in_kind as above, the operands' pointers taken as aligned, the workspace a
// handle's.  0, or 1 where the arguments or the text's length do not do.  Pure host code.
extern "C" int dbgemm_gated_plan(int op, int in_kind, int transB, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                                 int64_t ldb2, int sums, int cu_count, char* text, size_t len);
