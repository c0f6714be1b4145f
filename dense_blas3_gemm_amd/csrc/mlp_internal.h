// Internal interfaces of the MLP-block operators: products with an epilogue (bias,
// activation, residual, saved activation argument), the activation's 8-bit checkpoints
// and layer norm.
#pragma once

#include "gemm_internal.h"

namespace dbgemm {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };
enum { Z_NONE = 0, Z_BF16 = 1, Z_MX = 2 };
// element types of activations and weights (the values of C_BF16 and C_F32)
enum { T_BF16 = C_BF16, T_F32 = C_F32 };

// What an epilogue does with w = alpha * (the product), element (m, n):
//   forward: z = w + bias[n]; Z <- z (bf16, or E4M3 codes with a UE8M0 byte per 32 columns);
//            C <- act(z) + beta * R
//   grad:    C <- w * act'(Z); the column sums of that in fp32, before its rounding
struct EpArgs {
  int grad;
  int act;
  const void* bias;  // N values or null
  int bias_f32;
  const void* R;  // C's element type, or null
  int64_t ldr;
  float beta;
  int z_kind;
  void* Z;  // written (forward) or read (grad)
  int64_t ldz;
  uint8_t* S;  // Z_MX: ceil(N / 32) scale bytes per row
  int64_t lds;
  float* colsum;  // grad: fp32 partial sums, [part][whole8(N)], or null
};

// A product with an epilogue: the kernels take this in place of GemmArgs.
struct GemmEpArgs : GemmArgs {
  EpArgs ep;
};

// Products with an epilogue on the MFMA kernels: policy p (has_epilogue) on a, whose grid
// fields are set; with ep.colsum set, *parts receives the partial rows it writes.
hipError_t launch_mfma_ep(const Policy& p, const GemmEpArgs& a, int* parts, hipStream_t s);
// one per kernel family and (transA, transB) case, each in its own object
#define DBGEMM_EP_DECL(ab)                                                                               \
  hipError_t launch_mfma_pp_ep_##ab(const Policy& p, const GemmEpArgs& a, int* parts, hipStream_t s);     \
  hipError_t launch_mfma_dma_ep_##ab(const Policy& p, const GemmEpArgs& a, int* parts, hipStream_t s);
DBGEMM_EP_DECL(00)
DBGEMM_EP_DECL(01)
DBGEMM_EP_DECL(10)
DBGEMM_EP_DECL(11)
#undef DBGEMM_EP_DECL

// Products of a few rows, N a multiple of 8, operands as the MFMA kernels take them; ep.colsum,
// when set, receives the column sums themselves.
bool skinny_serves(int in_fp8, int transA, int transB, int64_t M, int64_t K);
hipError_t launch_skinny(const GemmEpArgs& a, hipStream_t s);

// ---- launchers (they return hipSuccess or the launch error)

// Epilogue of a product held in fp32: a.ws is rows [0, M) of alpha * op(A) op(B) with row
// stride ldw.  With ep.colsum set, *parts receives the number of partial rows written (at
// most max_parts >= 1).
hipError_t launch_ep_rows(const GemmEpArgs& a, int64_t ldw, int max_parts, int* parts, hipStream_t s);

// Columns of a partial row: whole eights, so that the kernels on both sides move whole vectors
// (the columns past the end hold nothing of use).
constexpr int64_t whole8(int64_t cols) { return (cols + 7) / 8 * 8; }

// out0[n] <- (accumulate ? out0[n] : 0) + sum over p < parts of src[p * ld + n], n < cols, and
// the same for out1 (or null) from column ld / 2 on; added in an order fixed by parts: the
// same bits every run.  parts == 0 writes zeros.  A row of src (each half of one) holds
// whole8(cols) columns.
hipError_t launch_colsum(const float* src, int parts, int64_t ld, int64_t cols, float* out0, float* out1,
                         int accumulate, hipStream_t s);

// H <- act(Z) (bf16) and Z's E4M3 codes and scales, Z bf16.
hipError_t launch_act_mx(int64_t rows, int64_t cols, int act, const void* z, int64_t ldz, void* h, int64_t ldh,
                         uint8_t* q, int64_t ldq, uint8_t* sc, int64_t ldsc, hipStream_t s);
// dZ <- dH * act'(Z), H <- act(Z) from Z's codes (dh with dz, h, dbias each optional).  *parts
// receives the partial rows of dbias written to `part` (at most max_parts); 0: dbias is done.
hipError_t launch_act_grad_mx(int64_t rows, int64_t cols, int act, const uint8_t* q, int64_t ldq, const uint8_t* sc,
                              int64_t ldsc, const void* dh, int64_t lddh, void* dz, int64_t lddz, void* h,
                              int64_t ldh, float* dbias, float* part, int max_parts, int* parts, hipStream_t s);

struct NormArgs {
  int64_t rows;
  int cols;
  const void* x;
  int64_t ldx;
  int x_kind;  // T_BF16 or T_F32
  const void* gamma;
  const void* beta;
  int w_kind;  // gamma and beta
  float* mean;
  float* rstd;
  float eps;  // forward
  void* y;    // forward: y; grad: dx (x's type)
  int64_t ldy;
  int y_kind;      // forward: y's type; grad: dy's type
  const void* dy;  // grad
  int64_t lddy;
  const void* dr;  // grad: added to dx (x's type), or null
  int64_t lddr;
  float* part;  // grad: partial sums of dgamma and dbeta, [part][2][whole8(cols)], or null
  float* dgamma;  // grad: the sums themselves, either may be null
  float* dbeta;
};
hipError_t launch_layernorm(const NormArgs& a, hipStream_t s);
// *parts receives the number of partial rows written to a.part (at most max_parts); 0: a.dgamma
// and a.dbeta are done.
hipError_t launch_layernorm_grad(const NormArgs& a, int max_parts, int* parts, hipStream_t s);

}  // namespace dbgemm
