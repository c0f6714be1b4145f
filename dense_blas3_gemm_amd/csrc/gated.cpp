// C-ABI of the gated feed-forward operators and of the 8-bit integer products (include/gemm.h):
// argument checks, workspace and launches.
#include "gemm.h"

#include <cmath>
#include <cstdint>

#include "gated_internal.h"
#include "mlp_host.h"

using namespace dbgemm;

namespace {

// Longest sum of products of two 8-bit integers (at most 2^14 each) that 32 bits hold.
constexpr int64_t kMaxK8 = 131071;

// The generic kernel over all of a; dbias: fp32 column sums, the second set from dbias2.
gemm_status_t run_simt(const HandleView& v, GatedArgs a, float* dbias, float* dbias2) {
  const bool sums = dbias || dbias2;
  const int mp = sums ? max_parts(v, 2 * whole8(a.N)) : 1;
  if (mp < 1) return GEMM_STATUS_NOT_SUPPORTED;
  a.ep.colsum = sums ? (float*)v.ws : nullptr;
  int parts = 0;
  hipError_t e = launch_gated_simt(a, mp, &parts, v.stream);
  if (e == hipSuccess && sums)
    e = launch_colsum((const float*)v.ws, parts, 2 * whole8(a.N), a.N, dbias, dbias2, 0, v.stream);
  return status(e);
}

gemm_status_t run(gemm_handle_t h, GatedArgs a, float* dbias = nullptr, float* dbias2 = nullptr) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  OnDevice on(v.device);
  if (!on.ok) return GEMM_STATUS_INTERNAL;
  if (a.M == 0 || a.N == 0) {  // no element; the sums over no rows are zeros
    if ((!dbias && !dbias2) || a.N == 0) return GEMM_STATUS_SUCCESS;
    return status(launch_colsum(nullptr, 0, 2 * whole8(a.N), a.N, dbias, dbias2, 0, v.stream));
  }
  if (a.alpha == 0.f) a.K = 0;
  return run_simt(v, a, dbias, dbias2);
}

// Operands (the second B is checked by the same rules) and C of one call.
struct Operands {
  int transB;
  int64_t M, N, K;
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  void* C;
  int64_t ldc;
};

gemm_status_t check(const Operands& p, float alpha, int dtype) {
  if (dtype != GEMM_BF16_F32 && dtype != GEMM_BF16_BF16 && dtype != GEMM_E4M3_BF16 && dtype != GEMM_E4M3_F32)
    return GEMM_STATUS_INVALID_VALUE;
  return gemm_check_args(GEMM_OP_N, p.transB, p.M, p.N, p.K, alpha, p.A, p.lda, p.B, p.ldb, 0.f, p.C, p.ldc, dtype);
}

// 8-bit integers: E4M3's sizes, and the factors.
gemm_status_t check_i8(const Operands& p, const float* sa, const float* sb, int c_type) {
  if (!valid_type(c_type)) return GEMM_STATUS_INVALID_VALUE;
  const gemm_status_t st = check(p, 1.f, c_type == GEMM_TYPE_F32 ? GEMM_E4M3_F32 : GEMM_E4M3_BF16);
  if (st != GEMM_STATUS_SUCCESS) return st;
  if (p.M > 0 && p.N > 0 && (!sa || !sb)) return GEMM_STATUS_INVALID_VALUE;
  return p.K > kMaxK8 ? GEMM_STATUS_NOT_SUPPORTED : GEMM_STATUS_SUCCESS;
}

GatedArgs args_of(const Operands& p, int op, int in_kind, float alpha, int c_kind) {
  GatedArgs a{};
  a.A = p.A;
  a.B = p.B;
  a.C = p.C;
  a.lda = p.lda;
  a.ldb = p.ldb;
  a.ldc = p.ldc;
  a.M = (int)p.M;
  a.N = (int)p.N;
  a.K = (int)p.K;
  a.alpha = alpha;
  a.c_kind = c_kind;
  a.in_fp8 = in_kind == GT_E4M3;
  a.transB = p.transB;
  a.splits = 1;
  a.op = op;
  a.in_kind = in_kind;
  return a;
}
int c_kind_of(int dtype) { return dtype == GEMM_BF16_F32 || dtype == GEMM_E4M3_F32 ? C_F32 : C_BF16; }
int in_kind_of(int dtype) { return dtype == GEMM_BF16_F32 || dtype == GEMM_BF16_BF16 ? GT_BF16 : GT_E4M3; }

gemm_status_t check_gate(const gemm_gate_t* ep, int64_t N) {
  if (!ep || !valid_act(ep->act) || ((ep->bias_g || ep->bias_u) && !valid_type(ep->bias_type)) ||
      (ep->g && !valid_ld(ep->ld_g, N)) || (ep->u && !valid_ld(ep->ld_u, N)))
    return GEMM_STATUS_INVALID_VALUE;
  return GEMM_STATUS_SUCCESS;
}

void set_gate(GatedArgs& a, const gemm_gate_t* ep, const void* B2, int64_t ldb2) {
  a.B2 = B2;
  a.ldb2 = ldb2;
  a.ep.act = ep->act;
  a.ep.bias_f32 = ep->bias_type == GEMM_TYPE_F32;
  a.ep.bias = ep->bias_g;
  a.ep.bias2 = ep->bias_u;
  a.ep.G = ep->g;
  a.ep.ldg = ep->ld_g;
  a.ep.U = ep->u;
  a.ep.ldu = ep->ld_u;
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_gated(gemm_handle_t h, int transB, int64_t M, int64_t N, int64_t K, float alpha, const void* A,
                             int64_t lda, const void* Bg, int64_t ldbg, const void* Bu, int64_t ldbu,
                             const gemm_gate_t* ep, void* C, int64_t ldc, int dtype) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  const Operands p{transB, M, N, K, A, lda, Bg, ldbg, C, ldc};
  Operands p2 = p;
  p2.B = Bu;
  p2.ldb = ldbu;
  gemm_status_t st = check(p, alpha, dtype);
  if (st == GEMM_STATUS_SUCCESS) st = check(p2, alpha, dtype);
  if (st == GEMM_STATUS_SUCCESS) st = check_gate(ep, N);
  if (st != GEMM_STATUS_SUCCESS) return st;
  GatedArgs a = args_of(p, GT_GATED, in_kind_of(dtype), alpha, c_kind_of(dtype));
  set_gate(a, ep, Bu, ldbu);
  return run(h, a);
}

gemm_status_t gemm_run_dgated(gemm_handle_t h, int transB, int64_t M, int64_t N, int64_t K, float alpha, const void* A,
                              int64_t lda, const void* B, int64_t ldb, int act, const void* g, int64_t ld_g,
                              const void* u, int64_t ld_u, void* dg, int64_t ld_dg, void* du, int64_t ld_du, void* out,
                              int64_t ld_out, float* dbias_g, float* dbias_u, int dtype) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  const Operands p{transB, M, N, K, A, lda, B, ldb, dg, ld_dg};
  gemm_status_t st = check(p, alpha, dtype);
  if (st != GEMM_STATUS_SUCCESS) return st;
  if (!valid_act(act) || !valid_ld(ld_g, N) || !valid_ld(ld_u, N) || !valid_ld(ld_du, N) || (out && !valid_ld(ld_out, N)) ||
      (M > 0 && N > 0 && (!g || !u || !du)))
    return GEMM_STATUS_INVALID_VALUE;
  GatedArgs a = args_of(p, GT_GRAD, in_kind_of(dtype), alpha, c_kind_of(dtype));
  a.ep.act = act;
  a.ep.G = const_cast<void*>(g);
  a.ep.ldg = ld_g;
  a.ep.U = const_cast<void*>(u);
  a.ep.ldu = ld_u;
  a.ep.D2 = du;
  a.ep.ldd2 = ld_du;
  a.ep.H = out;
  a.ep.ldh = ld_out;
  return run(h, a, dbias_g, dbias_u);
}

gemm_status_t gemm_quantize_i8(gemm_handle_t h, int64_t rows, int64_t cols, const void* src, int64_t ld_src,
                               int src_type, int8_t* dst, int64_t ld_dst, float* scales) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  if (!valid_size(rows) || !valid_size(cols) || !valid_type(src_type) || !valid_ld(ld_src, cols) || !valid_ld(ld_dst, cols))
    return GEMM_STATUS_INVALID_VALUE;
  if (rows == 0) return GEMM_STATUS_SUCCESS;
  if (!scales || (cols > 0 && (!src || !dst))) return GEMM_STATUS_INVALID_VALUE;
  OnDevice on(v.device);
  if (!on.ok) return GEMM_STATUS_INTERNAL;
  return status(launch_quantize_i8(rows, cols, src, ld_src, src_type, dst, ld_dst, scales, v.stream));
}

gemm_status_t gemm_run_i8(gemm_handle_t h, int transB, int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                          const float* scale_a, const int8_t* B, int64_t ldb, const float* scale_b,
                          const gemm_epilogue_t* ep, void* C, int64_t ldc, int c_type) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  const Operands p{transB, M, N, K, A, lda, B, ldb, C, ldc};
  const gemm_status_t st = check_i8(p, scale_a, scale_b, c_type);
  if (st != GEMM_STATUS_SUCCESS) return st;
  if (!ep || !valid_act(ep->act) || ep->z_kind != GEMM_Z_NONE || (ep->bias && !valid_type(ep->bias_type)) ||
      (ep->residual && !valid_ld(ep->ld_residual, N)))
    return GEMM_STATUS_INVALID_VALUE;
  if (ep->residual && !std::isfinite(ep->beta)) return GEMM_STATUS_NOT_SUPPORTED;
  GatedArgs a = args_of(p, GT_LINEAR, GT_I8, 1.f, c_type);
  a.ep.act = ep->act;
  a.ep.bias = ep->bias;
  a.ep.bias_f32 = ep->bias_type == GEMM_TYPE_F32;
  a.ep.sa = scale_a;
  a.ep.sb = scale_b;
  if (ep->beta != 0.f) a.ep.R = ep->residual;
  a.ep.ldr = ep->ld_residual;
  a.ep.beta = ep->beta;
  return run(h, a);
}

gemm_status_t gemm_run_gated_i8(gemm_handle_t h, int transB, int64_t M, int64_t N, int64_t K, const int8_t* A,
                                int64_t lda, const float* scale_a, const int8_t* Bg, int64_t ldbg,
                                const float* scale_bg, const int8_t* Bu, int64_t ldbu, const float* scale_bu,
                                const gemm_gate_t* ep, void* C, int64_t ldc, int c_type) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  const Operands p{transB, M, N, K, A, lda, Bg, ldbg, C, ldc};
  Operands p2 = p;
  p2.B = Bu;
  p2.ldb = ldbu;
  gemm_status_t st = check_i8(p, scale_a, scale_bg, c_type);
  if (st == GEMM_STATUS_SUCCESS) st = check_i8(p2, scale_a, scale_bu, c_type);
  if (st == GEMM_STATUS_SUCCESS) st = check_gate(ep, N);
  if (st != GEMM_STATUS_SUCCESS) return st;
  GatedArgs a = args_of(p, GT_GATED, GT_I8, 1.f, c_type);
  set_gate(a, ep, Bu, ldbu);
  a.ep.sa = scale_a;
  a.ep.sb = scale_bg;
  a.ep.sb2 = scale_bu;
  return run(h, a);
}

}  // extern "C"
