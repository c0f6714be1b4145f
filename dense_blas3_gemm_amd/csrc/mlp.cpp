// C-ABI of the MLP-block operators (include/gemm.h): argument checks, workspace and launches.
#include "gemm.h"

#include <cmath>
#include <cstdint>

#include "mlp_host.h"

using namespace dbgemm;

static_assert(GEMM_ACT_NONE == ACT_NONE && GEMM_ACT_RELU == ACT_RELU && GEMM_ACT_GELU == ACT_GELU &&
                  GEMM_ACT_GELU_TANH == ACT_GELU_TANH && GEMM_ACT_SILU == ACT_SILU,
              "the kernels' activation codes are the C-ABI's");
static_assert(GEMM_Z_NONE == Z_NONE && GEMM_Z_BF16 == Z_BF16 && GEMM_Z_MX == Z_MX, "the kernels' Z kinds");
static_assert(GEMM_TYPE_BF16 == T_BF16 && GEMM_TYPE_F32 == T_F32, "the kernels' element types");

namespace {

// Operand checks shared by the two products; bf16 or E4M3 operands, bf16 or fp32 C.
gemm_status_t check_product(int transA, int transB, int64_t M, int64_t N, int64_t K, float alpha, const void* A,
                            int64_t lda, const void* B, int64_t ldb, const void* C, int64_t ldc, int dtype) {
  if (dtype != GEMM_BF16_F32 && dtype != GEMM_BF16_BF16 && dtype != GEMM_E4M3_BF16 && dtype != GEMM_E4M3_F32)
    return GEMM_STATUS_INVALID_VALUE;
  return gemm_check_args(transA, transB, M, N, K, alpha, A, lda, B, ldb, 0.f, C, ldc, dtype);
}

// Z of M x N: bf16 rows, or codes with their scale rows.
gemm_status_t check_z(int kind, const void* z, int64_t ldz, const uint8_t* s, int64_t lds, int64_t M, int64_t N) {
  if (kind == GEMM_Z_NONE) return GEMM_STATUS_SUCCESS;
  if (kind != GEMM_Z_BF16 && kind != GEMM_Z_MX) return GEMM_STATUS_INVALID_VALUE;
  if (!valid_ld(ldz, N) || (kind == GEMM_Z_MX && !valid_ld(lds, (N + 31) / 32))) return GEMM_STATUS_INVALID_VALUE;
  if (M > 0 && N > 0 && (!z || (kind == GEMM_Z_MX && !s))) return GEMM_STATUS_INVALID_VALUE;
  return GEMM_STATUS_SUCCESS;
}

// The product in fp32 into the workspace, a block of rows at a time, and the epilogue over it.
gemm_status_t run_by_rows(const HandleView& v, GemmEpArgs a, int transA, int transB, int dtype, float* dbias) {
  const int f32_dtype = (dtype == GEMM_BF16_F32 || dtype == GEMM_BF16_BF16) ? GEMM_BF16_F32 : GEMM_E4M3_F32;
  const int64_t es = f32_dtype == GEMM_BF16_F32 ? 2 : 1;
  const int64_t M = a.M, ldw = ((int64_t)a.N + 3) / 4 * 4;
  if (!v.ws || v.ws_bytes <= kPartBytes) return GEMM_STATUS_NOT_SUPPORTED;
  int64_t step = (int64_t)((v.ws_bytes - kPartBytes) / sizeof(float)) / ldw;
  if (step > (1 << 21)) step = 1 << 21;  // the generic product's grid
  if (step >= 256) step -= step % 256;   // blocks of rows keep the operands' alignment
  if (step > M) step = M;
  const int mp = dbias ? max_parts(v, whole8(a.N)) : 1;
  if (step < 1 || mp < 1) return GEMM_STATUS_NOT_SUPPORTED;
  float* part = (float*)v.ws;
  float* w = (float*)((char*)v.ws + kPartBytes);
  const char* A = (const char*)a.A;
  char* C = (char*)a.C;
  EpArgs e = a.ep;
  const int64_t ce = a.c_kind == C_F32 ? 4 : 2, ze = e.z_kind == Z_MX ? 1 : 2;
  for (int64_t m0 = 0; m0 < M; m0 += step) {
    const int64_t rows = M - m0 < step ? M - m0 : step;
    const void* am = A ? A + (transA ? m0 : m0 * a.lda) * es : nullptr;
    hipError_t err = gemm_enqueue(v, transA, transB, rows, a.N, a.K, a.alpha, am, a.lda, a.B, a.ldb, 0.f, w, ldw,
                                  f32_dtype, GemmExtras{});
    if (err != hipSuccess) return GEMM_STATUS_LAUNCH_FAILED;
    a.M = (int)rows;
    a.ws = w;
    a.C = C + m0 * a.ldc * ce;
    a.ep.R = e.R ? (const char*)e.R + m0 * e.ldr * ce : nullptr;
    a.ep.Z = e.Z ? (char*)e.Z + m0 * e.ldz * ze : nullptr;
    a.ep.S = e.S ? e.S + m0 * e.lds : nullptr;
    a.ep.colsum = dbias ? part : nullptr;
    int parts = 0;
    err = launch_ep_rows(a, ldw, mp, &parts, v.stream);
    if (err == hipSuccess && dbias) err = launch_colsum(part, parts, whole8(a.N), a.N, dbias, nullptr, m0 > 0, v.stream);
    if (err != hipSuccess) return GEMM_STATUS_LAUNCH_FAILED;
  }
  return GEMM_STATUS_SUCCESS;
}

// One launch on policy p with sp splits; dbias partials into ep.colsum, *parts rows of them.
hipError_t run_tiles(const HandleView& v, GemmEpArgs a, const Policy& p, int sp, int* parts) {
  a.tiles_m = (a.M + p.BM - 1) / p.BM;
  a.tiles_n = (a.N + p.BN - 1) / p.BN;
  a.group = p.group;
  a.raster_n = p.raster_n;
  a.xcd = p.xcd;
  a.swizzle = p.swizzle;
  a.splits = sp;
  a.kt_per_split = (int)split_kt(p, a.K, sp);
  a.ws = sp > 1 ? (float*)v.ws : nullptr;
  return launch_mfma_ep(p, a, parts, v.stream);
}

// the partial rows of column sums that run_tiles leaves: a row of waves each, or after a split
// a row of fragments
int64_t partial_rows(const Policy& p, int64_t M, int sp) {
  return (M + p.BM - 1) / p.BM * (sp > 1 ? p.BM / p.WM / 16 : p.WM);
}

// a's rows [m0, m0 + M) and columns [n0, n0 + N); n0 a multiple of 32.
GemmEpArgs part_of(const GemmEpArgs& a, int64_t m0, int64_t n0, int64_t M, int64_t N) {
  GemmEpArgs r = a;
  const int64_t es = a.in_fp8 ? 1 : 2, ce = a.c_kind == C_F32 ? 4 : 2, ze = a.ep.z_kind == Z_MX ? 1 : 2;
  r.M = (int)M;
  r.N = (int)N;
  r.A = (const char*)a.A + (a.transA ? m0 : m0 * a.lda) * es;
  r.B = (const char*)a.B + (a.transB ? n0 * a.ldb : n0) * es;
  r.C = (char*)a.C + (m0 * a.ldc + n0) * ce;
  if (a.ep.bias) r.ep.bias = (const char*)a.ep.bias + n0 * (a.ep.bias_f32 ? 4 : 2);
  if (a.ep.R) r.ep.R = (const char*)a.ep.R + (m0 * a.ep.ldr + n0) * ce;
  if (a.ep.Z) r.ep.Z = (char*)a.ep.Z + (m0 * a.ep.ldz + n0) * ze;
  if (a.ep.S) r.ep.S = a.ep.S + m0 * a.ep.lds + n0 / 32;
  return r;
}

// The product with its epilogue in the kernel that computes it; false when no such kernel
// takes the operands.
bool run_fused(const HandleView& v, GemmEpArgs a, int transA, int transB, int dtype, float* dbias, gemm_status_t* st) {
  if (a.K == 0 || a.alpha == 0.f || a.N % 8 != 0) return false;
  Problem pr = gemm_problem(transA, transB, a.M, a.N, a.K, a.A, a.lda, a.B, a.ldb, a.C, a.ldc, dtype);
  if (!pr.fast_ok) return false;
  a.in_fp8 = pr.in_fp8;
  a.transA = transA;
  a.transB = transB;
  if (skinny_serves(a.in_fp8, transA, transB, a.M, a.K)) {
    a.ep.colsum = dbias;
    *st = status(launch_skinny(a, v.stream));
    return true;
  }
  pr.ep = true;
  int sp = 1;
  double cost = 0.0;
  const int64_t split_floats = v.ws ? (int64_t)(kPartBytes / sizeof(float)) : 0;
  int idx = policy_select(pr, v.cu_count, split_floats, &sp, &cost);
  if (policy_at(idx).kind != KIND_MFMA) return false;
  const Cut cut = policy_cut(pr, v.cu_count, split_floats, cost);
  const int64_t M1 = cut.p >= 0 && cut.by_rows ? cut.at : a.M, N1 = cut.p >= 0 && !cut.by_rows ? cut.at : a.N;
  GemmEpArgs a1 = part_of(a, 0, 0, M1, N1), a2{};
  int idx2 = 0, sp2 = 1;
  if (cut.p >= 0) {
    a2 = part_of(a, a.M - M1 ? M1 : 0, a.N - N1 ? N1 : 0, cut.by_rows ? a.M - M1 : a.M, cut.by_rows ? a.N : a.N - N1);
    idx = cut.p;
    sp = 1;
    pr.M = a2.M;
    pr.N = a2.N;
    idx2 = policy_select(pr, v.cu_count, split_floats, &sp2);
    if (policy_at(idx2).kind != KIND_MFMA) return false;
  }
  float* part = nullptr;
  if (dbias) {
    const int64_t floats = partial_rows(policy_at(idx), a1.M, sp) * a1.N +
                           (cut.p >= 0 ? partial_rows(policy_at(idx2), a2.M, sp2) * a2.N : 0);
    if (!v.ws || v.ws_bytes < kPartBytes + (size_t)floats * sizeof(float)) return false;
    part = a1.ep.colsum = (float*)((char*)v.ws + kPartBytes);
  }
  int parts = 0, parts2 = 0;
  hipError_t e = run_tiles(v, a1, policy_at(idx), sp, &parts);
  if (e == hipSuccess && dbias && !cut.by_rows)
    e = launch_colsum(part, parts, a1.N, a1.N, dbias, nullptr, 0, v.stream);
  if (e == hipSuccess && cut.p >= 0) {
    if (dbias) a2.ep.colsum = part + (int64_t)parts * a1.N;
    e = run_tiles(v, a2, policy_at(idx2), sp2, &parts2);
    if (e == hipSuccess && dbias)
      e = cut.by_rows ? launch_colsum(part, parts + parts2, a.N, a.N, dbias, nullptr, 0, v.stream)
                      : launch_colsum(a2.ep.colsum, parts2, a2.N, a2.N, dbias + N1, nullptr, 0, v.stream);
  }
  *st = status(e);
  return true;
}

gemm_status_t run_product(gemm_handle_t h, int transA, int transB, int64_t M, int64_t N, int64_t K, float alpha,
                          const void* A, int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc, int dtype,
                          const EpArgs& e, float* dbias) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  OnDevice on(v.device);
  if (!on.ok) return GEMM_STATUS_INTERNAL;
  if (M == 0 || N == 0)  // no element of C; the sums over no rows are zeros
    return dbias && N > 0 ? status(launch_colsum(nullptr, 0, N, N, dbias, nullptr, 0, v.stream)) : GEMM_STATUS_SUCCESS;
  GemmEpArgs a{};
  a.A = A;
  a.B = B;
  a.C = C;
  a.lda = lda;
  a.ldb = ldb;
  a.ldc = ldc;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.alpha = alpha;
  a.c_kind = (dtype == GEMM_BF16_F32 || dtype == GEMM_E4M3_F32) ? C_F32 : C_BF16;
  a.ep = e;
  gemm_status_t st;
  if (run_fused(v, a, transA, transB, dtype, dbias, &st)) return st;
  return run_by_rows(v, a, transA, transB, dtype, dbias);
}

}  // namespace

namespace dbgemm {
hipError_t launch_mfma_ep(const Policy& p, const GemmEpArgs& a, int* parts, hipStream_t s) {
#define DBGEMM_EP_CASE(ab) \
  return p.pipe == 2 ? launch_mfma_pp_ep_##ab(p, a, parts, s) : launch_mfma_dma_ep_##ab(p, a, parts, s)
  switch (a.transA * 2 + a.transB) {
    case 0: DBGEMM_EP_CASE(00);
    case 1: DBGEMM_EP_CASE(01);
    case 2: DBGEMM_EP_CASE(10);
    default: DBGEMM_EP_CASE(11);
  }
#undef DBGEMM_EP_CASE
}
}  // namespace dbgemm

extern "C" {

gemm_status_t gemm_run_act(gemm_handle_t h, int transA, int transB, int64_t M, int64_t N, int64_t K, float alpha,
                           const void* A, int64_t lda, const void* B, int64_t ldb, const gemm_epilogue_t* ep,
                           void* C, int64_t ldc, int dtype) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  if (!ep || !valid_act(ep->act)) return GEMM_STATUS_INVALID_VALUE;
  gemm_status_t st = check_product(transA, transB, M, N, K, alpha, A, lda, B, ldb, C, ldc, dtype);
  if (st != GEMM_STATUS_SUCCESS) return st;
  if (ep->bias && !valid_type(ep->bias_type)) return GEMM_STATUS_INVALID_VALUE;
  if (ep->residual && !valid_ld(ep->ld_residual, N)) return GEMM_STATUS_INVALID_VALUE;
  st = check_z(ep->z_kind, ep->z, ep->ld_z, ep->z_scales, ep->ld_z_scales, M, N);
  if (st != GEMM_STATUS_SUCCESS) return st;
  if (ep->residual && !std::isfinite(ep->beta)) return GEMM_STATUS_NOT_SUPPORTED;
  EpArgs e{};
  e.act = ep->act;
  e.bias = ep->bias;
  e.bias_f32 = ep->bias_type == GEMM_TYPE_F32;
  if (ep->beta != 0.f) e.R = ep->residual;
  e.ldr = ep->ld_residual;
  e.beta = ep->beta;
  e.z_kind = ep->z_kind;
  e.Z = ep->z;
  e.ldz = ep->ld_z;
  e.S = ep->z_scales;
  e.lds = ep->ld_z_scales;
  return run_product(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, C, ldc, dtype, e, nullptr);
}

gemm_status_t gemm_run_dact(gemm_handle_t h, int transA, int transB, int64_t M, int64_t N, int64_t K, float alpha,
                            const void* A, int64_t lda, const void* B, int64_t ldb, int act, int z_kind,
                            const void* z, int64_t ld_z, const uint8_t* z_scales, int64_t ld_z_scales, float* dbias,
                            void* C, int64_t ldc, int dtype) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  if (!valid_act(act) || z_kind == GEMM_Z_NONE) return GEMM_STATUS_INVALID_VALUE;
  gemm_status_t st = check_product(transA, transB, M, N, K, alpha, A, lda, B, ldb, C, ldc, dtype);
  if (st != GEMM_STATUS_SUCCESS) return st;
  st = check_z(z_kind, z, ld_z, z_scales, ld_z_scales, M, N);
  if (st != GEMM_STATUS_SUCCESS) return st;
  EpArgs e{};
  e.grad = 1;
  e.act = act;
  e.z_kind = z_kind;
  e.Z = const_cast<void*>(z);
  e.ldz = ld_z;
  e.S = const_cast<uint8_t*>(z_scales);
  e.lds = ld_z_scales;
  return run_product(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, C, ldc, dtype, e, dbias);
}

gemm_status_t gemm_act_mx(gemm_handle_t h, int64_t rows, int64_t cols, int act, const void* z, int64_t ld_z, void* out,
                          int64_t ld_out, void* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  if (!valid_act(act) || !valid_size(rows) || !valid_size(cols)) return GEMM_STATUS_INVALID_VALUE;
  if (!valid_ld(ld_z, cols) || !valid_ld(ld_out, cols) || !valid_ld(ld_codes, cols) ||
      !valid_ld(ld_scales, (cols + 31) / 32))
    return GEMM_STATUS_INVALID_VALUE;
  if (rows == 0 || cols == 0) return GEMM_STATUS_SUCCESS;
  if (!z || !out || !codes || !scales) return GEMM_STATUS_INVALID_VALUE;
  OnDevice on(v.device);
  if (!on.ok) return GEMM_STATUS_INTERNAL;
  return status(launch_act_mx(rows, cols, act, z, ld_z, out, ld_out, (uint8_t*)codes, ld_codes, scales, ld_scales,
                              v.stream));
}

gemm_status_t gemm_act_grad_mx(gemm_handle_t h, int64_t rows, int64_t cols, int act, const void* codes,
                               int64_t ld_codes, const uint8_t* scales, int64_t ld_scales, const void* dout,
                               int64_t ld_dout, void* dz, int64_t ld_dz, float* dbias, void* out, int64_t ld_out) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  if (!valid_act(act) || !valid_size(rows) || !valid_size(cols)) return GEMM_STATUS_INVALID_VALUE;
  if (!valid_ld(ld_codes, cols) || !valid_ld(ld_scales, (cols + 31) / 32) || (dout && !valid_ld(ld_dout, cols)) ||
      (dz && !valid_ld(ld_dz, cols)) || (out && !valid_ld(ld_out, cols)))
    return GEMM_STATUS_INVALID_VALUE;
  const bool empty = rows == 0 || cols == 0;
  if (!empty && (!codes || !scales)) return GEMM_STATUS_INVALID_VALUE;
  // dz and dbias come from dout; there has to be something to write
  if (!empty && ((dz || dbias) != (dout != nullptr) || (!dout && !out))) return GEMM_STATUS_INVALID_VALUE;
  OnDevice on(v.device);
  if (!on.ok) return GEMM_STATUS_INTERNAL;
  if (empty)
    return dbias && cols > 0 ? status(launch_colsum(nullptr, 0, cols, cols, dbias, nullptr, 0, v.stream))
                             : GEMM_STATUS_SUCCESS;
  const int mp = dbias ? max_parts(v, whole8(cols)) : 1;
  if (mp < 1) return GEMM_STATUS_NOT_SUPPORTED;
  int parts = 0;
  hipError_t e = launch_act_grad_mx(rows, cols, act, (const uint8_t*)codes, ld_codes, scales, ld_scales, dout, ld_dout,
                                    dz, ld_dz, out, ld_out, dbias, (float*)v.ws, mp, &parts, v.stream);
  if (e == hipSuccess && parts) e = launch_colsum((const float*)v.ws, parts, whole8(cols), cols, dbias, nullptr, 0, v.stream);
  return status(e);
}

gemm_status_t gemm_layernorm(gemm_handle_t h, int64_t rows, int64_t cols, const void* x, int64_t ld_x, int x_type,
                             const void* gamma, const void* beta, int weight_type, float eps, void* y, int64_t ld_y,
                             int y_type, float* mean, float* rstd) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  if (!valid_size(rows) || !valid_size(cols) || !valid_type(x_type) || !valid_type(y_type) ||
      ((gamma || beta) && !valid_type(weight_type)) || !valid_ld(ld_x, cols) || !valid_ld(ld_y, cols))
    return GEMM_STATUS_INVALID_VALUE;
  if (!std::isfinite(eps) || eps < 0.f) return GEMM_STATUS_NOT_SUPPORTED;
  if (rows == 0 || cols == 0) return GEMM_STATUS_SUCCESS;
  if (!x || !y) return GEMM_STATUS_INVALID_VALUE;
  OnDevice on(v.device);
  if (!on.ok) return GEMM_STATUS_INTERNAL;
  NormArgs a{};
  a.rows = rows;
  a.cols = (int)cols;
  a.x = x;
  a.ldx = ld_x;
  a.x_kind = x_type;
  a.gamma = gamma;
  a.beta = beta;
  a.w_kind = weight_type;
  a.mean = mean;
  a.rstd = rstd;
  a.eps = eps;
  a.y = y;
  a.ldy = ld_y;
  a.y_kind = y_type;
  return status(launch_layernorm(a, v.stream));
}

gemm_status_t gemm_layernorm_grad(gemm_handle_t h, int64_t rows, int64_t cols, const void* dy, int64_t ld_dy,
                                  int y_type, const void* x, int64_t ld_x, int x_type, const float* mean,
                                  const float* rstd, const void* gamma, int weight_type, const void* residual,
                                  int64_t ld_residual, void* dx, int64_t ld_dx, float* dgamma, float* dbeta) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  if (!valid_size(rows) || !valid_size(cols) || !valid_type(x_type) || !valid_type(y_type) ||
      (gamma && !valid_type(weight_type)) || !valid_ld(ld_dy, cols) || !valid_ld(ld_x, cols) ||
      (residual && !valid_ld(ld_residual, cols)) || !valid_ld(ld_dx, cols))
    return GEMM_STATUS_INVALID_VALUE;
  if (cols == 0) return GEMM_STATUS_SUCCESS;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return GEMM_STATUS_INVALID_VALUE;
  OnDevice on(v.device);
  if (!on.ok) return GEMM_STATUS_INTERNAL;
  const bool sums = dgamma || dbeta;
  // the sums' two sets of columns in one launch: the first output carries dgamma
  float* const part = (float*)v.ws;
  auto add_up = [&](int parts) {
    return launch_colsum(part, parts, 2 * whole8(cols), cols, dgamma, dbeta, 0, v.stream);
  };
  if (rows == 0) return sums ? status(add_up(0)) : GEMM_STATUS_SUCCESS;
  const int mp = sums ? max_parts(v, 2 * whole8(cols)) : 0;
  if (sums && mp < 1) return GEMM_STATUS_NOT_SUPPORTED;
  NormArgs a{};
  a.rows = rows;
  a.cols = (int)cols;
  a.x = x;
  a.ldx = ld_x;
  a.x_kind = x_type;
  a.gamma = gamma;
  a.w_kind = weight_type;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.y = dx;
  a.ldy = ld_dx;
  a.y_kind = y_type;
  a.dy = dy;
  a.lddy = ld_dy;
  a.dr = residual;
  a.lddr = ld_residual;
  a.part = sums ? part : nullptr;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  int parts = 0;
  hipError_t e = launch_layernorm_grad(a, mp, &parts, v.stream);
  if (e == hipSuccess && parts) e = add_up(parts);
  return status(e);
}

}  // extern "C"
