// C-ABI of the gated feed-forward operators and of the 8-bit integer products (include/gemm.h):
// argument checks, workspace and launches.
#include "gemm.h"

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <string>
#include <type_traits>

#include "gated_internal.h"
#include "mlp_host.h"

using namespace dbgemm;

namespace {

// What an epilogue reads past the caches (GatedEp::past, with both sides measured): half of them.
constexpr double kPastBytes = (double)(128 << 20);

// Columns that the generic kernels take in a launch: a launch ends at 2^32 threads, the one for few
// elements (8 columns to 256 threads) at 2^27 columns.
constexpr int64_t kSimtCols = (int64_t)1 << 26;
// and where a partial row of column sums of all of them does not fit the workspace (from 2^23 on): two do
constexpr int64_t kSimtSumCols = (int64_t)1 << 22;

// Longest sum of products of two 8-bit integers (at most 2^14 each) that 32 bits hold.
constexpr int64_t kMaxK8 = 131071;

// bytes per element of the operands, of C
int64_t in_bytes(const GatedArgs& a) { return a.in_kind == GT_BF16 ? 2 : 1; }
int64_t c_bytes(const GatedArgs& a) { return a.c_kind == C_F32 ? 4 : 2; }

// a's rows [m0, m0 + M) and columns [n0, n0 + N)
GatedArgs part_of(const GatedArgs& a, int64_t m0, int64_t n0, int64_t M, int64_t N) {
  GatedArgs r = a;
  const int64_t es = in_bytes(a), ce = c_bytes(a), be = a.ep.bias_f32 ? 4 : 2;
  auto at = [](auto*& p, int64_t bytes) {
    if (p) p = (std::remove_reference_t<decltype(p)>)((const char*)p + bytes);
  };
  r.M = (int)M;
  r.N = (int)N;
  at(r.A, m0 * a.lda * es);
  at(r.B, (a.transB ? n0 * a.ldb : n0) * es);
  at(r.B2, (a.transB ? n0 * a.ldb2 : n0) * es);
  at(r.C, (m0 * a.ldc + n0) * ce);
  at(r.ep.bias, n0 * be);
  at(r.ep.bias2, n0 * be);
  at(r.ep.sa, m0 * 4);
  at(r.ep.sb, n0 * 4);
  at(r.ep.sb2, n0 * 4);
  at(r.ep.R, (m0 * a.ep.ldr + n0) * ce);
  at(r.ep.G, (m0 * a.ep.ldg + n0) * 2);
  at(r.ep.U, (m0 * a.ep.ldu + n0) * 2);
  at(r.ep.D2, (m0 * a.ep.ldd2 + n0) * ce);
  at(r.ep.H, (m0 * a.ep.ldh + n0) * 2);
  return r;
}

// The columns of a launch of the generic kernels over all of a.
int64_t simt_cols(const HandleView& v, const GatedArgs& a, bool sums) {
  const int64_t most = a.N < kSimtCols ? a.N : kSimtCols;
  return sums && max_parts(v, 2 * whole8(most)) < 1 && most > kSimtSumCols ? kSimtSumCols : most;
}

// The generic kernels over all of a; dbias: fp32 column sums, the second set from dbias2.
gemm_status_t run_simt(const HandleView& v, const GatedArgs& all, float* dbias, float* dbias2) {
  const bool sums = dbias || dbias2;
  const int64_t most = simt_cols(v, all, sums);
  const int mp = sums ? max_parts(v, 2 * whole8(most)) : 1;
  if (mp < 1) return GEMM_STATUS_NOT_SUPPORTED;
  for (int64_t n0 = 0; n0 < all.N; n0 += most) {
    const int64_t N = all.N - n0 < most ? all.N - n0 : most;
    GatedArgs a = part_of(all, 0, n0, all.M, N);
    a.ep.colsum = sums ? (float*)v.ws : nullptr;
    int parts = 0;
    hipError_t e = launch_gated_simt(a, mp, &parts, v.stream);
    if (e == hipSuccess && sums)
      e = launch_colsum((const float*)v.ws, parts, 2 * whole8(N), N, dbias ? dbias + n0 : nullptr,
                        dbias2 ? dbias2 + n0 : nullptr, 0, v.stream);
    if (e != hipSuccess) return status(e);
  }
  return GEMM_STATUS_SUCCESS;
}

// One launch on policy p with sp splits; partial column sums into ep.colsum, *parts rows of them.
hipError_t run_tiles(const HandleView& v, GatedArgs a, const Policy& p, int sp, int* parts) {
  const int64_t cols = a.op == GT_GATED ? p.BN / 2 : p.BN;
  a.tiles_m = (a.M + p.BM - 1) / p.BM;
  a.tiles_n = (int)((a.N + cols - 1) / cols);
  a.group = p.group;
  a.raster_n = p.raster_n;
  a.xcd = p.xcd;
  a.swizzle = p.swizzle;
  a.splits = sp;
  a.kt_per_split = (int)split_kt(p, a.in_kind == GT_I8 ? (a.K + 1) / 2 : a.K, sp);
  a.ws = sp > 1 ? (float*)v.ws : nullptr;
  return launch_mfma_gated(p, a, parts, v.stream);
}

// The partial rows of column sums that run_tiles leaves: a row of waves each, or after a split a
// row of fragments.
int64_t partial_rows(const Policy& p, int64_t M, int sp) {
  return (M + p.BM - 1) / p.BM * (sp > 1 ? p.BM / p.WM / 16 : p.WM);
}

// What the tile policies see of a: a product of both B side by side; 8-bit integers as bf16 of
// half the K (the same bytes, and the integer MFMA takes as long for them).
Problem problem_of(const GatedArgs& a) {
  Problem pr{};
  pr.transB = a.transB;
  pr.M = a.M;
  pr.N = a.op == GT_GATED ? 2 * (int64_t)a.N : a.N;
  pr.K = a.in_kind == GT_I8 ? (a.K + 1) / 2 : a.K;
  pr.in_fp8 = a.in_kind == GT_E4M3;
  pr.c_kind = a.c_kind;
  pr.fast_ok = true;
  pr.ep = true;
  pr.products = a.op == GT_GATED ? 2 : 1;
  pr.elem = (int)in_bytes(a);
  return pr;
}

// Whether the MFMA kernels take the operands: 16-byte aligned, strides and contiguous extents in
// whole 16 bytes (`cols`: of B's columns), and spans that 32-bit offsets cover.
bool operands_ok(const GatedArgs& a, int64_t cols) {
  const int64_t es = in_bytes(a), vec = 16 / es;
  auto fits = [&](const void* p, int64_t ld, int64_t rows) {
    return ((uintptr_t)p & 15) == 0 && ld * es % 16 == 0 && (double)(rows + 256) * (double)ld * (double)es < 2147483647.0;
  };
  const int64_t b_rows = a.transB ? a.N : a.K;
  return a.K % vec == 0 && (a.transB || cols % vec == 0) && fits(a.A, a.lda, a.M) && fits(a.B, a.ldb, b_rows) &&
         (a.op != GT_GATED || fits(a.B2, a.ldb2, b_rows));
}

// The tile model's cost (2e6 units to about a microsecond) as the time of a call of a few rows,
// each kind with its own factor: a fit, 9 to 10 % off in the mean square, so that near ties may go to the
// slower side (24 x 13696 x 5120 of 8-bit integers, both B [N][K]: 32.5 us on the tiles that are chosen,
// 29.5 on the few-row kernel).  Column sums are one more launch.
double tiles_us(int in_kind, double cost, bool sums) {
  const double factor = in_kind == GT_BF16 ? 0.77 : in_kind == GT_E4M3 ? 0.64 : 0.79;
  return 3.6 + factor * cost / 2.0e6 + (sums ? 4.0 : 0.0);
}
// (no tile's time is less: the search among them is a microsecond of the host's)
constexpr double kLeastTilesUs = 5.0;

// How a product of whole eights of columns is run on the MFMA kernels.
struct Choice {
  bool ok = false;   // not: they, or the workspace, cannot
  int few_cols = 0;  // the few-row kernel at this width, or
  int idx = 0, sp = 1;
  Cut cut;  // two launches, the second one's
  int idx2 = 0, sp2 = 1;
  GatedArgs a1, a2;
  int64_t floats1 = 0, floats2 = 0;  // of partial column sums
};

// accumulate: the sums are added to those of other rows.
Choice choose(const HandleView& v, const GatedArgs& a, bool sums, bool accumulate) {
  Choice c;
  const int nb = a.op == GT_GATED ? 2 : 1;
  double cost = 0.0;
  const int64_t split_floats = v.ws ? (int64_t)(kPartBytes / sizeof(float)) : 0;
  // a few rows: their own kernel where its time by its model is less than any tile's, or than the
  // chosen ones'
  int few_cols = 0;
  const double few = !accumulate && a.M <= kFewRows
                         ? few_rows_us(a.op, a.in_kind, a.transB, a.M, a.N, a.K, v.cu_count, &few_cols)
                         : 0.0;
  if (few_cols && few < kLeastTilesUs) {
    c.ok = true;
    c.few_cols = few_cols;
    return c;
  }
  Problem pr = problem_of(a);
  c.idx = policy_select(pr, v.cu_count, split_floats, &c.sp, &cost);
  if (policy_at(c.idx).kind != KIND_MFMA) return c;
  if (few_cols && few < tiles_us(a.in_kind, cost, sums)) {
    c.ok = true;
    c.few_cols = few_cols;
    return c;
  }
  c.cut = policy_cut(pr, v.cu_count, split_floats, cost);
  c.a1 = a;
  if (c.cut.p >= 0) {
    const int64_t at = c.cut.at = c.cut.by_rows ? c.cut.at : c.cut.at / nb;
    c.a1 = c.cut.by_rows ? part_of(a, 0, 0, at, a.N) : part_of(a, 0, 0, a.M, at);
    c.a2 = c.cut.by_rows ? part_of(a, at, 0, a.M - at, a.N) : part_of(a, 0, at, a.M, a.N - at);
    c.idx = c.cut.p;
    c.sp = 1;
    pr.M = c.a2.M;
    pr.N = (int64_t)c.a2.N * nb;
    c.idx2 = policy_select(pr, v.cu_count, split_floats, &c.sp2);
    if (policy_at(c.idx2).kind != KIND_MFMA) return c;
  }
  if (sums) {
    c.floats1 = partial_rows(policy_at(c.idx), c.a1.M, c.sp) * 2 * c.a1.N;
    if (c.cut.p >= 0) c.floats2 = partial_rows(policy_at(c.idx2), c.a2.M, c.sp2) * 2 * c.a2.N;
    if (!v.ws || v.ws_bytes < kPartBytes + (size_t)(c.floats1 + c.floats2) * sizeof(float)) return c;
  }
  c.ok = true;
  return c;
}

// c's launches; accumulate: the sums are added to dbias and dbias2.
hipError_t run_choice(const HandleView& v, GatedArgs a, Choice& c, float* dbias, float* dbias2, int accumulate) {
  if (c.few_cols) {
    a.ep.sum1 = dbias;
    a.ep.sum2 = dbias2;
    return launch_gated_skinny(a, c.few_cols, v.stream);
  }
  const bool sums = dbias || dbias2;
  if (sums) {
    c.a1.ep.colsum = (float*)((char*)v.ws + kPartBytes);
    c.a2.ep.colsum = c.a1.ep.colsum + c.floats1;
  }
  auto add_up = [&](const GatedArgs& p, int parts, int64_t n0) {
    return launch_colsum(p.ep.colsum, parts, 2 * (int64_t)p.N, p.N, dbias ? dbias + n0 : nullptr,
                         dbias2 ? dbias2 + n0 : nullptr, accumulate, v.stream);
  };
  const bool two = c.cut.p >= 0;
  int parts = 0, parts2 = 0;
  hipError_t e = run_tiles(v, c.a1, policy_at(c.idx), c.sp, &parts);
  if (two && e == hipSuccess) e = run_tiles(v, c.a2, policy_at(c.idx2), c.sp2, &parts2);
  if (!sums || e != hipSuccess) return e;
  if (two && c.cut.by_rows) return add_up(c.a1, parts + parts2, 0);  // (the rows of both follow each other)
  e = add_up(c.a1, parts, 0);
  if (two && e == hipSuccess) e = add_up(c.a2, parts2, c.cut.at);
  return e;
}

// The columns of the MFMA kernels, whole eights (of [K][N] operands whole 16 bytes; the generic kernels
// have the rest), and the rows of a call on them that 32-bit offsets into A cover and whose partial column
// sums (at most one row of them to 32 rows) the workspace holds, whole tiles of them; no columns where
// those kernels do not take the operands.
struct Blocks {
  int64_t cols = 0, rows = 0;
};
Blocks blocks_of(const HandleView& v, const GatedArgs& a, bool sums) {
  Blocks b;
  const int64_t step = a.transB ? 8 : 16 / in_bytes(a), N1 = a.K > 0 ? a.N / step * step : 0;
  if (N1 == 0) return b;
  int64_t most = (int64_t)(2147483647.0 / ((double)a.lda * (double)in_bytes(a))) / 256 * 256 - 512;
  if (sums && v.ws) {
    const int64_t fit = (int64_t)((v.ws_bytes - kPartBytes) / sizeof(float)) / (2 * N1) * 32 / 256 * 256 - 512;
    if (fit >= 1 && fit < most) most = fit;
  }
  b.rows = most >= a.M ? a.M : most;
  if (b.rows >= 1 && operands_ok(part_of(a, 0, 0, b.rows, a.N), N1)) b.cols = N1;
  return b;
}

gemm_status_t run(gemm_handle_t h, GatedArgs a, float* dbias = nullptr, float* dbias2 = nullptr) {
  HandleView v;
  if (!handle_view(h, &v)) return GEMM_STATUS_NOT_INITIALIZED;
  OnDevice on(v.device);
  if (!on.ok) return GEMM_STATUS_INTERNAL;
  const bool sums = dbias || dbias2;
  if (a.M == 0 || a.N == 0) {  // no element; the sums over no rows are zeros
    if (!sums || a.N == 0) return GEMM_STATUS_SUCCESS;
    return status(launch_colsum(nullptr, 0, 2 * whole8(a.N), a.N, dbias, dbias2, 0, v.stream));
  }
  if (a.alpha == 0.f) a.K = 0;
  a.ep.past = (double)a.M * a.N * (a.op == GT_GRAD ? 4 : a.ep.R ? (double)c_bytes(a) : 0) >= kPastBytes;
  const Blocks b = blocks_of(v, a, sums);
  if (b.cols == 0) return run_simt(v, a, dbias, dbias2);
  for (int64_t m0 = 0; m0 < a.M; m0 += b.rows) {
    const GatedArgs part = part_of(a, m0, 0, a.M - m0 < b.rows ? a.M - m0 : b.rows, b.cols);
    Choice c = choose(v, part, sums, m0 > 0);
    if (!c.ok) {
      if (m0 > 0) return GEMM_STATUS_INTERNAL;
      return run_simt(v, a, dbias, dbias2);
    }
    const hipError_t e = run_choice(v, part, c, dbias, dbias2, m0 > 0);
    if (e != hipSuccess) return status(e);
  }
  if (b.cols == a.N) return GEMM_STATUS_SUCCESS;
  return run_simt(v, part_of(a, 0, b.cols, a.M, a.N - b.cols), dbias ? dbias + b.cols : nullptr,
                  dbias2 ? dbias2 + b.cols : nullptr);
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

namespace dbgemm {
hipError_t launch_mfma_gated(const Policy& p, const GatedArgs& a, int* parts, hipStream_t s) {
#define DBGEMM_GT_CASE(in, b) \
  return p.pipe == 2 ? launch_mfma_pp_gt_##in##b(p, a, parts, s) : launch_mfma_dma_gt_##in##b(p, a, parts, s)
  switch (a.in_kind * 2 + (a.transB != 0)) {
    case 0: DBGEMM_GT_CASE(0, 0);
    case 1: DBGEMM_GT_CASE(0, 1);
    case 2: DBGEMM_GT_CASE(1, 0);
    case 3: DBGEMM_GT_CASE(1, 1);
    case 4: DBGEMM_GT_CASE(2, 0);
    default: DBGEMM_GT_CASE(2, 1);
  }
#undef DBGEMM_GT_CASE
}
}  // namespace dbgemm

extern "C" {

int dbgemm_gated_plan(int op, int in_kind, int transB, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                      int64_t ldb2, int sums, int cu_count, char* text, size_t len) {
  if (!text || len == 0 || M < 1 || N < 1 || K < 0) return 1;
  HandleView v{};
  v.cu_count = cu_count;
  v.ws = (void*)0x1000;  // (never dereferenced, as the operands')
  v.ws_bytes = kWorkspaceBytes;
  GatedArgs a{};
  a.A = a.B = a.B2 = a.C = (void*)0x1000;
  a.lda = lda;
  a.ldb = ldb;
  a.ldb2 = ldb2;
  a.ldc = N;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.transB = transB;
  a.op = op;
  a.in_kind = in_kind;
  std::string s;
  auto add = [&](const std::string& kernel, const GatedArgs& p) {
    s += (s.empty() ? "" : "; ") + kernel + " " + std::to_string(p.M) + "x" + std::to_string(p.N);
  };
  auto tiles = [](int idx, int sp) { return std::string(policy_at(idx).name) + (sp > 1 ? "+sk" + std::to_string(sp) : ""); };
  auto simt = [&](const GatedArgs& all) {
    const int64_t most = simt_cols(v, all, sums);
    for (int64_t n0 = 0; n0 < all.N; n0 += most) {
      const GatedArgs p = part_of(all, 0, n0, all.M, all.N - n0 < most ? all.N - n0 : most);
      add(gated_simt_thin(p) ? "simt_thin" : "simt_tiles", p);
    }
  };
  const Blocks b = blocks_of(v, a, sums);
  bool ok = b.cols > 0;
  for (int64_t m0 = 0; ok && m0 < M; m0 += b.rows) {
    const GatedArgs part = part_of(a, m0, 0, M - m0 < b.rows ? M - m0 : b.rows, b.cols);
    const Choice c = choose(v, part, sums, m0 > 0);
    ok = c.ok;
    if (!ok) break;
    if (c.few_cols)
      add("few_rows_n" + std::to_string(c.few_cols), part);
    else
      add(tiles(c.idx, c.sp), c.a1);
    if (!c.few_cols && c.cut.p >= 0) add(tiles(c.idx2, c.sp2), c.a2);
  }
  if (!ok)
    simt(a);
  else if (b.cols < N)
    simt(part_of(a, 0, b.cols, M, N - b.cols));
  std::snprintf(text, len, "%s", s.c_str());
  return s.size() < len ? 0 : 1;
}

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
