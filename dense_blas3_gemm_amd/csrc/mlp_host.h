// Host-side pieces that the entry points of the MLP-block and gated operators share.
#pragma once

#include "blas3_internal.h"
#include "mlp_internal.h"

namespace dbgemm {
namespace {

// The workspace: partial column sums, or a split product's partial tiles, first; behind them a
// product in fp32, or the column sums of a product with an epilogue.
constexpr size_t kPartBytes = (size_t)64 << 20;
constexpr int kMaxParts = 1024;

// Makes the handle's device current for its lifetime.
struct OnDevice {
  int cur = -1;
  int dev;
  bool ok;
  explicit OnDevice(int device) : dev(device) {
    ok = hipGetDevice(&cur) == hipSuccess && (cur == device || hipSetDevice(device) == hipSuccess);
  }
  ~OnDevice() {
    if (ok && cur != dev) (void)hipSetDevice(cur);
  }
};

gemm_status_t status(hipError_t e) { return e == hipSuccess ? GEMM_STATUS_SUCCESS : GEMM_STATUS_LAUNCH_FAILED; }

bool valid_act(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }
bool valid_type(int t) { return t == GEMM_TYPE_BF16 || t == GEMM_TYPE_F32; }
bool valid_size(int64_t v) { return v >= 0 && v <= 0x7FFFFFFF; }
bool valid_ld(int64_t ld, int64_t cols) { return ld >= (cols > 1 ? cols : 1); }

// partial rows of `width` floats that fit the workspace's first part, at most kMaxParts
int max_parts(const HandleView& v, int64_t width) {
  if (!v.ws || width <= 0) return 0;
  const int64_t n = (int64_t)(kPartBytes / sizeof(float)) / width;
  return (int)(n < kMaxParts ? n : kMaxParts);
}

}  // namespace
}  // namespace dbgemm
