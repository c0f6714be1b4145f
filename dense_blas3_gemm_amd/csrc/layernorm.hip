// Layer norm and its gradient, fp32 statistics.
//
//   forward   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) r gamma + beta
//   gradient  xh = (x - mu) r, g = dy gamma,
//             dx = r (g - mean(g) - xh mean(g xh)) [+ dr],
//             dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
#include "epilogue.h"

namespace dbgemm {
namespace {

__device__ __forceinline__ float ln_load(const void* p, int64_t i, int kind) {
  return kind == T_F32 ? ((const float*)p)[i] : ep_bf16f(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void ln_store(void* p, int64_t i, int kind, float v) {
  if (kind == T_F32)
    ((float*)p)[i] = v;
  else
    ((uint16_t*)p)[i] = ep_f32bf(v);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
// Sums of two values over a workgroup of 256 threads, the same in every thread.
__device__ __forceinline__ void group_sum(float& u, float& v, float (*s)[2]) {
  u = wave_sum(u);
  v = wave_sum(v);
  __syncthreads();  // the previous use of s is over
  if ((threadIdx.x & 63) == 0) {
    s[threadIdx.x >> 6][0] = u;
    s[threadIdx.x >> 6][1] = v;
  }
  __syncthreads();
  u = s[0][0] + s[1][0] + s[2][0] + s[3][0];
  v = s[0][1] + s[1][1] + s[2][1] + s[3][1];
}

// One workgroup to a row, which is read three times (any width).
__global__ __launch_bounds__(256) void layernorm_rows_kernel(NormArgs a) {
  __shared__ float s[4][2];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float sum = 0.f, none = 0.f, sq = 0.f;
    for (int i = threadIdx.x; i < a.cols; i += 256) sum += ln_load(a.x, r * a.ldx + i, a.x_kind);
    group_sum(sum, none, s);
    const float mu = sum / (float)a.cols;
    for (int i = threadIdx.x; i < a.cols; i += 256) {
      const float d = ln_load(a.x, r * a.ldx + i, a.x_kind) - mu;
      sq += d * d;
    }
    group_sum(sq, none, s);
    const float rs = 1.0f / __builtin_sqrtf(sq / (float)a.cols + a.eps);
    for (int i = threadIdx.x; i < a.cols; i += 256) {
      float v = (ln_load(a.x, r * a.ldx + i, a.x_kind) - mu) * rs;
      if (a.gamma) v *= ln_load(a.gamma, i, a.w_kind);
      if (a.beta) v += ln_load(a.beta, i, a.w_kind);
      ln_store(a.y, r * a.ldy + i, a.y_kind, v);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mu;
      if (a.rstd) a.rstd[r] = rs;
    }
  }
}

// dx: one workgroup to a row, read twice.
__global__ __launch_bounds__(256) void layernorm_dx_kernel(NormArgs a) {
  __shared__ float s[4][2];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float mu = a.mean[r], rs = a.rstd[r];
    float c1 = 0.f, c2 = 0.f;
    for (int i = threadIdx.x; i < a.cols; i += 256) {
      float g = ln_load(a.dy, r * a.lddy + i, a.y_kind);
      if (a.gamma) g *= ln_load(a.gamma, i, a.w_kind);
      c1 += g;
      c2 += g * ((ln_load(a.x, r * a.ldx + i, a.x_kind) - mu) * rs);
    }
    group_sum(c1, c2, s);
    c1 /= (float)a.cols;
    c2 /= (float)a.cols;
    for (int i = threadIdx.x; i < a.cols; i += 256) {
      float g = ln_load(a.dy, r * a.lddy + i, a.y_kind);
      if (a.gamma) g *= ln_load(a.gamma, i, a.w_kind);
      const float xh = (ln_load(a.x, r * a.ldx + i, a.x_kind) - mu) * rs;
      float v = rs * (g - c1 - xh * c2);
      if (a.dr) v += ln_load(a.dr, r * a.lddr + i, a.x_kind);
      ln_store(a.y, r * a.ldy + i, a.x_kind, v);
    }
  }
}

// Partial sums of dgamma and dbeta: a thread to a column, workgroup row y takes rows y, y +
// gridDim.y, ...
__global__ __launch_bounds__(256) void layernorm_dw_kernel(NormArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.cols) return;
  float dg = 0.f, db = 0.f;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float dy = ln_load(a.dy, r * a.lddy + i, a.y_kind);
    dg += dy * ((ln_load(a.x, r * a.ldx + i, a.x_kind) - a.mean[r]) * a.rstd[r]);
    db += dy;
  }
  a.part[((int64_t)blockIdx.y * 2) * a.cols + i] = dg;
  a.part[((int64_t)blockIdx.y * 2 + 1) * a.cols + i] = db;
}

}  // namespace

hipError_t launch_layernorm(const NormArgs& a, hipStream_t s) {
  const unsigned g = (unsigned)(a.rows < 65536 ? a.rows : 65536);
  hipLaunchKernelGGL(layernorm_rows_kernel, dim3(g), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_layernorm_grad(const NormArgs& a, int max_parts, int* parts, hipStream_t s) {
  const unsigned g = (unsigned)(a.rows < 65536 ? a.rows : 65536);
  // dx may overwrite dr: the weights' sums read neither
  hipLaunchKernelGGL(layernorm_dx_kernel, dim3(g), dim3(256), 0, s, a);
  *parts = 0;
  if (a.part) {
    *parts = (int)(a.rows < max_parts ? a.rows : max_parts);
    hipLaunchKernelGGL(layernorm_dw_kernel, dim3((unsigned)((a.cols + 255) / 256), (unsigned)*parts), dim3(256), 0, s,
                       a);
  }
  return hipGetLastError();
}

}  // namespace dbgemm
