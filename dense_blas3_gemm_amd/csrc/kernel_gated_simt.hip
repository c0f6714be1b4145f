// The gated operators' products for any sizes, strides and alignments (the MFMA kernels take
// whole 16-byte pieces), and the columns that those leave: 64 x 64 tiles on the VALU, sums in
// fp32 or (8-bit integers) in exact 32-bit integers, then the epilogue element by element.
//
// Bound by the LDS and the VALU, and meant for what the other kernels cannot take, or for a few
// columns.
#include "epilogue.h"
#include "gated_internal.h"

namespace dbgemm {
namespace {

constexpr int TS = 64;  // tile edge
constexpr int TK = 16;  // K step

template <bool INT>
__device__ __forceinline__ auto gs_load(const void* p, int64_t i, int e4m3) {
  if constexpr (INT)
    return (int)((const int8_t*)p)[i];
  else
    return e4m3 ? __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)p)[i], 0) : ep_bf16f(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ float gs_value(const void* p, int64_t i, int f32) {
  return f32 ? ((const float*)p)[i] : ep_bf16f(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void gs_store(void* p, int64_t i, int f32, float v) {
  if (f32)
    ((float*)p)[i] = v;
  else
    ((uint16_t*)p)[i] = ep_f32bf(v);
}

// 256 threads = 16 x 16, each with rows ty + 16 i and columns tx + 16 j of a tile.  A workgroup
// takes the row tiles blockIdx.y, + gridDim.y, ... of its columns, whose sums it keeps.
template <bool INT, int OP>
__global__ __launch_bounds__(256) void gated_simt_kernel(GatedArgs a) {
  using T = std::conditional_t<INT, int, float>;
  constexpr int NB = OP == GT_GATED ? 2 : 1;
  __shared__ T As[TK][TS + 1];
  __shared__ T Bs[NB][TK][TS + 1];
  const GatedEp& e = a.ep;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t n0 = (int64_t)blockIdx.x * TS, tiles_m = ((int64_t)a.M + TS - 1) / TS;
  float cs[2][4] = {};
  for (int64_t tm = blockIdx.y; tm < tiles_m; tm += gridDim.y) {
    const int64_t m0 = tm * TS;
    T acc[NB][4][4] = {};
    for (int64_t k0 = 0; k0 < a.K; k0 += TK) {
      for (int x = threadIdx.x; x < TK * TS; x += 256) {
        {  // neighbouring threads on neighbouring addresses
          const int kk = x % TK, r = x / TK;
          const int64_t k = k0 + kk, m = m0 + r;
          As[kk][r] = k < a.K && m < a.M ? gs_load<INT>(a.A, m * a.lda + k, a.in_fp8) : T(0);
        }
        const int kk = a.transB ? x % TK : x / TS, r = a.transB ? x / TK : x % TS;
        const int64_t k = k0 + kk, n = n0 + r;
        const bool in = k < a.K && n < a.N;
        Bs[0][kk][r] = in ? gs_load<INT>(a.B, a.transB ? n * a.ldb + k : k * a.ldb + n, a.in_fp8) : T(0);
        if constexpr (NB == 2)
          Bs[1][kk][r] = in ? gs_load<INT>(a.B2, a.transB ? n * a.ldb2 + k : k * a.ldb2 + n, a.in_fp8) : T(0);
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < TK; ++kk)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][i][j] += As[kk][ty + 16 * i] * Bs[b][kk][tx + 16 * j];
      __syncthreads();
    }
    ep_with_act(e.act, [&](auto ac) EP_INLINE {
      constexpr int ACT = decltype(ac)::value;
      const bool f32 = a.c_kind == C_F32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty + 16 * i;
        if (m >= a.M) continue;
        const float sa = INT ? e.sa[m] : a.alpha;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = n0 + tx + 16 * j;
          if (n >= a.N) continue;
          float w = (float)acc[0][i][j] * sa;
          if constexpr (INT) w *= e.sb[n];
          if constexpr (OP == GT_GRAD) {
            const float g = ep_bf16f(((const uint16_t*)e.G)[m * e.ldg + n]);
            const float u = ep_bf16f(((const uint16_t*)e.U)[m * e.ldu + n]);
            const float h = ep_act<ACT>(g), dg = w * u * ep_slope<ACT>(g), du = w * h;
            gs_store(a.C, m * a.ldc + n, f32, dg);
            gs_store(e.D2, m * e.ldd2 + n, f32, du);
            if (e.H) gs_store(e.H, m * e.ldh + n, 0, h * u);
            cs[0][j] += dg;
            cs[1][j] += du;
          } else {
            if (e.bias) w += gs_value(e.bias, n, e.bias_f32);
            float c = ep_act<ACT>(w);
            if constexpr (OP == GT_GATED) {
              float w2 = (float)acc[NB - 1][i][j] * sa;
              if constexpr (INT) w2 *= e.sb2[n];
              if (e.bias2) w2 += gs_value(e.bias2, n, e.bias_f32);
              if (e.G) gs_store(e.G, m * e.ldg + n, 0, w);
              if (e.U) gs_store(e.U, m * e.ldu + n, 0, w2);
              c *= w2;
            } else if (e.R) {
              c += e.beta * gs_value(e.R, m * e.ldr + n, f32);
            }
            gs_store(a.C, m * a.ldc + n, f32, c);
          }
        }
      }
    });
  }
  if constexpr (OP == GT_GRAD) {
    if (!e.colsum) return;
    __shared__ float sums[2][16][TS];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[s][ty][tx + 16 * j] = cs[s][j];
    __syncthreads();
    if (threadIdx.x < 2 * TS) {
      const int s = threadIdx.x / TS, x = threadIdx.x % TS;
      float v = 0.f;
#pragma unroll
      for (int y = 0; y < 16; ++y) v += sums[s][y][x];
      if (n0 + x < a.N) e.colsum[((int64_t)blockIdx.y * 2 + s) * whole8(a.N) + n0 + x] = v;
    }
  }
}

}  // namespace

hipError_t launch_gated_simt(const GatedArgs& a, int max_parts, int* parts, hipStream_t s) {
  const int64_t tm = ((int64_t)a.M + TS - 1) / TS, tn = ((int64_t)a.N + TS - 1) / TS;
  int64_t gy = tm < 65535 ? tm : 65535;
  if (a.ep.colsum && gy > max_parts) gy = max_parts;
  if (gy < 1 || tn < 1) return hipErrorInvalidConfiguration;
  *parts = (int)gy;
  const dim3 grid((unsigned)tn, (unsigned)gy);
  const bool i8 = a.in_kind == GT_I8;
  if (a.op == GT_GRAD && !i8)
    hipLaunchKernelGGL((gated_simt_kernel<false, GT_GRAD>), grid, dim3(256), 0, s, a);
  else if (a.op == GT_GATED && !i8)
    hipLaunchKernelGGL((gated_simt_kernel<false, GT_GATED>), grid, dim3(256), 0, s, a);
  else if (a.op == GT_GATED)
    hipLaunchKernelGGL((gated_simt_kernel<true, GT_GATED>), grid, dim3(256), 0, s, a);
  else if (a.op == GT_LINEAR && i8)
    hipLaunchKernelGGL((gated_simt_kernel<true, GT_LINEAR>), grid, dim3(256), 0, s, a);
  else
    return hipErrorInvalidConfiguration;
  return hipGetLastError();
}

}  // namespace dbgemm
