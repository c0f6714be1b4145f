// The epilogue of a product's tile, from the MFMA kernels' accumulators: the tile goes through
// LDS in whole rows (written straight from 16x16 fragments, one instruction would touch 16
// rows x 32 bytes), eight columns to a thread.  Included by the kernels' translation units
// when they are built for products with an epilogue (DBGEMM_EPILOGUE).
#pragma once

#include "epilogue.h"
#include "mfma_common.h"

namespace dbgemm {
namespace {

// The column sums of the workgroup's rows: thread t holds those of columns 8 (t % CH) .. + 7
// over its rows; the THREADS / CH sets are added in order through LDS (16 KiB at most) and one
// partial row of the tile's columns is written.
template <int THREADS, int BN>
__device__ __forceinline__ void ep_put_colsum(const GemmEpArgs& a, const float (&cs)[8], int64_t part, int n0, int t,
                                              uint32_t lds0) {
  constexpr int CH = BN / 8, SETS = THREADS / CH;
  __syncthreads();  // the LDS is free again
  const uint32_t at = lds0 + (uint32_t)((t / CH) * BN * 4 + (t % CH) * 32);
  *(__attribute__((address_space(3))) f32x4*)(uintptr_t)at = (f32x4){cs[0], cs[1], cs[2], cs[3]};
  *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(at + 16) = (f32x4){cs[4], cs[5], cs[6], cs[7]};
  __syncthreads();
  if (t < BN && n0 + t < a.N) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < SETS; ++k)
      v += *(__attribute__((address_space(3))) float*)(uintptr_t)(lds0 + (uint32_t)(k * BN * 4 + t * 4));
    a.ep.colsum[part * a.N + n0 + t] = v;
  }
}

// acc: the 16x16 fragments of wave (wm, wn), alpha not applied.  One pass per row of waves:
// they write alpha * acc as fp32 to LDS (16-byte chunks XOR-swizzled by row, so that the
// sixteen rows of a fragment store spread over the banks), then every thread takes eight
// columns of its rows.  What the rows bring from memory (residual or Z) is asked for before
// the pass's barrier, for all of the thread's rows at once.  lds0: LDS of at least WTM x BN
// fp32, free once every wave has passed the first barrier here.
template <class C, bool NT>
__device__ __forceinline__ void ep_tile(const GemmEpArgs& a, const typename AccOf<C::MT>::T (&acc)[C::FM][C::FN],
                                        int m0, int n0, int tm, int wm, int xb0, int lane, int t, uint32_t lds0) {
  static_assert(C::MT == 16 && C::ACC == 4, "16x16 fragments");
  constexpr int RB = C::BN * 4, CH = C::BN / 8, RPS = C::THREADS / CH, STEPS = C::WTM / RPS;
  static_assert(C::WTM % RPS == 0 && C::BN % 64 == 0 && RPS * C::BN * 4 <= C::WTM * RB, "whole steps of rows");
  const int row = t / CH, ch = (t % CH) * 2, n = n0 + (t % CH) * 8;
  const int nvc = min(max(a.N - n, 0), 8);
  const float alpha = a.alpha;
  float cs[8] = {}, b[8];
  ep_bias8(a, n, nvc, b);
  ep_dispatch(a.ep, [&](auto gc, auto ac) {
    constexpr bool GRAD = decltype(gc)::value;
    constexpr int ACT = decltype(ac)::value;
#pragma unroll 1
    for (int g = 0; g < C::WM; ++g) {
      const int mg = m0 + g * C::WTM + row;
      EpRaw raw[STEPS];
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int m = mg + s * RPS;
        ep_fetch8<GRAD>(a, m, n, m < a.M ? nvc : 0, raw[s]);
      }
      __syncthreads();  // the LDS is free: the K loop's reads, or the previous pass's
      if (wm == g) {
        static_for<C::FM * C::FN>([&](auto pc) {
          constexpr int p = decltype(pc)::value;
          constexpr int i = p / C::FN, j = p % C::FN;
          const int r = i * 16 + lane % 16, c = xb0 + j * 16 + 4 * (lane / 16);
          const int chunk = (c >> 2) ^ (r & 15);
          *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(lds0 + (uint32_t)(r * RB + chunk * 16)) =
              (f32x4){alpha * acc[i][j][0], alpha * acc[i][j][1], alpha * acc[i][j][2], alpha * acc[i][j][3]};
        });
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int r = s * RPS + row, m = mg + s * RPS;
        const uint32_t at = lds0 + (uint32_t)(r * RB);
        const f32x4 lo = *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(at + ((ch ^ (r & 15)) * 16));
        const f32x4 hi = *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(at + (((ch + 1) ^ (r & 15)) * 16));
        float w[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        ep_finish8<NT, GRAD, ACT>(a, w, raw[s], b, m, n, m < a.M ? nvc : 0, cs);
      }
    }
  });
  if (a.ep.grad && a.ep.colsum) ep_put_colsum<C::THREADS, C::BN>(a, cs, tm, n0, t, lds0);
}

}  // namespace
}  // namespace dbgemm
