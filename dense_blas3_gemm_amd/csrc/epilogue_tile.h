// The epilogue of a product's tile, from the MFMA kernels' accumulators.  Included by the
// kernels' translation units when they are built for products with an epilogue
// (DBGEMM_EPILOGUE).  N is a multiple of 8 here (the host sends other widths elsewhere): the
// paths of partial eights, in every unrolled row, would cost the 256 x 256 tiles their
// registers.
//
// Every wave puts its own part of the tile through its own part of the LDS, some rows at a
// time, and takes it back in whole rows, eight columns to a lane (written straight from 16x16
// fragments, one instruction would touch 16 rows x 32 bytes).  No wave waits for another, and
// a wave's accumulators are dead once they are in LDS: with the two groups of waves of the
// 256 x 256 tile taking the whole LDS in turn instead, every wave held its 128 accumulators
// through the other group's rows, and the epilogue ran from spilled registers.
//
// What it adds is arithmetic and traffic that nothing of the same CU hides (the 256 x 256 tile
// fills its LDS): 2048 x 20480 x 5120 takes 349 us with no activation, 356 with GELU (tanh), 365 with
// codes, 372 with both; the gradient from codes 368, with bias sums 378.
#pragma once

#include "epilogue.h"
#include "mfma_common.h"

namespace dbgemm {
namespace {

// Rows of a wave's part that go through the LDS at a time: whole fragments, as many as fit.
template <class C, int LDS_BYTES>
constexpr int ep_pass_rows() {
  int rows = C::WTM;
  while (rows > 16 && (rows * C::WTN * 4 * (C::THREADS / 64) > LDS_BYTES || C::WTM % rows != 0)) rows -= 16;
  return rows;
}

// acc: the 16x16 fragments of this wave (wave_m: its row among the tile's waves), alpha not
// applied; its part of C starts at row m0, column n0.  lds0: LDS_BYTES of LDS, free once
// every wave has passed the barrier here.  The 16-byte chunks of an LDS row are XOR-swizzled by
// the row, so that the sixteen rows of a fragment store spread over the banks.  What the rows
// bring from memory (residual or Z) is asked for ahead, up to four steps of rows at a time.
template <class C, int LDS_BYTES, bool NT>
__device__ __forceinline__ void ep_tile(const GemmEpArgs& a, const typename AccOf<C::MT>::T (&acc)[C::FM][C::FN],
                                        int m0, int n0, int part, int wave, int lane, uint32_t lds0) {
  static_assert(C::MT == 16 && C::ACC == 4, "16x16 fragments");
  constexpr int PASS = ep_pass_rows<C, LDS_BYTES>();
  constexpr int RB = C::WTN * 4, CPR = C::WTN / 4;  // bytes and 16-byte chunks of an LDS row
  constexpr int LPR = C::WTN / 8, RPS = 64 / LPR;   // lanes to a row, rows to a step
  constexpr int STEPS = PASS / RPS, BATCH = STEPS < 4 ? STEPS : 4;
  constexpr int ALL = C::WTM / RPS;
  static_assert(PASS * RB * (C::THREADS / 64) <= LDS_BYTES, "a pass of every wave fits");
  static_assert(LPR % 4 == 0 && (CPR & (CPR - 1)) == 0 && PASS % RPS == 0 && STEPS % BATCH == 0,
                "whole blocks of 32 columns, whole steps and batches");
  const uint32_t mine = lds0 + (uint32_t)(wave * PASS * RB);
  const int row = lane / LPR, ch = (lane % LPR) * 2, n = n0 + (lane % LPR) * 8;
  const int nvc = n < a.N ? 8 : 0;
  const float alpha = a.alpha;
  float cs[8] = {}, b[8];
  ep_bias8(a, n, nvc, b);
  ep_dispatch(a.ep, [&](auto mc, auto ac) EP_INLINE {
    constexpr int MODE = decltype(mc)::value;
    constexpr int ACT = decltype(ac)::value;
    EpRaw raw[BATCH];
    auto fetch = [&](int step) EP_INLINE {
      const int m = m0 + row + step * RPS;
      return ep_fetch8<MODE, false>(a, m, n, step < ALL && m < a.M ? nvc : 0);
    };
#pragma unroll
    for (int s = 0; s < BATCH; ++s) raw[s] = fetch(s);
    __syncthreads();  // the LDS is free: the K loop's reads are done
    static_for<C::WTM / PASS>([&](auto hc) EP_INLINE {
      constexpr int h = decltype(hc)::value;
      const int mp = m0 + h * PASS + row;
      static_for<PASS / 16 * C::FN>([&](auto pc) EP_INLINE {
        constexpr int p = decltype(pc)::value;
        constexpr int li = p / C::FN, i = h * (PASS / 16) + li, j = p % C::FN;
        const int r = li * 16 + lane % 16;
        const int chunk = (j * 4 + lane / 16) ^ (r & (CPR - 1));
        *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(mine + (uint32_t)(r * RB + chunk * 16)) =
            (f32x4){alpha * acc[i][j][0], alpha * acc[i][j][1], alpha * acc[i][j][2], alpha * acc[i][j][3]};
      });
#pragma unroll 1
      for (int s0 = 0; s0 < STEPS; s0 += BATCH) {
#pragma unroll
        for (int s = 0; s < BATCH; ++s) {
          const int r = (s0 + s) * RPS + row, m = mp + (s0 + s) * RPS;
          const uint32_t at = mine + (uint32_t)(r * RB), x = (uint32_t)(r & (CPR - 1));
          const f32x4 lo = *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(at + ((ch ^ x) * 16));
          const f32x4 hi = *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(at + (((ch + 1) ^ x) * 16));
          float w[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          ep_finish8<NT, MODE, ACT, false>(a, w, raw[s], b, m, n, m < a.M ? nvc : 0, cs);
          raw[s] = fetch(h * STEPS + s0 + s + BATCH);
        }
      }
    });
  });
  if (a.ep.grad && a.ep.colsum) {
    // the wave's rows of each column: over the lanes that share the columns, then out
#pragma unroll
    for (int o = LPR; o < 64; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] += __shfl_xor(cs[i], o);
    if (lane < LPR && nvc) ep_store8<false, EP_NONE>(a.ep.colsum + (int64_t)part * a.N + n, nvc, cs);
  }
}

// The column sums of a workgroup's rows: thread t holds those of columns 8 (t % CH) .. + 7
// over its rows; the THREADS / CH sets are added in order through LDS and one partial row of
// the tile's columns is written.
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

}  // namespace
}  // namespace dbgemm
