// What the MFMA kernels of the gated operators do with their sums (GatedEp).  Included by the
// kernels' translation units when they are built for these operators (DBGEMM_GATED).  N is a
// multiple of 8 here (the host sends other columns elsewhere).
//
// A tile goes through the LDS wave by wave, in whole rows, eight columns to a lane, as the other
// epilogue's does.  Where two products share a tile, a wave has the same columns of both, side by
// side in its part of the LDS: the gate and what it is multiplied with meet in one lane, and
// neither product exists outside the registers.
//
// The K loops around it are bound by the MFMA at large sizes (4096 x 13696 x 5120 with G and U kept
// 935 us, 1229 TFLOP/s; 8192 x 13696 x 5120 of 8-bit integers 938 us, 2450 T op/s).  The epilogue is
// bound by memory, and by the VALU for GELU (erf), and nothing of it runs beside the next tile's
// products: a gradient at 4096 x 13696 x 5120, 561 MB in and out of its epilogue, 521 us where its
// products alone take 430.  (Asking for four steps of G and U ahead instead of two, staggering the
// workgroups' starts and leaving out the partial sums changed nothing.)
#pragma once

#include "epilogue.h"
#include "gated_internal.h"
#include "mfma_common.h"

namespace dbgemm {
namespace {

// Column constants of a lane: the biases and, for 8-bit integers, the factors of its columns.
template <bool I8, int OP>
struct GtCols {
  float b[8], b2[8], s[8], s2[8];
  __device__ __forceinline__ GtCols(const GatedArgs& a, int n, int nv) {
    const GatedEp& e = a.ep;
    if constexpr (OP != GT_GRAD) {
      load(e.bias, e.bias_f32, n, nv, b);
      if constexpr (OP == GT_GATED) load(e.bias2, e.bias_f32, n, nv, b2);
    }
    if constexpr (I8) {
      load(e.sb, 1, n, nv, s);
      if constexpr (OP == GT_GATED) load(e.sb2, 1, n, nv, s2);
    }
  }
  __device__ __forceinline__ static void load(const void* p, int f32, int n, int nv, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (p && nv) ep_load8(p, n, f32, 8, v);
  }
};

// What a row brings for columns [n, n + 8): a residual (8 bf16 in lo, or fp32 in both), or G and U;
// and the row's factor.  NT: past the caches, for what does not fit them anyway (GatedEp::past).
struct GtRaw {
  ep_u32x4 lo, hi;
  float s;
};

template <bool NT, class V>
__device__ __forceinline__ ep_u32x4 gt_load(const V* p) {
  if constexpr (NT)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}

template <bool NT, bool I8, int OP>
__device__ __forceinline__ GtRaw gt_fetch8(const GatedArgs& a, int64_t m, int n, int nv) {
  const GatedEp& e = a.ep;
  GtRaw r;
  r.lo = r.hi = (ep_u32x4){0, 0, 0, 0};
  r.s = 0.f;
  if (nv == 0) return r;
  if constexpr (I8) r.s = e.sa[m];
  if constexpr (OP == GT_GRAD) {
    r.lo = gt_load<NT>((const ep_u32x4_2*)((const uint16_t*)e.G + m * e.ldg + n));
    r.hi = gt_load<NT>((const ep_u32x4_2*)((const uint16_t*)e.U + m * e.ldu + n));
  } else if constexpr (OP == GT_LINEAR) {
    if (e.R && a.c_kind == C_F32) {
      const float* p = (const float*)e.R + m * e.ldr + n;
      r.lo = gt_load<NT>((const ep_u32x4_4*)p);
      r.hi = gt_load<NT>((const ep_u32x4_4*)(p + 4));
    } else if (e.R) {
      r.lo = gt_load<NT>((const ep_u32x4_2*)((const uint16_t*)e.R + m * e.ldr + n));
    }
  }
  return r;
}

__device__ __forceinline__ void gt_bf16(const ep_u32x4& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __builtin_bit_cast(float, r[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
  }
}

// Eight sums of a row times its factor s and their columns' c, plus b (kFarFactor).
__device__ __forceinline__ void gt_scale8(float (&w)[8], float s, const float (&c)[8], const float (&b)[8], bool far) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __builtin_fmaf(w[i] * (far ? c[i] : s), far ? s : c[i], b[i]);
}

// Eight columns of row m: w, w2 the products (w2 of the second B), alpha applied, or the whole
// numbers as floats.  A gradient's unrounded results are added to cs and cs2.
template <bool NT, bool I8, int OP, int ACT>
__device__ __forceinline__ void gt_finish8(const GatedArgs& a, float (&w)[8], float (&w2)[8], const GtRaw& r,
                                           const GtCols<I8, OP>& c, int64_t m, int n, float (&cs)[8], float (&cs2)[8]) {
  const GatedEp& e = a.ep;
  const int f32 = a.c_kind == C_F32;
  if constexpr (OP == GT_GRAD) {
    float g[8], u[8], h[8], du[8];
    gt_bf16(r.lo, g);
    gt_bf16(r.hi, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = ep_act<ACT>(g[i]);
      du[i] = w[i] * h[i];
      w[i] *= u[i] * ep_slope<ACT>(g[i]);
      cs[i] += w[i];
      cs2[i] += du[i];
      h[i] *= u[i];
    }
    ep_store8<NT, EP_NONE>(e.D2, m * e.ldd2 + n, f32, 8, du);
    if (e.H) ep_store8<NT, EP_NONE>((uint16_t*)e.H + m * e.ldh + n, 8, h);
  } else {
    if constexpr (I8) {
      const bool far = __builtin_fabsf(r.s) > kFarFactor;
      if (__builtin_expect(__any(far), 0)) {  // (a branch of the whole wave: selects would be two an element)
        gt_scale8(w, r.s, c.s, c.b, far);
        if constexpr (OP == GT_GATED) gt_scale8(w2, r.s, c.s2, c.b2, far);
      } else {
        gt_scale8(w, r.s, c.s, c.b, false);
        if constexpr (OP == GT_GATED) gt_scale8(w2, r.s, c.s2, c.b2, false);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] += c.b[i];
        if constexpr (OP == GT_GATED) w2[i] += c.b2[i];
      }
    }
    if constexpr (OP == GT_GATED) {
      if (e.G) ep_store8<NT, EP_NONE>((uint16_t*)e.G + m * e.ldg + n, 8, w);
      if (e.U) ep_store8<NT, EP_NONE>((uint16_t*)e.U + m * e.ldu + n, 8, w2);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = ep_act<ACT>(w[i]);
    if constexpr (OP == GT_GATED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] *= w2[i];
    } else if (e.R) {
      float v[8];
      if (f32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = __builtin_bit_cast(float, (uint32_t)r.lo[i]);
          v[4 + i] = __builtin_bit_cast(float, (uint32_t)r.hi[i]);
        }
      } else {
        gt_bf16(r.lo, v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] += e.beta * v[i];
    }
  }
  ep_store8<NT, EP_NONE>(a.C, m * a.ldc + n, f32, 8, w);
}

// Four sums as floats: times alpha, or the whole numbers that their bits are.
template <class C>
__device__ __forceinline__ f32x4 gt_sums(const f32x4& v, float alpha) {
  if constexpr (C::I8) {
    const i32x4 k = __builtin_bit_cast(i32x4, v);
    return (f32x4){(float)k[0], (float)k[1], (float)k[2], (float)k[3]};
  } else {
    return (f32x4){alpha * v[0], alpha * v[1], alpha * v[2], alpha * v[3]};
  }
}

// the eight floats of 16-byte chunks ch and ch + 1 of an LDS row at `at`, swizzled by x
__device__ __forceinline__ void gt_row8(uint32_t at, uint32_t ch, uint32_t x, float (&w)[8]) {
  const f32x4 lo = *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(at + ((ch ^ x) * 16));
  const f32x4 hi = *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(at + (((ch + 1) ^ x) * 16));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = lo[i];
    w[4 + i] = hi[i];
  }
}

// Rows of a wave's part that go through the LDS at a time: whole fragments and whole steps of
// `step` rows, as many as fit.
template <class C, int LDS_BYTES>
constexpr int gt_pass_rows(int step) {
  int rows = C::WTM;
  while (rows > 16 && (rows * C::WTN * 4 * (C::THREADS / 64) > LDS_BYTES || C::WTM % rows != 0 || rows % step != 0))
    rows -= 16;
  return rows;
}

// acc: the 16x16 fragments of this wave, whose results start at row m0, column n0 (of both
// products).  lds0: LDS_BYTES of LDS, free once every wave has passed the barrier here.  The
// 16-byte chunks of an LDS row are XOR-swizzled by the row.  What the rows bring from memory is
// asked for ahead, up to BATCH steps of rows at a time.  NT: the outputs go past the caches (the 256 x 256
// tiles, whatever their size: a gated product alone up to 13 % faster than with cached stores at 8 to 107 MB of H,
// 2048 x 8192 x 2048 104 us and 118; with the product that reads H behind it 0.4 to 2 %, but for the
// smallest, 1531 x 2736 x 1000 with 8 MB, where the two take 62.1 and 58.1).  NTL: so do the rows that are read.
template <class C, int OP, int LDS_BYTES, bool NT, bool NTL>
__device__ __forceinline__ void gt_tile(const GatedArgs& a, const typename AccOf<C::MT>::T (&acc)[C::FM][C::FN], int m0,
                                        int n0, int part, int wave, int lane, uint32_t lds0) {
  static_assert(C::MT == 16 && C::ACC == 4 && C::DUAL == (OP == GT_GATED), "16x16 fragments");
  constexpr int OUT = C::WTN / C::NSUB;            // result columns of a wave
  constexpr int LPR = OUT / 8, RPS = 64 / LPR;     // lanes to a row, rows to a step
  constexpr int PASS = gt_pass_rows<C, LDS_BYTES>(RPS);
  constexpr int RB = C::WTN * 4, CPR = C::WTN / 4;  // bytes and 16-byte chunks of an LDS row
  constexpr int STEPS = PASS / RPS, ALL = C::WTM / RPS;
  constexpr int WANT = OP == GT_GRAD ? 2 : 4, BATCH = STEPS < WANT ? STEPS : WANT;
  static_assert(PASS * RB * (C::THREADS / 64) <= LDS_BYTES && C::WTM % PASS == 0, "a pass of every wave fits");
  static_assert((CPR & (CPR - 1)) == 0 && PASS % RPS == 0 && STEPS % BATCH == 0, "whole steps and batches");
  const uint32_t mine = lds0 + (uint32_t)(wave * PASS * RB);
  const int row = lane / LPR, ch = (lane % LPR) * 2, n = n0 + (lane % LPR) * 8;
  const int nvc = n < a.N ? 8 : 0;
  const float alpha = a.alpha;
  float cs[8] = {}, cs2[8] = {};
  const GtCols<C::I8, OP> cols(a, n, nvc);
  ep_with_act(a.ep.act, [&](auto ac) EP_INLINE {
    constexpr int ACT = decltype(ac)::value;
    GtRaw raw[BATCH];
    auto fetch = [&](int step) EP_INLINE {
      const int m = m0 + row + step * RPS;
      return gt_fetch8<NTL, C::I8, OP>(a, m, n, step < ALL && m < a.M ? nvc : 0);
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
            gt_sums<C>(acc[i][j], alpha);
      });
#pragma unroll 1
      for (int s0 = 0; s0 < STEPS; s0 += BATCH) {
#pragma unroll
        for (int s = 0; s < BATCH; ++s) {
          const int r = (s0 + s) * RPS + row, m = mp + (s0 + s) * RPS;
          const uint32_t at = mine + (uint32_t)(r * RB), x = (uint32_t)(r & (CPR - 1));
          float w[8], w2[8];
          gt_row8(at, ch, x, w);
          if constexpr (C::DUAL) gt_row8(at, ch + OUT / 4, x, w2);
          if (m < a.M && nvc) gt_finish8<NT, C::I8, OP, ACT>(a, w, w2, raw[s], cols, m, n, cs, cs2);
          raw[s] = fetch(h * STEPS + s0 + s + BATCH);
        }
      }
    });
  });
  if constexpr (OP == GT_GRAD) {
    if (a.ep.colsum) {
      // the wave's rows of each column: over the lanes that share the columns, then out
#pragma unroll
      for (int o = LPR; o < 64; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cs[i] += __shfl_xor(cs[i], o);
          cs2[i] += __shfl_xor(cs2[i], o);
        }
      if (lane < LPR && nvc) {
        float* p = a.ep.colsum + (int64_t)part * 2 * a.N + n;
        ep_store8<false, EP_NONE>(p, 8, cs);
        ep_store8<false, EP_NONE>(p + a.N, 8, cs2);
      }
    }
  }
}

// A split product's tile, fragment row i of every row of waves: the partial tiles added in split
// order (8-bit integers as whole numbers), put together in LDS as WM x 16 rows, and finished.
template <class C, int OP>
__device__ __forceinline__ void gt_strip(const GatedArgs& a, int tile, int i, int t) {
  constexpr int OUT = C::WTN / C::NSUB;
  constexpr int ROWS = C::WM * 16, RB = C::BN * 4, CH = C::SUB_BN / 8, RPS = C::THREADS / CH;
  constexpr int STEPS = ROWS < RPS ? 1 : ROWS / RPS;
  static_assert(C::ACC == 4 && (ROWS % RPS == 0 || ROWS < RPS), "16x16 fragments, whole steps of rows");
  __shared__ __attribute__((aligned(1024))) char lds[ROWS * RB];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
  const int tm = tile / a.tiles_n, tn = tile % a.tiles_n;
  const int lane = t & 63, wave = t >> 6;
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int m0 = tm * C::BM, n0 = tn * C::SUB_BN;
  // local row r of the strip is row (r / 16) WTM + 16 i + r % 16 of the tile; its columns are the
  // waves' parts side by side
  auto row_of = [&](int r) { return m0 + (r >> 4) * C::WTM + i * 16 + (r & 15); };
  const int row = t / CH, c = (t % CH) * 8, n = n0 + c;
  const uint32_t ch = (uint32_t)(c / OUT * C::WTN + c % OUT) / 4;
  const int nvc = n < a.N && row < ROWS ? 8 : 0;
  float cs[8] = {}, cs2[8] = {};
  const GtCols<C::I8, OP> cols(a, n, nvc);
  const f32x4* src = (const f32x4*)(a.ws + (size_t)tile * a.splits * (C::BM * C::BN)) + i * C::FN * C::THREADS + t;
  constexpr size_t stride = (size_t)C::FM * C::FN * C::THREADS;  // float4s per partial
  ep_with_act(a.ep.act, [&](auto ac) EP_INLINE {
    GtRaw raw[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int m = row_of(s * RPS + row);
      raw[s] = gt_fetch8<false, C::I8, OP>(a, m, n, m < a.M ? nvc : 0);
    }
    if (row_of(wm * 16) < a.M) {  // (this wave's rows past M hold no sums)
      f32x4 v[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) v[j] = src[j * C::THREADS];
#pragma unroll 4
      for (int s = 1; s < a.splits; ++s)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
          const f32x4 p = src[s * stride + j * C::THREADS];
          if constexpr (C::I8)
            v[j] = __builtin_bit_cast(f32x4, __builtin_bit_cast(i32x4, v[j]) + __builtin_bit_cast(i32x4, p));
          else
            v[j] += p;
        }
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const int r = wm * 16 + lane % 16, chunk = ((wn * C::WTN + j * 16 + 4 * (lane / 16)) >> 2) ^ (r & 15);
        *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(lds0 + (uint32_t)(r * RB + chunk * 16)) =
            gt_sums<C>(v[j], a.alpha);
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * RPS + row, m = row_of(r);
      const uint32_t at = lds0 + (uint32_t)(r * RB), x = (uint32_t)(r & 15);
      if (!nvc || m >= a.M) continue;
      float w[8], w2[8];
      gt_row8(at, ch, x, w);
      if constexpr (C::DUAL) gt_row8(at, ch + OUT / 4, x, w2);
      gt_finish8<false, C::I8, OP, decltype(ac)::value>(a, w, w2, raw[s], cols, m, n, cs, cs2);
    }
  });
  if constexpr (OP == GT_GRAD) {
    if (!a.ep.colsum) return;
    // the threads' sums meet in LDS, one set after the other, and one partial row of the tile's
    // columns is written for each
    constexpr int SETS = C::THREADS / CH;
    static_assert(SETS * C::SUB_BN <= ROWS * C::BN, "a set of sums fits the strip");
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __syncthreads();  // the LDS is free again
      const uint32_t at = lds0 + (uint32_t)((t / CH) * C::SUB_BN * 4 + (t % CH) * 32);
      const float(&v)[8] = k ? cs2 : cs;
      *(__attribute__((address_space(3))) f32x4*)(uintptr_t)at = (f32x4){v[0], v[1], v[2], v[3]};
      *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(at + 16) = (f32x4){v[4], v[5], v[6], v[7]};
      __syncthreads();
      if (t < C::SUB_BN && n0 + t < a.N) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < SETS; ++q)
          sum += *(__attribute__((address_space(3))) float*)(uintptr_t)(lds0 + (uint32_t)(q * C::SUB_BN * 4 + t * 4));
        a.ep.colsum[(((int64_t)tm * C::FM + i) * 2 + k) * a.N + n0 + t] = sum;
      }
    }
  }
}

}  // namespace
}  // namespace dbgemm
