// Device side of the epilogues and of the activations: the functions and their slopes, and
// what is done with eight consecutive columns of a product (or of a stored activation).
// Included by kernel translation units only.
#pragma once

#include <type_traits>

#include "e4m3_codec.h"
#include "mlp_internal.h"

// Lambdas over an activation: called, their captured arrays would live in scratch memory.
#define EP_INLINE __attribute__((always_inline))

namespace dbgemm {
namespace {

// Vectors at element alignment: global memory takes 8- and 16-byte accesses at any address,
// so an odd leading dimension needs no path of its own.
typedef unsigned short ep_u16x8 __attribute__((ext_vector_type(8)));
typedef float ep_f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int ep_u32x2 __attribute__((ext_vector_type(2)));
typedef ep_u16x8 ep_u16x8_u __attribute__((aligned(2)));
typedef ep_f32x4 ep_f32x4_u __attribute__((aligned(4)));
typedef ep_u32x2 ep_u32x2_u __attribute__((aligned(1)));
typedef unsigned int ep_u32x4 __attribute__((ext_vector_type(4)));
typedef ep_u32x4 ep_u32x4_4 __attribute__((aligned(4)));
typedef ep_u32x4 ep_u32x4_2 __attribute__((aligned(2)));
typedef ep_u32x2 ep_u32x2_2 __attribute__((aligned(2)));
typedef uint32_t ep_u32_2 __attribute__((aligned(2)));
typedef uint32_t ep_u32_1 __attribute__((aligned(1)));
typedef uint16_t ep_u16_1 __attribute__((aligned(1)));

__device__ __forceinline__ float ep_bf16f(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
__device__ __forceinline__ uint16_t ep_f32bf(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// The last columns of a row that is no multiple of eight: one by one, or (fewer accesses, more
// registers: the layer norm kernels of wide rows spilled) in pieces of four, two and one; none
// where the host sees to it that there are no such columns.
enum EpPart { EP_NONE = 0, EP_ONES = 1, EP_PIECES = 2 };

// The first nv < 8 elements of ES bytes at p, zeros behind them: four, two and one of them in
// one access each (an access per element cost the last lane of an odd row, and so its wave,
// most of the time: 59881 x 671 from codes 155 us, now 61, against 51 at 672 columns).
template <int ES>
__device__ __forceinline__ ep_u32x4 ep_raw_part(const void* p, int nv) {
  static_assert(ES == 1 || ES == 2, "bytes or halves");
  ep_u32x4 r = {0, 0, 0, 0};
  if constexpr (ES == 1) {
    const uint8_t* q = (const uint8_t*)p;
    uint32_t a = 0, t = 0;
    if (nv & 4) {
      a = *(const ep_u32_1*)q;
      q += 4;
    }
    if (nv & 2) {
      t = *(const ep_u16_1*)q;
      q += 2;
    }
    if (nv & 1) t |= (uint32_t)*q << ((nv & 2) * 8);
    r[0] = nv & 4 ? a : t;
    r[1] = nv & 4 ? t : 0u;
  } else {
    const uint16_t* q = (const uint16_t*)p;
    ep_u32x2 a = {0, 0}, t = {0, 0};
    if (nv & 4) {
      a = *(const ep_u32x2_2*)q;
      q += 4;
    }
    if (nv & 2) {
      t[0] = *(const ep_u32_2*)q;
      q += 2;
    }
    if (nv & 1) {
      const uint32_t one = *q;
      t[0] = nv & 2 ? t[0] : one;
      t[1] = nv & 2 ? one : 0u;
    }
    r[0] = nv & 4 ? a[0] : t[0];
    r[1] = nv & 4 ? a[1] : t[1];
    r[2] = nv & 4 ? t[0] : 0u;
    r[3] = nv & 4 ? t[1] : 0u;
  }
  return r;
}

// 8 elements at p, the first nv of them valid (the others read as zeros).
template <int PART = EP_ONES>
__device__ __forceinline__ void ep_load8(const uint16_t* p, int nv, float (&v)[8]) {
  if (nv == 8) {
    const ep_u16x8 w = *(const ep_u16x8_u*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ep_bf16f(w[i]);
  } else if constexpr (PART == EP_PIECES) {
    const ep_u32x4 w = ep_raw_part<2>(p, nv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < nv ? ep_bf16f(p[i]) : 0.f;
  }
}
__device__ __forceinline__ void ep_load8(const float* p, int nv, float (&v)[8]) {
  if (nv == 8) {
    const ep_f32x4 a = *(const ep_f32x4_u*)p, b = *(const ep_f32x4_u*)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < nv ? p[i] : 0.f;
  }
}
// 8 elements of a matrix of either type
__device__ __forceinline__ void ep_load8(const void* p, int64_t idx, int f32, int nv, float (&v)[8]) {
  if (f32)
    ep_load8((const float*)p + idx, nv, v);
  else
    ep_load8((const uint16_t*)p + idx, nv, v);
}

// The whole-vector stores of large outputs are non-temporal (NT): the kernel does not read
// them again.
template <bool NT, int PART = EP_ONES>
__device__ __forceinline__ void ep_store8(uint16_t* p, int nv, const float (&v)[8]) {
  if (nv == 8) {
    ep_u16x8 w;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = ep_f32bf(v[i]);
    if constexpr (NT)
      __builtin_nontemporal_store(w, (ep_u16x8_u*)p);
    else
      *(ep_u16x8_u*)p = w;
  } else if constexpr (PART == EP_ONES) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nv) p[i] = ep_f32bf(v[i]);
  } else if constexpr (PART == EP_PIECES) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ep_f32bf(v[2 * i]) | (uint32_t)ep_f32bf(v[2 * i + 1]) << 16;
    if (nv & 4) {
      *(ep_u32x2_2*)p = (ep_u32x2){w[0], w[1]};
      p += 4;
      w[0] = w[2];
      w[1] = w[3];
    }
    if (nv & 2) {
      *(ep_u32_2*)p = w[0];
      p += 2;
      w[0] = w[1];
    }
    if (nv & 1) *p = (uint16_t)w[0];
  }
}
template <bool NT, int PART = EP_ONES>
__device__ __forceinline__ void ep_store8(float* p, int nv, const float (&v)[8]) {
  if (nv == 8) {
    const ep_f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    if constexpr (NT) {
      __builtin_nontemporal_store(a, (ep_f32x4_u*)p);
      __builtin_nontemporal_store(b, (ep_f32x4_u*)(p + 4));
    } else {
      *(ep_f32x4_u*)p = a;
      *(ep_f32x4_u*)(p + 4) = b;
    }
  } else if constexpr (PART == EP_ONES) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nv) p[i] = v[i];
  } else if constexpr (PART == EP_PIECES) {
    float a = v[0], b = v[1], c = v[2];
    if (nv & 4) {
      *(ep_f32x4_u*)p = (ep_f32x4){v[0], v[1], v[2], v[3]};
      p += 4;
      a = v[4];
      b = v[5];
      c = v[6];
    }
    if (nv & 2) {
      p[0] = a;
      p[1] = b;
      p += 2;
      a = c;
    }
    if (nv & 1) *p = a;
  }
}
template <bool NT, int PART = EP_ONES>
__device__ __forceinline__ void ep_store8(void* p, int64_t idx, int f32, int nv, const float (&v)[8]) {
  if (f32)
    ep_store8<NT, PART>((float*)p + idx, nv, v);
  else
    ep_store8<NT, PART>((uint16_t*)p + idx, nv, v);
}

// ---- activations.  logistic(v) = 1 / (1 + 2^(-v log2 e)) with the hardware's exponential
// and reciprocal (1 ulp each): 2^inf = inf and 1 / inf = 0, so both ends saturate.
__device__ __forceinline__ float ep_logistic2(float neg_v_log2e) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(neg_v_log2e));
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC0 = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluC1 = 0.044715f;

// q = 1 - Phi(|z|) and e = exp(-z^2 / 2): q = e t P(t), t = 1 / (1 + 0.345 |z|), P a polynomial of
// degree 6 fitted to the scaled complementary error function over |z| <= 14 (past it e is 0) to a
// relative error of 5.4e-8 (1 + 2 z^2), the growth of the exponential's own.  (Five terms and an
// absolute error of 1.5e-7, one operation less, were a few units of fp32 off near 0 and up to 4 % in the tail.)
__device__ __forceinline__ float ep_gauss_tail(float z, float& e) {
  const float x = __builtin_fabsf(z);
  e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.345f * x);
  return t * (0.1378859f + t * (0.133416782f + t * (0.14963316f + t * (-0.0108854157f + t * (0.238464067f +
         t * (-0.193563412f + t * 0.045048946f)))))) * e;
}

template <int ACT>
__device__ __forceinline__ float ep_act(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z < 0.f ? 0.f : z;  // NaN stays NaN
  } else if constexpr (ACT == ACT_GELU) {
    float e;
    const float q = ep_gauss_tail(z, e);
    return z * (z < 0.f ? q : 1.0f - q);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = logistic(2u)
    return z * ep_logistic2(z * (-2.f * kGeluC0 * kLog2e - 2.f * kGeluC0 * kGeluC1 * kLog2e * z * z));
  } else if constexpr (ACT == ACT_SILU) {
    return z * ep_logistic2(-kLog2e * z);
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float ep_slope(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z > 0.f ? 1.f : (z == z ? 0.f : z);
  } else if constexpr (ACT == ACT_GELU) {
    float e;
    const float q = ep_gauss_tail(z, e);
    return (z < 0.f ? q : 1.0f - q) + z * (0.3989422804014327f * e);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float s = ep_logistic2(z * (-2.f * kGeluC0 * kLog2e - 2.f * kGeluC0 * kGeluC1 * kLog2e * z * z));
    // past |z| = 64 the second term is 0 (s is 0 or 1); clamped so that z^2 stays finite
    const float c = __builtin_fminf(__builtin_fmaxf(z, -64.f), 64.f);
    return s + c * (s * (1.f - s)) * (2.f * kGeluC0 + 6.f * kGeluC0 * kGeluC1 * c * c);
  } else if constexpr (ACT == ACT_SILU) {
    const float s = ep_logistic2(-kLog2e * z);
    return s * (1.f + z * (1.f - s));
  } else {
    return 1.f;
  }
}

// f(integral_constant<int, act>) for the run-time act (uniform over the launch)
template <class F>
__device__ __forceinline__ void ep_with_act(int act, F&& f) {
  switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>{}); break;
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>{}); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>{}); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>{}); break;
    default: f(std::integral_constant<int, ACT_NONE>{}); break;
  }
}

// The largest magnitude goes round the four lanes in the VALU (DPP quads), and the clamp is one
// v_med3: that loses a NaN, so eights that hold one take the conversion that keeps it.
__device__ __forceinline__ float ep_quad_max(float v) {
  const int a = __builtin_bit_cast(int, v);
  v = __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(a, a, 0xB1, 0xF, 0xF, true)));
  const int b = __builtin_bit_cast(int, v);
  return __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, 0x4E, 0xF, 0xF, true)));
}
__device__ __forceinline__ uint32_t ep_sat4(float a, float b, float c, float d) {
  auto sat = [](float x) EP_INLINE { return __builtin_amdgcn_fmed3f(x, -448.f, 448.f); };
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), w, true);
}
// Eight values of a row to E4M3 codes: the four neighbouring lanes that hold one block of
// 32 columns (columns n & ~31 .. + 31) run this together, each with its eight (the invalid
// ones zero).  Stores the first nv codes at q and, from the block's first lane when it has
// any column, the scale byte at s.
template <bool PART = true>
__device__ __forceinline__ void ep_store_mx(const float (&v)[8], int nv, bool first, uint8_t* q, uint8_t* s) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[i]));  // NaN does not set it
  const int e = mx_scale(ep_quad_max(amax));
  const float inv = mx_inv(e);
  uint32_t lo = ep_sat4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  uint32_t hi = ep_sat4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  if (__builtin_isunordered(v[0], v[1]) | __builtin_isunordered(v[2], v[3]) | __builtin_isunordered(v[4], v[5]) |
      __builtin_isunordered(v[6], v[7])) {
    lo = e4m3x4_from_f32(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    hi = e4m3x4_from_f32(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  }
  if (first && nv > 0) *s = (uint8_t)e;
  if (nv == 8) {
    *(ep_u32x2_u*)q = (ep_u32x2){lo, hi};
  } else if constexpr (PART) {
    if (nv & 4) {
      *(ep_u32_1*)q = lo;
      q += 4;
      lo = hi;
    }
    if (nv & 2) {
      *(ep_u16_1*)q = (uint16_t)lo;
      q += 2;
      lo >>= 16;
    }
    if (nv & 1) *q = (uint8_t)lo;
  }
}

// Eight values from their codes (bytes of lo, then hi) and their block's scale byte.
__device__ __forceinline__ void ep_codes8(uint32_t lo, uint32_t hi, uint32_t scale, float (&v)[8]) {
  const float f = scale == 255u ? __builtin_nanf("") : __builtin_bit_cast(float, scale == 0u ? 0x00400000u : scale << 23);
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)lo, 0) * f;
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)lo, 1) * f;
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)lo, 2) * f;
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)lo, 3) * f;
  v[4] = __builtin_amdgcn_cvt_f32_fp8((int)hi, 0) * f;
  v[5] = __builtin_amdgcn_cvt_f32_fp8((int)hi, 1) * f;
  v[6] = __builtin_amdgcn_cvt_f32_fp8((int)hi, 2) * f;
  v[7] = __builtin_amdgcn_cvt_f32_fp8((int)hi, 3) * f;
}

// The epilogue of columns [n, n + 8) of row m (n a multiple of 8) in two parts: ep_fetch8
// issues the load of what the row brings (the residual, or Z for a gradient), ep_finish8 does
// the rest, so that a caller can have the loads of several rows in flight.  nv: the valid
// columns, 0 .. 8 (0: no row or column here).
//
// A gradient's Z is a compile-time choice: where the loads of codes and of bf16 met again in one
// register, the compiler waited for them at once and nothing was in flight (2048 x 20480 x 5120
// from codes: 380 us, so 369).  The same for a residual's kinds, with unconditional loads, made
// no difference.
enum { EP_FORWARD = 0, EP_GRAD_BF16 = 1, EP_GRAD_MX = 2 };
struct EpRaw {
  ep_u32x4 lo, hi;  // 8 bf16 in lo, 8 fp32, or 8 codes in lo[0..1] and their scale in lo[2]
};

template <int MODE, bool PART>
__device__ __forceinline__ EpRaw ep_fetch8(const GemmEpArgs& a, int64_t m, int n, int nv) {
  const EpArgs& e = a.ep;
  EpRaw r;
  r.lo = r.hi = (ep_u32x4){0, 0, 0, 0};
  if (nv == 0) return r;
  const bool whole = !PART || nv == 8;
  if constexpr (MODE == EP_GRAD_MX) {
    const uint8_t* p = (const uint8_t*)e.Z + m * e.ldz + n;
    if (whole) {
      const ep_u32x2 v = *(const ep_u32x2_u*)p;
      r.lo = (ep_u32x4){v[0], v[1], 0, 0};
    } else if constexpr (PART) {
      r.lo = ep_raw_part<1>(p, nv);
    }
    r.lo[2] = e.S[m * e.lds + (n >> 5)];
    return r;
  } else if constexpr (MODE == EP_FORWARD) {
    if (!e.R) return r;
    if (a.c_kind == C_F32) {
      const float* p = (const float*)e.R + m * e.ldr + n;
      if (whole) {
        r.lo = *(const ep_u32x4_4*)p;
        r.hi = *(const ep_u32x4_4*)(p + 4);
      } else if constexpr (PART) {
        float v[8];
        ep_load8(p, nv, v);
        r.lo = __builtin_bit_cast(ep_u32x4, (ep_f32x4){v[0], v[1], v[2], v[3]});
        r.hi = __builtin_bit_cast(ep_u32x4, (ep_f32x4){v[4], v[5], v[6], v[7]});
      }
      return r;
    }
  }
  const uint16_t* p = MODE != EP_FORWARD ? (const uint16_t*)e.Z + m * e.ldz + n : (const uint16_t*)e.R + m * e.ldr + n;
  if (whole)
    r.lo = *(const ep_u32x4_2*)p;
  else if constexpr (PART)
    r.lo = ep_raw_part<2>(p, nv);
  return r;
}

__device__ __forceinline__ void ep_raw_bf16(const EpRaw& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __builtin_bit_cast(float, r.lo[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, r.lo[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void ep_raw_f32(const EpRaw& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __builtin_bit_cast(float, (uint32_t)r.lo[i]);
    v[4 + i] = __builtin_bit_cast(float, (uint32_t)r.hi[i]);
  }
}

// w = alpha * product, b = the bias of these columns (zeros without one).  The four lanes of a
// block of 32 columns call it together.  A gradient's unrounded results are added to cs.
template <bool NT, int MODE, int ACT, bool PART>
__device__ __forceinline__ void ep_finish8(const GemmEpArgs& a, float (&w)[8], const EpRaw& r, const float (&b)[8],
                                           int64_t m, int n, int nv, float (&cs)[8]) {
  const EpArgs& e = a.ep;
  float v[8];
  if constexpr (MODE != EP_FORWARD) {
    if (nv == 0) return;
    if constexpr (MODE == EP_GRAD_MX)
      ep_codes8(r.lo[0], r.lo[1], r.lo[2], v);
    else
      ep_raw_bf16(r, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] *= ep_slope<ACT>(v[i]);
      cs[i] += !PART || i < nv ? w[i] : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] += b[i];
    if (e.z_kind == Z_MX) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (PART ? i < nv : nv > 0) ? w[i] : 0.f;
      ep_store_mx<PART>(v, nv, (n & 31) == 0, (uint8_t*)e.Z + m * e.ldz + n, e.S + m * e.lds + (n >> 5));
    }
    if (nv == 0) return;
    if (e.z_kind == Z_BF16) ep_store8<NT, PART ? EP_PIECES : EP_NONE>((uint16_t*)e.Z + m * e.ldz + n, nv, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = ep_act<ACT>(w[i]);
    if (e.R) {
      if (a.c_kind == C_F32)
        ep_raw_f32(r, v);
      else
        ep_raw_bf16(r, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] += e.beta * v[i];
    }
  }
  ep_store8<NT, PART ? EP_PIECES : EP_NONE>(a.C, m * a.ldc + n, a.c_kind == C_F32, nv, w);
}

// the bias of columns [n, n + 8)
__device__ __forceinline__ void ep_bias8(const GemmEpArgs& a, int n, int nv, float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.f;
  if (!a.ep.grad && a.ep.bias) ep_load8(a.ep.bias, n, a.ep.bias_f32, nv, b);
}

// f(integral_constant<int, mode>, integral_constant<int, act>) for the call's epilogue
template <class F>
__device__ __forceinline__ void ep_dispatch(const EpArgs& e, F&& f) {
  auto with = [&](auto mc) EP_INLINE { ep_with_act(e.act, [&](auto ac) EP_INLINE { f(mc, ac); }); };
  if (!e.grad)
    with(std::integral_constant<int, EP_FORWARD>{});
  else if (e.z_kind == Z_MX)
    with(std::integral_constant<int, EP_GRAD_MX>{});
  else
    with(std::integral_constant<int, EP_GRAD_BF16>{});
}

}  // namespace
}  // namespace dbgemm
