// Rows of bf16 or fp32 -> 8-bit integers with a factor for each row: s = max|x| / 127, the code of
// x the whole number nearest to 127 x / max|x|, ties to even.
//
// The codes are those of the exact quotient.  v = x * fl(127 / max|x|) as one fma is within 127 *
// 2^-24 of it before its rounding, so a code can only be wrong where v lies within 2^-16 of the
// middle between two codes; eights with such a value (3 % of the waves on random rows) are
// divided in 64 bits, where the quotient of 127 x (31 bits) and max|x| (24) is exact at a middle
// and, being no middle, at least 2^-26 away from it otherwise.
//
// A row that holds Inf or NaN has the factor NaN and codes 0, so that what is computed from it is
// NaN too; a row of zeros the factor 0 and codes 0.
#include "epilogue.h"
#include "gated_internal.h"

namespace dbgemm {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;

// eight codes of x at inv = fl(127 / top); `slow`: top is so small that inv may overflow
__device__ __forceinline__ ep_u32x2 qi_codes(const float (&x)[8], float inv, float top, bool slow) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to the nearest integer, ties to even
  float t[8], off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = __builtin_fmaf(x[i], inv, kMagic);
    off = __builtin_fmaxf(off, __builtin_fabsf(__builtin_fmaf(x[i], inv, -(t[i] - kMagic))));
  }
  if (slow || off > 0.5f - 0x1p-16f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = (float)__builtin_rint(127.0 * (double)x[i] / (double)top) + kMagic;
  }
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __builtin_bit_cast(uint32_t, t[i]) & 0xFFu;
  return (ep_u32x2){b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24};
}

// the first nv codes to d
__device__ __forceinline__ void qi_store(int8_t* d, int nv, ep_u32x2 w) {
  if (nv == 8) {
    *(ep_u32x2_u*)d = w;
    return;
  }
  if (nv & 4) {
    *(ep_u32_1*)d = w[0];
    d += 4;
    w[0] = w[1];
  }
  if (nv & 2) {
    *(ep_u16_1*)d = (uint16_t)w[0];
    d += 2;
    w[0] >>= 16;
  }
  if (nv & 1) *d = (int8_t)w[0];
}

template <class T>
__device__ __forceinline__ void qi_load(const T* p, int nv, float (&v)[8]) {
  if constexpr (sizeof(T) == 2)
    ep_load8<EP_PIECES>(p, nv, v);
  else
    ep_load8(p, nv, v);
}

// One workgroup to a row, two passes over it.
template <class T>
__global__ __launch_bounds__(256) void quantize_i8_kernel(int64_t rows, int64_t cols, const T* src, int64_t ld_src,
                                                          int8_t* dst, int64_t ld_dst, float* scales) {
  __shared__ uint32_t s[4];
  const int t = threadIdx.x;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* p = src + r * ld_src;
    uint32_t top = 0;  // the bits of the largest magnitude: an order that has Inf and NaN last
    for (int64_t c = (int64_t)t * 8; c < cols; c += 256 * 8) {
      float v[8];
      qi_load(p + c, cols - c < 8 ? (int)(cols - c) : 8, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    __syncthreads();  // (the previous row's readers are done)
    if ((t & 63) == 0) s[t >> 6] = top;
    __syncthreads();
    top = max(max(s[0], s[1]), max(s[2], s[3]));
    const float amax = __builtin_bit_cast(float, top);
    const bool finite = top < kInfBits, none = top == 0 || !finite;
    if (t == 0) scales[r] = finite ? amax / 127.f : __builtin_nanf("");
    const float inv = none ? 0.f : 127.f / amax;
    const bool slow = !none && amax < 0x1p-100f;
    int8_t* d = dst + r * ld_dst;
    for (int64_t c = (int64_t)t * 8; c < cols; c += 256 * 8) {
      const int nv = cols - c < 8 ? (int)(cols - c) : 8;
      float v[8];
      qi_load(p + c, nv, v);
      qi_store(d + c, nv, none ? (ep_u32x2){0, 0} : qi_codes(v, inv, amax, slow));
    }
  }
}

}  // namespace

hipError_t launch_quantize_i8(int64_t rows, int64_t cols, const void* src, int64_t ld_src, int src_kind, int8_t* dst,
                              int64_t ld_dst, float* scales, hipStream_t s) {
  const unsigned grid = (unsigned)(rows < (1 << 20) ? rows : (1 << 20));
  if (src_kind == T_F32)
    hipLaunchKernelGGL(quantize_i8_kernel<float>, dim3(grid), dim3(256), 0, s, rows, cols, (const float*)src, ld_src, dst,
                       ld_dst, scales);
  else
    hipLaunchKernelGGL(quantize_i8_kernel<uint16_t>, dim3(grid), dim3(256), 0, s, rows, cols, (const uint16_t*)src,
                       ld_src, dst, ld_dst, scales);
  return hipGetLastError();
}

}  // namespace dbgemm
