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

// Eight elements as they are in memory (zeros past the first nv).
template <class T>
struct QiRaw {
  ep_u32x4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, int nv) {
    if constexpr (sizeof(T) == 2) {
      w[0] = nv == 8 ? *(const ep_u32x4_2*)p : nv > 0 ? ep_raw_part<2>(p, nv) : (ep_u32x4){0, 0, 0, 0};
    } else {
      float v[8];
      if (nv > 0)
        ep_load8((const float*)p, nv, v);
      else
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i / 4][i % 4] = __builtin_bit_cast(uint32_t, v[i]);
    }
  }
  // the bits of the largest magnitude as fp32: an order that has Inf and NaN last
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) t = max(t, max(w[0][i] & 0x7FFF0000u, (w[0][i] & 0x7FFFu) << 16));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t = max(t, w[i / 4][i % 4] & 0x7FFFFFFFu);
    }
    return t;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __builtin_bit_cast(float, w[0][i] << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, w[0][i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __builtin_bit_cast(float, (uint32_t)w[i / 4][i % 4]);
    }
  }
};

// What the codes of a row take from its largest magnitude; its factor goes to *scale.
struct QiRow {
  float top, inv;
  bool none, slow;
  __device__ __forceinline__ QiRow(uint32_t bits, bool first, float* scale) {
    top = __builtin_bit_cast(float, bits);
    const bool finite = bits < kInfBits;
    none = bits == 0 || !finite;
    inv = none ? 0.f : 127.f / top;
    slow = !none && top < 0x1p-100f;
    if (first) *scale = finite ? top / 127.f : __builtin_nanf("");
  }
  __device__ __forceinline__ ep_u32x2 codes(const float (&v)[8]) const {
    return none ? (ep_u32x2){0, 0} : qi_codes(v, inv, top, slow);
  }
};

// A row in the registers of TEAM threads, C chunks of eight elements to a thread; one pass over
// memory, the next row's loads issued before this one's maximum goes round.  The last chunk of a
// row of at least eight ends at its end, over the one before it where the row is no multiple of
// eight: the same codes are written twice, and no access is less than a chunk (22648 x 361 13.0
// us; the last elements in pieces 14.2).
//
// Bound by memory: 16384 x 5120 bf16 52 us, 4.8 TB/s, fp32 82 us, 5.1 TB/s (a workgroup to a row and two
// passes over it: 55 us); 24 rows of 13696 4.1 us, the launch and one trip to memory, on 1024
// threads to a row (256 and two passes: 6.1).
template <class T, int TEAM, int C>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void quantize_i8_kernel(int64_t rows, int64_t cols, const T* src,
                                                                              int64_t ld_src, int8_t* dst,
                                                                              int64_t ld_dst, float* scales) {
  constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM, WAVES = TEAM / 64;
  __shared__ uint32_t s[2][WAVES > 1 ? WAVES : 1];
  const int t = threadIdx.x % TEAM;
  const int64_t stride = (int64_t)gridDim.x * TEAMS;
  int nv[C], at[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int n = (int)cols;  // (at most 8 * TEAM * C)
    at[i] = (i * TEAM + t) * 8;
    nv[i] = at[i] >= n ? 0 : n < 8 ? n : 8;
    if (at[i] + 8 > n && n >= 8) at[i] = n - 8;
  }
  QiRaw<T> raw[C];
  auto load = [&](int64_t r) EP_INLINE {
#pragma unroll
    for (int i = 0; i < C; ++i) raw[i].load(src + r * ld_src + at[i], r < rows ? nv[i] : 0);
  };
  int64_t r = (int64_t)blockIdx.x * TEAMS + threadIdx.x / TEAM;
  load(r);
  // (the teams of a workgroup of one wave each, or less, go on alone; a larger one is alone in its workgroup)
  for (int k = 0; r < rows; r += stride, k ^= 1) {
    QiRaw<T> now[C];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      now[i] = raw[i];
      top = max(top, now[i].top());
    }
    load(r + stride);
#pragma unroll
    for (int o = 1; o < (TEAM < 64 ? TEAM : 64); o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if constexpr (WAVES > 1) {
      // (two sets of slots: a wave that is a row ahead writes to the other one)
      if ((t & 63) == 0) s[k][t >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = max(top, s[k][w]);
    }
    const QiRow row(top, t == 0, scales + r);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[8];
      now[i].values(v);
      if (nv[i]) qi_store(dst + r * ld_dst + at[i], nv[i], row.codes(v));
    }
  }
}

// Rows past what the registers of a workgroup hold: two passes over each.
template <class T>
__global__ __launch_bounds__(1024) void quantize_i8_wide_kernel(int64_t rows, int64_t cols, const T* src,
                                                                int64_t ld_src, int8_t* dst, int64_t ld_dst,
                                                                float* scales) {
  __shared__ uint32_t s[2][16];
  const int t = threadIdx.x;
  int k = 0;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, k ^= 1) {
    const T* p = src + r * ld_src;
    uint32_t top = 0;
    QiRaw<T> raw;
    for (int64_t c = (int64_t)t * 8; c < cols; c += 1024 * 8) {
      raw.load(p + c, cols - c < 8 ? (int)(cols - c) : 8);
      top = max(top, raw.top());
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if ((t & 63) == 0) s[k][t >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) top = max(top, s[k][w]);
    const QiRow row(top, t == 0, scales + r);
    for (int64_t c = (int64_t)t * 8; c < cols; c += 1024 * 8) {
      const int nv = cols - c < 8 ? (int)(cols - c) : 8;
      float v[8];
      raw.load(p + c, nv);
      raw.values(v);
      qi_store(dst + r * ld_dst + c, nv, row.codes(v));
    }
  }
}

template <class T, int TEAM, int C>
hipError_t launch(int64_t rows, int64_t cols, const void* src, int64_t ld_src, int8_t* dst, int64_t ld_dst,
                  float* scales, hipStream_t s) {
  constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
  const int64_t all = (rows + TEAMS - 1) / TEAMS, most = 8 * 256 * 256 / THREADS;
  hipLaunchKernelGGL((quantize_i8_kernel<T, TEAM, C>), dim3((unsigned)(all < most ? all : most)), dim3(THREADS), 0, s, rows,
                     cols, (const T*)src, ld_src, dst, ld_dst, scales);
  return hipGetLastError();
}

template <class T>
hipError_t launch_type(int64_t rows, int64_t cols, const void* src, int64_t ld_src, int8_t* dst, int64_t ld_dst,
                       float* scales, hipStream_t s) {
  const int64_t n = (cols + 7) / 8;  // chunks of a row
#define QI(TEAM, C) return launch<T, TEAM, C>(rows, cols, src, ld_src, dst, ld_dst, scales, s)
  if (n <= 16) QI(16, 1);
  if (n <= 32) QI(32, 1);
  if (n <= 64) QI(64, 1);
  if (rows >= 1024) {
    if (n <= 128) QI(64, 2);
    if (n <= 256) QI(64, 4);
    if (n <= 512) QI(256, 2);
    if (n <= 1024) QI(256, 4);
  }
  if (n <= 256) QI(256, 1);
  if (n <= 1024) QI(1024, 1);
  if (n <= 2048) QI(1024, 2);
  if (n <= 4096) QI(1024, 4);
#undef QI
  hipLaunchKernelGGL(quantize_i8_wide_kernel<T>, dim3((unsigned)(rows < 512 ? rows : 512)), dim3(1024), 0, s, rows, cols,
                     (const T*)src, ld_src, dst, ld_dst, scales);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_i8(int64_t rows, int64_t cols, const void* src, int64_t ld_src, int src_kind, int8_t* dst,
                              int64_t ld_dst, float* scales, hipStream_t s) {
  if (src_kind == T_F32) return launch_type<float>(rows, cols, src, ld_src, dst, ld_dst, scales, s);
  return launch_type<uint16_t>(rows, cols, src, ld_src, dst, ld_dst, scales, s);
}

}  // namespace dbgemm
