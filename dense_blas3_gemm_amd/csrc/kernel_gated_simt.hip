// The gated operators' products for any sizes, strides and alignments (the MFMA kernels take
// whole 16-byte pieces), and the columns that those leave, on the VALU: sums in fp32 or (8-bit
// integers) in exact 32-bit integers, then the epilogue element by element.
//
// 64 x 64 tiles where there are many elements, bound by the LDS and the trip to memory of every step
// (1531 x 2736 x 1001, both B [N][K], 309 us, 54 TFLOP/s).  Where there are few a workgroup has 4 rows
// and 8 columns and its threads divide K: 3 left columns of 4096 x 4099 x 4096 21 us, on tiles 430; 1
// row against two 4099 x 4097 of B 16 us, 4.2 TB/s.
#include "epilogue.h"
#include "gated_internal.h"

namespace dbgemm {
namespace {

constexpr int TS = 64;  // tile edge
constexpr int TK = 16;  // K step
// What the kernel for few elements takes: B [N][K] up to kThin of them, B [K][N], whose rows it reads
// in pieces, few columns or few rows.  With 4097 terms to a sum and both B [N][K], us there and on
// 64 x 64 tiles: 1 x 4099 16 and 465, 64 x 4099 156 and 467, 4096 x 128 221 and 462, 1024 x 1024 432 and
// 461, 4096 x 512 845 and 538; both B [K][N]: 8 x 4099 273 and 468, 16 x 4099 508 and 469, 4096 x 16 234
// and 458, 4096 x 32 466 and 460.
constexpr int64_t kThin = 128 * TS * TS, kThinCols = 16, kThinRows = 8;

template <int IN, class I>
__device__ __forceinline__ auto gs_load(const void* p, I i) {
  if constexpr (IN == GT_I8)
    return (int)((const int8_t*)p)[i];
  else if constexpr (IN == GT_E4M3)
    return __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)p)[i], 0);
  else
    return ep_bf16f(((const uint16_t*)p)[i]);
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

// A sum times alpha, or times the factors of its row and its column (kFarFactor).
template <int IN>
__device__ __forceinline__ float gs_scale(const GatedArgs& a, float w, int64_t m, const float* sb, int64_t n) {
  if constexpr (IN != GT_I8) {
    return w * a.alpha;
  } else {
    const float s = a.ep.sa[m], c = sb[n];
    const bool far = __builtin_fabsf(s) > kFarFactor;
    return w * (far ? c : s) * (far ? s : c);
  }
}

// Element (m, n) from its sums (w2 of the second B); a gradient's results are added to cs.
template <int IN, int OP, int ACT>
__device__ __forceinline__ void gs_finish(const GatedArgs& a, int64_t m, int64_t n, float w, float w2, float& cs,
                                          float& cs2) {
  const GatedEp& e = a.ep;
  const bool f32 = a.c_kind == C_F32;
  w = gs_scale<IN>(a, w, m, e.sb, n);
  if constexpr (OP == GT_GRAD) {
    const float g = ep_bf16f(((const uint16_t*)e.G)[m * e.ldg + n]);
    const float u = ep_bf16f(((const uint16_t*)e.U)[m * e.ldu + n]);
    const float h = ep_act<ACT>(g), dg = w * u * ep_slope<ACT>(g), du = w * h;
    gs_store(a.C, m * a.ldc + n, f32, dg);
    gs_store(e.D2, m * e.ldd2 + n, f32, du);
    if (e.H) gs_store(e.H, m * e.ldh + n, 0, h * u);
    cs += dg;
    cs2 += du;
  } else {
    if (e.bias) w += gs_value(e.bias, n, e.bias_f32);
    float c = ep_act<ACT>(w);
    if constexpr (OP == GT_GATED) {
      w2 = gs_scale<IN>(a, w2, m, e.sb2, n);
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

// 256 threads = 16 x 16, each with 4 rows and 4 columns of a tile.  A workgroup
// takes the row tiles blockIdx.y, + gridDim.y, ... of its columns, whose sums it keeps.
template <int IN, int OP>
__global__ __launch_bounds__(256) void gated_simt_kernel(GatedArgs a) {
  using T = std::conditional_t<IN == GT_I8, int, float>;
  constexpr int NB = OP == GT_GATED ? 2 : 1, PER = TK * TS / 256;
  __shared__ __attribute__((aligned(16))) T As[TK][TS + 4];
  __shared__ __attribute__((aligned(16))) T Bs[NB][TK][TS + 4];
  const GatedEp& e = a.ep;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t n0 = (int64_t)blockIdx.x * TS, tiles_m = ((int64_t)a.M + TS - 1) / TS;
  float cs[2][4] = {};
  for (int64_t tm = blockIdx.y; tm < tiles_m; tm += gridDim.y) {
    const int64_t m0 = tm * TS;
    T acc[NB][4][4] = {};
    // the next step's elements are on their way while this one's are multiplied (what lies past an
    // edge: the last element, as a zero)
    T ra[PER], rb[NB][PER];
    auto fetch = [&](int64_t k0) EP_INLINE {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int x = threadIdx.x + 256 * i;
        const int64_t ka = k0 + x % TK, m = m0 + x / TK;
        const T va = gs_load<IN>(a.A, (m < a.M ? m : a.M - 1) * a.lda + (ka < a.K ? ka : a.K - 1));
        ra[i] = ka < a.K && m < a.M ? va : T(0);
        const int64_t k = k0 + (a.transB ? x % TK : x / TS), n = n0 + (a.transB ? x / TK : x % TS);
        const int64_t kc = k < a.K ? k : a.K - 1, nc = n < a.N ? n : a.N - 1;
        const bool in = k < a.K && n < a.N;
        const T vb = gs_load<IN>(a.B, a.transB ? nc * a.ldb + kc : kc * a.ldb + nc);
        rb[0][i] = in ? vb : T(0);
        if constexpr (NB == 2) {
          const T vb2 = gs_load<IN>(a.B2, a.transB ? nc * a.ldb2 + kc : kc * a.ldb2 + nc);
          rb[1][i] = in ? vb2 : T(0);
        }
      }
    };
    if (a.K > 0) fetch(0);
    for (int64_t k0 = 0; k0 < a.K; k0 += TK) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int x = threadIdx.x + 256 * i;
        As[x % TK][x / TK] = ra[i];
#pragma unroll
        for (int b = 0; b < NB; ++b) Bs[b][a.transB ? x % TK : x / TS][a.transB ? x / TK : x % TS] = rb[b][i];
      }
      __syncthreads();
      if (k0 + TK < a.K) fetch(k0 + TK);
#pragma unroll
      for (int kk = 0; kk < TK; ++kk) {
        using V = T __attribute__((ext_vector_type(4)));
        const V x = *(const V*)&As[kk][ty * 4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const V y = *(const V*)&Bs[b][kk][tx * 4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][i][j] += x[i] * y[j];
        }
      }
      __syncthreads();
    }
    ep_with_act(e.act, [&](auto ac) EP_INLINE {
      constexpr int ACT = decltype(ac)::value;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = n0 + tx * 4 + j;
          if (n < a.N)
            gs_finish<IN, OP, ACT>(a, m, n, (float)acc[0][i][j], (float)acc[NB - 1][i][j], cs[0][j], cs[1][j]);
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
      for (int j = 0; j < 4; ++j) sums[s][ty][tx * 4 + j] = cs[s][j];
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

// Few elements: a workgroup takes 4 rows and 8 columns, its threads every 256th term of each sum, so
// that a long K is read at once and not in steps.  (The row blocks blockIdx.y, + gridDim.y, ..., as
// above.)
constexpr int TR = 4, TC = 8;

template <int IN, int OP, bool KC>
__global__ __launch_bounds__(256, 4) void gated_thin_kernel(GatedArgs a) {
  using T = std::conditional_t<IN == GT_I8, int, float>;
  constexpr int NB = OP == GT_GATED ? 2 : 1;
  constexpr int NV = NB * TR * TC;
  __shared__ T sums[4][NB][TR][TC];
  __shared__ float cols[2][TR][TC];
  const GatedEp& e = a.ep;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t n0 = (int64_t)blockIdx.x * TC, blocks = ((int64_t)a.M + TR - 1) / TR;
  const int r1 = threadIdx.x / TC, c1 = threadIdx.x % TC;  // the first TR x TC threads: an element each
  float cs = 0.f, cs2 = 0.f;
  using E = std::conditional_t<IN == GT_BF16, uint16_t, uint8_t>;
  const E* pb[NB][TC];  // (rows and columns past the last: the last one again)
#pragma unroll
  for (int c = 0; c < TC; ++c) {
    const int64_t n = n0 + c < a.N ? n0 + c : a.N - 1;
    pb[0][c] = (const E*)a.B + (KC ? n * a.ldb : n);
    if constexpr (NB == 2) pb[1][c] = (const E*)a.B2 + (KC ? n * a.ldb2 : n);
  }
  for (int64_t blk = blockIdx.y; blk < blocks; blk += gridDim.y) {
    const int64_t m0 = blk * TR;
    T acc[NB][TR][TC] = {};
    const E* pa[TR];
#pragma unroll
    for (int r = 0; r < TR; ++r) pa[r] = (const E*)a.A + (m0 + r < a.M ? m0 + r : a.M - 1) * a.lda;
#pragma unroll 1
    for (uint32_t k = threadIdx.x; k < (uint32_t)a.K; k += 256) {
      T x[TR], y[NB][TC];
#pragma unroll
      for (int r = 0; r < TR; ++r) x[r] = gs_load<IN>(pa[r], k);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < TC; ++c) {
          if constexpr (KC)
            y[b][c] = gs_load<IN>(pb[b][c], k);
          else
            y[b][c] = gs_load<IN>(pb[b][c], k * (b ? a.ldb2 : a.ldb));
        }
      __builtin_amdgcn_sched_barrier(0);  // every load on its way before the first wait
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < TR; ++r)
#pragma unroll
          for (int c = 0; c < TC; ++c) acc[b][r][c] += x[r] * y[b][c];
    }
    T v[NV];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < TR; ++r)
#pragma unroll
        for (int c = 0; c < TC; ++c) v[(b * TR + r) * TC + c] = acc[b][r][c];
    // over the lanes: each step halves what a lane still has to add, until lane l is left with sum
    // l (or l / 2)
#pragma unroll
    for (int q = 0; q < (NB == 2 ? 6 : 5); ++q) {
      const int o = 32 >> q, h = NV >> (q + 1);
#pragma unroll
      for (int i = 0; i < h; ++i) {
        // (the pair, the other way round in the upper lanes)
        const uint32_t lo = __builtin_bit_cast(uint32_t, v[i]), hi = __builtin_bit_cast(uint32_t, v[i + h]);
        const uint32_t d = (lo ^ hi) & (lane & o ? ~0u : 0u);
        v[i] = __builtin_bit_cast(T, lo ^ d) + __shfl_xor(__builtin_bit_cast(T, hi ^ d), o);
      }
    }
    if constexpr (NB == 1) v[0] += __shfl_xor(v[0], 1);
    if (NB == 2 || lane % 2 == 0) (&sums[wave][0][0][0])[NB == 2 ? lane : lane / 2] = v[0];
    __syncthreads();
    const int64_t m = m0 + r1, n = n0 + c1;
    if (threadIdx.x < TR * TC && m < a.M && n < a.N) {
      T w[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        w[b] = (sums[0][b][r1][c1] + sums[1][b][r1][c1]) + (sums[2][b][r1][c1] + sums[3][b][r1][c1]);
      ep_with_act(e.act, [&](auto ac) EP_INLINE {
        gs_finish<IN, OP, decltype(ac)::value>(a, m, n, (float)w[0], (float)w[NB - 1], cs, cs2);
      });
    }
    __syncthreads();  // the sums are read
  }
  if constexpr (OP == GT_GRAD) {
    if (!e.colsum) return;
    if (threadIdx.x < TR * TC) {
      cols[0][r1][c1] = cs;
      cols[1][r1][c1] = cs2;
    }
    __syncthreads();
    if (threadIdx.x < 2 * TC && n0 + c1 < a.N) {
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < TR; ++r) v += cols[r1][r][c1];
      e.colsum[((int64_t)blockIdx.y * 2 + r1) * whole8(a.N) + n0 + c1] = v;
    }
  }
}

template <int IN, int OP>
void launch_simt(const GatedArgs& a, bool thin, dim3 grid, hipStream_t s) {
  if (thin && a.transB)
    hipLaunchKernelGGL((gated_thin_kernel<IN, OP, true>), grid, dim3(256), 0, s, a);
  else if (thin)
    hipLaunchKernelGGL((gated_thin_kernel<IN, OP, false>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((gated_simt_kernel<IN, OP>), grid, dim3(256), 0, s, a);
}

}  // namespace

bool gated_simt_thin(const GatedArgs& a) {
  return a.transB ? (int64_t)a.M * a.N <= kThin : a.N <= kThinCols || a.M <= kThinRows;
}

hipError_t launch_gated_simt(const GatedArgs& a, int max_parts, int* parts, hipStream_t s) {
  const bool thin = gated_simt_thin(a);
  const int64_t mb = thin ? TR : TS, nb = thin ? TC : TS;
  const int64_t tm = ((int64_t)a.M + mb - 1) / mb, tn = ((int64_t)a.N + nb - 1) / nb;
  int64_t gy = tm < 65535 ? tm : 65535;
  if (a.ep.colsum && gy > max_parts) gy = max_parts;
  if (gy < 1 || tn < 1) return hipErrorInvalidConfiguration;
  *parts = (int)gy;
  const dim3 grid((unsigned)tn, (unsigned)gy);
  switch (a.op * 3 + a.in_kind) {
    case GT_LINEAR * 3 + GT_I8: launch_simt<GT_I8, GT_LINEAR>(a, thin, grid, s); break;
    case GT_GATED * 3 + GT_BF16: launch_simt<GT_BF16, GT_GATED>(a, thin, grid, s); break;
    case GT_GATED * 3 + GT_E4M3: launch_simt<GT_E4M3, GT_GATED>(a, thin, grid, s); break;
    case GT_GATED * 3 + GT_I8: launch_simt<GT_I8, GT_GATED>(a, thin, grid, s); break;
    case GT_GRAD * 3 + GT_BF16: launch_simt<GT_BF16, GT_GRAD>(a, thin, grid, s); break;
    case GT_GRAD * 3 + GT_E4M3: launch_simt<GT_E4M3, GT_GRAD>(a, thin, grid, s); break;
    default: return hipErrorInvalidConfiguration;
  }
  return hipGetLastError();
}

}  // namespace dbgemm
