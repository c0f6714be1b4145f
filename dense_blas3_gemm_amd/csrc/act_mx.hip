// Elementwise kernels of the MLP-block operators: the activation that leaves its argument
// behind in block-scaled E4M3, the backward pass that reads it, the epilogue of a product
// held in fp32, and the column sums that they share (bias gradients).
//
// Rows are walked by workgroups of up to 256 threads, 8 columns to a thread: a thread keeps its
// columns over the rows that its workgroup takes, so a column sum is one register per
// column, written once per thread as a partial row and added up by a second launch in a
// fixed order (no atomics: the same bits every run).
//
// Bound by memory (8192 x 20480 with SiLU and codes: 159 us for 844 MB, 5.3 TB/s); a gradient
// with GELU (erf) by its arithmetic too (2047 x 5000 with all outputs and the sums' launch 22.8 us
// for 72 MB).
#include "epilogue.h"

namespace dbgemm {
namespace {

constexpr int kThreads = 256;

// Threads along the columns (whole blocks of 32 columns: 4 neighbouring threads), rows of
// threads of a workgroup, and the grid: at most max_wgs workgroups.  With partial rows (at most
// max_parts, one per row of workgroups) there are no more rows of workgroups than eighths of the
// matrix's rows or, where those are fewer, than make 512 workgroups: a partial row is written and
// read again.
struct RowGrid {
  dim3 grid, block;
};
RowGrid row_grid(int64_t rows, int64_t cols, int64_t max_wgs, int max_parts) {
  const int64_t chunks = (cols + 31) / 32 * 4;
  const int64_t gx = (chunks + kThreads - 1) / kThreads;
  const int64_t tx = ((chunks + gx - 1) / gx + 3) / 4 * 4, ty = kThreads / tx;
  const int64_t all = (rows + ty - 1) / ty;  // one row to a thread
  int64_t gy = all;
  if (max_parts > 0) {
    const int64_t eight = (rows + 7) / 8, some = (512 + gx - 1) / gx;
    if (gy > eight && gy > some) gy = eight > some ? eight : some;
    if (gy > max_parts) gy = max_parts;
    if (all <= 4) gy = 1;  // (few rows: no second launch)
  }
  const int64_t cap = max_wgs / gx > 1 ? max_wgs / gx : 1;
  if (gy > cap) gy = cap;
  if (gy > 65535) gy = 65535;
  if (gy < 1) gy = 1;
  return {dim3((unsigned)gx, (unsigned)gy), dim3((unsigned)tx, (unsigned)ty)};
}

// The workgroup's column sums: this thread's eight, added over the rows of threads through LDS,
// as one row of `part`, of whole eights, per row of workgroups; or, from a single row of them,
// the sums themselves into `out`.  Every thread calls it (n >= cols: no columns).
__device__ __forceinline__ void put_partial(float* part, float* out, int64_t cols, int64_t n, float (&cs)[8]) {
  __shared__ float s[8][kThreads];
  if (!part && !out) return;
  if (blockDim.y > 1) {
    const int t = threadIdx.y * blockDim.x + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i][t] = cs[i];
    __syncthreads();
    if (threadIdx.y > 0) return;
    for (unsigned y = 1; y < blockDim.y; ++y)
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] += s[i][y * blockDim.x + t];
  }
  if (n >= cols) return;
  if (out)
    ep_store8<false>(out + n, cols - n < 8 ? (int)(cols - n) : 8, cs);
  else
    ep_store8<false>(part + (int64_t)blockIdx.y * whole8(cols) + n, 8, cs);
}

// Epilogue of a product in fp32 (the path of operands that the fused kernels do not take).
__global__ __launch_bounds__(kThreads) void ep_rows_kernel(GemmEpArgs a, int64_t ldw) {
  const int64_t n64 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  const int n = n64 < a.N ? (int)n64 : a.N;  // (a thread past the columns has none)
  const int nv = a.N - n < 8 ? a.N - n : 8;
  float cs[8] = {}, b[8];
  ep_bias8(a, n, nv, b);
  ep_dispatch(a.ep, [&](auto mc, auto ac) EP_INLINE {
    for (int64_t m = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; m < a.M; m += (int64_t)gridDim.y * blockDim.y) {
      float w[8];
      const EpRaw r = ep_fetch8<decltype(mc)::value, true>(a, m, n, nv);
      ep_load8(a.ws + m * ldw + n, nv, w);
      ep_finish8<false, decltype(mc)::value, decltype(ac)::value, true>(a, w, r, b, m, n, nv, cs);
    }
  });
  put_partial(a.ep.colsum, nullptr, a.N, n64, cs);
}

// Sums of the partial rows: 64 columns to a workgroup, four to a thread, the rows dealt to 64
// groups of 16 lanes, whose sums are added in order through LDS.  blockIdx.y: which of the two
// sets of columns of a row.
constexpr int kSumGroups = 64;
__global__ __launch_bounds__(16 * kSumGroups) void colsum_kernel(const float* src, int parts, int64_t ld, int64_t cols,
                                                                 float* out0, float* out1, int accumulate) {
  __shared__ float s[kSumGroups][64 + 4];
  float* out = blockIdx.y ? out1 : out0;
  if (!out) return;
  const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t n = (int64_t)blockIdx.x * 64 + l * 4;
  const float* p = src + blockIdx.y * (ld / 2) + n;
  ep_f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (n < cols) {
#pragma unroll 4
    for (int r = g; r < parts; r += kSumGroups) v += *(const ep_f32x4_u*)(p + (int64_t)r * ld);
  }
  *(ep_f32x4*)&s[g][l * 4] = v;
  __syncthreads();
  // 16 threads to a column: four groups each, then over the 16
  const int c = threadIdx.x >> 4;
  float t = s[4 * l][c] + s[4 * l + 1][c] + s[4 * l + 2][c] + s[4 * l + 3][c];
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) t += __shfl_xor(t, o);
  const int64_t m = (int64_t)blockIdx.x * 64 + c;
  if (l == 0 && m < cols) out[m] = accumulate ? out[m] + t : t;
}

__global__ __launch_bounds__(kThreads) void act_mx_kernel(int64_t rows, int64_t cols, int act, const uint16_t* z,
                                                          int64_t ldz, uint16_t* h, int64_t ldh, uint8_t* q,
                                                          int64_t ldq, uint8_t* sc, int64_t ldsc) {
  const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= (cols + 31) / 32 * 4) return;
  const int64_t n = k * 8;
  const int nv = cols - n < 8 ? (cols > n ? (int)(cols - n) : 0) : 8;
  for (int64_t m = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; m < rows; m += (int64_t)gridDim.y * blockDim.y) {
    float v[8];
    ep_load8<EP_PIECES>(z + m * ldz + n, nv, v);
    ep_store_mx(v, nv, (n & 31) == 0, q + m * ldq + n, sc + m * ldsc + (n >> 5));
    ep_with_act(act, [&](auto ac) EP_INLINE {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = ep_act<decltype(ac)::value>(v[i]);
    });
    ep_store8<true, EP_PIECES>(h + m * ldh + n, nv, v);
  }
}

// eight halves without the first k (0 < k < 8), zeros behind the rest
__device__ __forceinline__ ep_u32x4 drop_halves(ep_u32x4 v, int k) {
  uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  if (k >= 4) {
    lo = hi;
    hi = 0;
    k -= 4;
  }
  if (k > 0) {
    lo = lo >> (16 * k) | hi << (64 - 16 * k);
    hi >>= 16 * k;
  }
  return (ep_u32x4){(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Backward from the checkpoint, kAhead rows of a thread at a time: their loads go out together.
// ODD: cols is no multiple of 8; the others' kernel has no path of partial eights in its rows
// (2047 x 5000 with GELU and all outputs 23 us, with that path 27).
constexpr int kAhead = 4;
template <bool ODD>
__global__ __launch_bounds__(kThreads) void act_grad_mx_kernel(int64_t rows, int64_t cols, int act, const uint8_t* q,
                                                               int64_t ldq, const uint8_t* sc, int64_t ldsc,
                                                               const uint16_t* dh, int64_t lddh, uint16_t* dz,
                                                               int64_t lddz, uint16_t* h, int64_t ldh, float* part,
                                                               float* dbias) {
  const int64_t n = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  const int nv = cols <= n ? 0 : ODD && cols - n < 8 ? (int)(cols - n) : 8;
  if (nv == 0) rows = 0;  // (a thread past the columns)
  // the last columns of an odd row come with the seven or fewer before them, in loads as wide
  // as the others' (a row of fewer than eight columns takes them one by one)
  const int back = ODD && cols >= 8 ? 8 - nv : 0;
  const bool whole = !ODD || cols >= 8;
  const int64_t step = (int64_t)gridDim.y * blockDim.y;
  float cs[8] = {};
  ep_with_act(act, [&](auto ac) EP_INLINE {
    constexpr int ACT = decltype(ac)::value;
    for (int64_t m0 = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; m0 < rows; m0 += kAhead * step) {
      ep_u32x4 codes[kAhead], d[kAhead];  // codes and scale, dh
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t m = m0 + j * step;
        const bool live = m < rows;
        codes[j] = d[j] = (ep_u32x4){0, 0, 0, 0};
        if (live && whole) {
          const ep_u32x2 w = *(const ep_u32x2_u*)(q + m * ldq + n - back);
          codes[j] = (ep_u32x4){w[0], w[1], sc[m * ldsc + (n >> 5)], 0};
          if (dh) d[j] = *(const ep_u32x4_2*)(dh + m * lddh + n - back);
        } else if (ODD && live) {
          codes[j] = ep_raw_part<1>(q + m * ldq + n, nv);
          codes[j][2] = sc[m * ldsc + (n >> 5)];
          if (dh) d[j] = ep_raw_part<2>(dh + m * lddh + n, nv);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t m = m0 + j * step;
        if (m >= rows) break;
        float z[8], g[8];
        if (ODD && back) {
          const uint64_t w = ((uint64_t)codes[j][1] << 32 | codes[j][0]) >> (8 * back);
          codes[j][0] = (uint32_t)w;
          codes[j][1] = (uint32_t)(w >> 32);
          d[j] = drop_halves(d[j], back);
        }
        ep_codes8(codes[j][0], codes[j][1], codes[j][2], z);
        if (dh) {
          EpRaw r;
          r.lo = d[j];
          ep_raw_bf16(r, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            g[i] *= ep_slope<ACT>(z[i]);
            cs[i] += !ODD || i < nv ? g[i] : 0.f;
          }
          if (dz) ep_store8<true, ODD ? EP_PIECES : EP_NONE>(dz + m * lddz + n, nv, g);
        }
        if (h) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = ep_act<ACT>(z[i]);
          ep_store8<true, ODD ? EP_PIECES : EP_NONE>(h + m * ldh + n, nv, z);
        }
      }
    }
  });
  put_partial(part, dbias, cols, n, cs);
}

}  // namespace

hipError_t launch_ep_rows(const GemmEpArgs& a, int64_t ldw, int max_parts, int* parts, hipStream_t s) {
  const RowGrid g = row_grid(a.M, a.N, 2048, a.ep.colsum ? max_parts : 0);
  *parts = (int)g.grid.y;
  hipLaunchKernelGGL(ep_rows_kernel, g.grid, g.block, 0, s, a, ldw);
  return hipGetLastError();
}

hipError_t launch_colsum(const float* src, int parts, int64_t ld, int64_t cols, float* out0, float* out1,
                         int accumulate, hipStream_t s) {
  if (cols == 0) return hipSuccess;
  hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((cols + 63) / 64), out1 ? 2 : 1), dim3(16 * kSumGroups), 0, s, src, parts, ld,
                     cols, out0, out1, accumulate);
  return hipGetLastError();
}

hipError_t launch_act_mx(int64_t rows, int64_t cols, int act, const void* z, int64_t ldz, void* h, int64_t ldh,
                         uint8_t* q, int64_t ldq, uint8_t* sc, int64_t ldsc, hipStream_t s) {
  const RowGrid g = row_grid(rows, cols, 4096, 0);
  hipLaunchKernelGGL(act_mx_kernel, g.grid, g.block, 0, s, rows, cols, act, (const uint16_t*)z, ldz, (uint16_t*)h, ldh,
                     q, ldq, sc, ldsc);
  return hipGetLastError();
}

hipError_t launch_act_grad_mx(int64_t rows, int64_t cols, int act, const uint8_t* q, int64_t ldq, const uint8_t* sc,
                              int64_t ldsc, const void* dh, int64_t lddh, void* dz, int64_t lddz, void* h,
                              int64_t ldh, float* dbias, float* part, int max_parts, int* parts, hipStream_t s) {
  const RowGrid g = row_grid(rows, cols, 2048, dbias ? max_parts : 0);
  // a single row of workgroups has the sums themselves
  *parts = g.grid.y > 1 ? (int)g.grid.y : 0;
  const bool partial = dbias && *parts;
  const auto kernel = cols % 8 ? act_grad_mx_kernel<true> : act_grad_mx_kernel<false>;
  hipLaunchKernelGGL(kernel, g.grid, g.block, 0, s, rows, cols, act, q, ldq, sc, ldsc,
                     (const uint16_t*)dh, lddh, (uint16_t*)dz, lddz, (uint16_t*)h, ldh, partial ? part : nullptr,
                     partial ? nullptr : dbias);
  return hipGetLastError();
}

}  // namespace dbgemm
