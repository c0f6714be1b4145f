// Layer norm and its gradient, fp32 statistics.
//
//   forward   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) r gamma + beta;
//             with m the fp32 number next to mu and d = mu - m: mean((x - mu)^2) = mean((x - m)^2) - d^2
//   gradient  xh = (x - mu) r, g = dy gamma,
//             dx = r (g - mean(g) - xh mean(g xh)) [+ dr],
//             dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
//
// Bound by memory: a row is read once and held in registers over its sums, so a pass moves what
// it has to (16384 x 5120 bf16: forward 60 us, 5.6 TB/s; gradient with a residual and both weight
// sums 141, 4.8 TB/s).  One row (1 x 5120: 4.2 us) is launch latency.
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

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
// over the 8, 16 or 32 lanes of a part of a wave
template <class T>
__device__ __forceinline__ T lanes_sum(T v, int lanes) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    if (o < lanes) v += __shfl_xor(v, o);
  return v;
}

// Eight elements of a row as they come from memory; the loads of the next rows are in flight
// in this form while a row is worked on.
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  ep_u16x8 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *(const ep_u16x8_u*)p; }
  __device__ __forceinline__ void set(int i, uint16_t v) { w[i] = v; }
  __device__ __forceinline__ float get(int i) const { return ep_bf16f(w[i]); }
};
template <>
struct Raw8<float> {
  ep_f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *(const ep_f32x4_u*)p;
    b = *(const ep_f32x4_u*)(p + 4);
  }
  __device__ __forceinline__ void set(int i, float v) { (i < 4 ? a : b)[i & 3] = v; }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};
// the first nv (<= 8) elements at p, zeros behind them
template <class T>
__device__ __forceinline__ void raw_load(Raw8<T>& r, const T* p, int nv) {
  if (nv >= 8) {
    r.load(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.set(i, i < nv ? p[i] : T(0));
  }
}

// The mean of a row from its sum: m and d = mu - m.  Sums of fp32 rows are taken in 64 bits: in 32 a
// constant row is one or more units from its own mean, all columns alike, and normalises to +-0.02
// at 1000.1 and to +-1 at 1e6 + 0.3 where it is 0; in 64 its mean is exact and d = 0.  Sums of up to
// 2^15 bf16 values of one size are exact in fp32 (8 bits each), and others have a spread that its
// rounding does not show in: d is 0 there (in 64 bits 16384 x 5120 took 69 us, with d 63, so 59).
struct Mean {
  float m, d;
  __device__ Mean(double sum, int cols) {
    const double mu = sum / cols;
    m = (float)mu;
    d = (float)(mu - m);
    d = d == d ? d : 0.f;  // (an infinite mean)
  }
  __device__ Mean(float sum, int cols) : m(sum / (float)cols), d(0.f) {}
};
template <class X>
using RowSum = std::conditional_t<sizeof(X) == 2, float, double>;
__device__ __forceinline__ float row_rstd(float sq, float n, float d, float eps) {
  return 1.0f / __builtin_sqrtf(sq / n - d * d + eps);
}
// (x - m) r as (x - mu) r
template <class X>
__device__ __forceinline__ float row_norm(float v, float rs, float off) {
  return sizeof(X) == 2 ? v * rs : v * rs + off;
}

// ---- the row kernels.  A team of blockDim.x threads (whole waves, or for narrow rows 8, 16 or
// 32 lanes of one) holds a row in registers:
// thread t its columns 8 (t + c blockDim.x) .. + 7 for c < CPT.  blockDim.y teams make up a
// workgroup, and a workgroup walks the rows with R rows per team at a time: one exchange over
// the waves of a team serves R rows, the weights stay in registers, and the next R rows'
// loads are issued before the present rows' sums are waited for.  Wide rows (CPT = 4) have no
// registers for either: the weights are read where they are used and the rows one by one.
struct Team {
  int t, T, waves, wave;  // thread and wave within the team (waves: 0 for part of a wave)
  int first_wave;         // the team's first wave within the workgroup
  __device__ Team()
      : t(threadIdx.x), T(blockDim.x), waves(blockDim.x >> 6), wave(threadIdx.x >> 6),
        first_wave(threadIdx.y * (blockDim.x >> 6)) {}
};

// Sums over the team of V values per thread, the same in every thread.  s: two halves of 16 x V
// values (of the widest V and T), used in turn: the barrier of the use between two of one half
// keeps them apart.  Every team of the workgroup calls it together.
template <int V, class T, int BYTES>
__device__ __forceinline__ void team_sum(const Team& m, T (&v)[V], char (&s)[BYTES], int& half) {
  static_assert(16 * V * sizeof(T) <= BYTES / 2, "a half holds it");
  if (m.waves == 0) {  // (uniform over the workgroup, and so is the next)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = lanes_sum(v[i], m.T);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = wave_sum(v[i]);
  if (m.waves == 1) return;
  T* h = (T*)(s + half * (BYTES / 2));
  half ^= 1;
  if ((m.t & 63) == 0)
#pragma unroll
    for (int i = 0; i < V; ++i) h[(m.first_wave + m.wave) * V + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0;
  for (int w = 0; w < m.waves; ++w)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += h[(m.first_wave + w) * V + i];
}

// Waves to a SIMD that the registers have to leave room for: three workgroups of five waves to a CU
// (5120 columns) take five on one SIMD.  (Left to the compiler, fp32 rows take 106-108 registers.)
template <class X, int CPT, int R, int MAXT>
constexpr int fwd_waves() {
  return sizeof(X) == 4 && CPT == 2 && R == 1 && MAXT == 512 ? 5 : 1;
}

// Forward: reads x once, writes y once.  Bound by those bytes.
template <class X, class Y, int CPT, int R, int MAXT>
__global__ __launch_bounds__(MAXT, (fwd_waves<X, CPT, R, MAXT>())) void layernorm_kernel(NormArgs a) {
  constexpr bool kWide = CPT >= 4;
  __shared__ __attribute__((aligned(16))) char s[2 * 16 * R * sizeof(RowSum<X>)];
  const Team m;
  int half = 0;
  const X* x = (const X*)a.x;
  Y* y = (Y*)a.y;
  int col[CPT], nv[CPT];
  float g[kWide ? 1 : CPT][8], b[kWide ? 1 : CPT][8];
  auto weights = [&](int c, float (&gc)[8], float (&bc)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gc[i] = 1.f;
      bc[i] = 0.f;
    }
    if (a.gamma) ep_load8(a.gamma, col[c], a.w_kind, nv[c], gc);
    if (a.beta) ep_load8(a.beta, col[c], a.w_kind, nv[c], bc);
  };
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    col[c] = 8 * (m.t + c * m.T);
    nv[c] = min(max(a.cols - col[c], 0), 8);
    if constexpr (!kWide) weights(c, g[c], b[c]);
  }
  const int64_t step = (int64_t)gridDim.x * blockDim.y * R;
  const int64_t mine = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * R;
  Raw8<X> in[R][CPT];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int c = 0; c < CPT; ++c) raw_load(in[j][c], x + (r + j) * a.ldx + col[c], r + j < a.rows ? nv[c] : 0);
  };
  if constexpr (!kWide) load(mine);
  const float n = (float)a.cols;
  // (the workgroup's teams run the same number of rounds: they share the barriers)
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y * R; r0 < a.rows; r0 += step) {
    const int64_t r = r0 + (mine - (int64_t)blockIdx.x * blockDim.y * R);
    float v[R][CPT][8], q[R];
    RowSum<X> sum[R];
    if constexpr (kWide) load(r);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      sum[j] = 0;
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[j][c][i] = in[j][c].get(i);
          sum[j] += v[j][c][i];
        }
    }
    if constexpr (!kWide)
      if (r0 + step < a.rows) load(r + step);
    team_sum(m, sum, s, half);
    float mu[R], d[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const Mean mean(sum[j], a.cols);
      mu[j] = mean.m;
      d[j] = mean.d;
      q[j] = 0.f;
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[j][c][i] -= mu[j];
          q[j] += i < nv[c] ? v[j][c][i] * v[j][c][i] : 0.f;
        }
    }
    team_sum(m, q, s, half);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (r + j >= a.rows) continue;
      const float rs = row_rstd(q[j], n, d[j], a.eps), off = -d[j] * rs;
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        if (nv[c] == 0) continue;
        if constexpr (kWide) weights(c, g[0], b[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[j][c][i] = row_norm<X>(v[j][c][i], rs, off) * g[kWide ? 0 : c][i] + b[kWide ? 0 : c][i];
        ep_store8<true>(y + (r + j) * a.ldy + col[c], nv[c], v[j][c]);
      }
      if (m.t == 0) {
        if (a.mean) a.mean[r + j] = mu[j];
        if (a.rstd) a.rstd[r + j] = rs;
      }
    }
  }
}

// Gradient: reads x, dy (and dr) once, writes dx once; SUMS: a thread adds up dgamma and dbeta
// of its columns over all rows of its team, the teams of a workgroup are added through LDS,
// and each workgroup leaves one partial row.
template <class X, class Y, int CPT, int R, int MAXT, bool SUMS>
__global__ __launch_bounds__(MAXT) void layernorm_grad_kernel(NormArgs a) {
  constexpr bool kWide = CPT >= 4;
  static_assert(!(kWide && SUMS), "no registers for the sums of a wide row");
  constexpr bool kAhead = !kWide && (CPT == 1 || MAXT <= 512);  // the next rows' loads ahead
  __shared__ __attribute__((aligned(16))) char s[2 * 16 * 2 * R * sizeof(float)];
  const Team m;
  int half = 0;
  const X* x = (const X*)a.x;
  const Y* dy = (const Y*)a.dy;
  X* dx = (X*)a.y;
  int col[CPT], nv[CPT];
  float gam[kWide ? 1 : CPT][8], dg[SUMS ? CPT : 1][8] = {}, db[SUMS ? CPT : 1][8] = {};
  auto weights = [&](int c, float (&gc)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) gc[i] = 1.f;
    if (a.gamma) ep_load8(a.gamma, col[c], a.w_kind, nv[c], gc);
  };
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    col[c] = 8 * (m.t + c * m.T);
    nv[c] = min(max(a.cols - col[c], 0), 8);
    if constexpr (!kWide) weights(c, gam[c]);
  }
  const int64_t step = (int64_t)gridDim.x * blockDim.y * R;
  const int64_t mine = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * R;
  Raw8<X> xin[R][CPT];
  Raw8<Y> gin[R][CPT];
  float mu[R], rs[R];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool live = r + j < a.rows;
      mu[j] = live ? a.mean[r + j] : 0.f;
      rs[j] = live ? a.rstd[r + j] : 0.f;
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        raw_load(xin[j][c], x + (r + j) * a.ldx + col[c], live ? nv[c] : 0);
        raw_load(gin[j][c], dy + (r + j) * a.lddy + col[c], live ? nv[c] : 0);
      }
    }
  };
  if constexpr (kAhead) load(mine);
  const float n = (float)a.cols;
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y * R; r0 < a.rows; r0 += step) {
    const int64_t r = r0 + (mine - (int64_t)blockIdx.x * blockDim.y * R);
    // (a wide row's xh and g are formed twice instead of being held)
    float xh[R][kWide ? 1 : CPT][8], g[R][kWide ? 1 : CPT][8], c12[2 * R], rr[R];
    if constexpr (!kAhead) load(r);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float c1 = 0.f, c2 = 0.f;
      rr[j] = rs[j];
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        if constexpr (kWide) weights(c, gam[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (a column past the row has dy = 0 and adds nothing)
          const float d = gin[j][c].get(i);
          const float xn = (xin[j][c].get(i) - mu[j]) * rs[j], gn = d * gam[kWide ? 0 : c][i];
          c1 += gn;
          c2 += gn * xn;
          if constexpr (!kWide) {
            xh[j][c][i] = xn;
            g[j][c][i] = gn;
          }
          if constexpr (SUMS) {
            dg[c][i] += d * xn;
            db[c][i] += d;
          }
        }
      }
      c12[2 * j] = c1;
      c12[2 * j + 1] = c2;
    }
    Raw8<X> res[R][kWide ? 1 : CPT];
    if constexpr (!kWide) {
      if (a.dr) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int c = 0; c < CPT; ++c)
            raw_load(res[j][c], (const X*)a.dr + (r + j) * a.lddr + col[c], r + j < a.rows ? nv[c] : 0);
      }
    }
    if constexpr (kAhead)
      if (r0 + step < a.rows) load(r + step);
    team_sum(m, c12, s, half);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (r + j >= a.rows) continue;
      const float c1 = c12[2 * j] / n, c2 = c12[2 * j + 1] / n;
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        if (nv[c] == 0) continue;
        if constexpr (kWide) {
          weights(c, gam[0]);
          if (a.dr) raw_load(res[j][0], (const X*)a.dr + (r + j) * a.lddr + col[c], nv[c]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            xh[j][0][i] = (xin[j][c].get(i) - mu[j]) * rs[j];
            g[j][0][i] = gin[j][c].get(i) * gam[0][i];
          }
        }
        const int k = kWide ? 0 : c;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = rr[j] * (g[j][k][i] - c1 - xh[j][k][i] * c2);
          if (a.dr) v[i] += res[j][k].get(i);
        }
        ep_store8<true>(dx + (r + j) * a.ldy + col[c], nv[c], v);
      }
    }
  }
  if constexpr (SUMS) {
    // the teams' sums, one set of eight columns at a time: team y > 0 leaves its own in LDS
    // and team 0 adds them in order
    __shared__ float t8[8 * 1024];
    // (a single workgroup has the sums themselves)
    const bool one = gridDim.x == 1;
    float* const out[2] = {one ? a.dgamma : a.part + (int64_t)blockIdx.x * 2 * whole8(a.cols),
                           one ? a.dbeta : a.part + ((int64_t)blockIdx.x * 2 + 1) * whole8(a.cols)};
    // the teams of one wave by exchange, then a row of sums per wave (or team) through LDS: added
    // up by the first team alone, 32 teams of 16 lanes took a microsecond (27214 x 128: 13.6, so 12.4)
    const unsigned rows = m.T < 64 ? (blockDim.y * m.T + 63) / 64 : blockDim.y;
    const unsigned mine_row = m.T < 64 ? (threadIdx.y * m.T + m.t) >> 6 : threadIdx.y;
    const bool lead = m.T >= 64 || (threadIdx.y * m.T) % 64 == 0;
    auto put = [&](float (&v)[8], int c, int set) {
      for (int o = m.T; o < 64; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += __shfl_xor(v[i], o);
      if (rows > 1) {
        __syncthreads();
        if (lead && mine_row > 0)
#pragma unroll
          for (int i = 0; i < 8; ++i) t8[i * 1024 + mine_row * m.T + m.t] = v[i];
        __syncthreads();
        if (threadIdx.y == 0)
          for (unsigned k = 1; k < rows; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += t8[i * 1024 + k * m.T + m.t];
      }
      if (threadIdx.y == 0 && nv[c] > 0 && out[set]) ep_store8<false>(out[set] + col[c], one ? nv[c] : 8, v);
    };
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      put(dg[c], c, 0);
      put(db[c], c, 1);
    }
  }
}

// ---- rows too wide for the registers of a workgroup
// Sums of two values over a workgroup of 256 threads, the same in every thread.
template <class T>
__device__ __forceinline__ void group_sum(T& u, T& v, T (*s)[2]) {
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
  __shared__ double s[4][2];
  const uint32_t cols = (uint32_t)a.cols;  // (up to 2^31 - 1: an int index would pass its end by one step)
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    double sum = 0.0, sq = 0.0, none = 0.0;
    for (uint32_t i = threadIdx.x; i < cols; i += 256) sum += ln_load(a.x, r * a.ldx + i, a.x_kind);
    group_sum(sum, none, s);
    const Mean mean(sum, a.cols);
    const float mu = mean.m;
    float q = 0.f;
    for (uint32_t i = threadIdx.x; i < cols; i += 256) {
      const float d = ln_load(a.x, r * a.ldx + i, a.x_kind) - mu;
      q += d * d;
    }
    sq = q;
    group_sum(sq, none, s);
    const float rs = row_rstd((float)sq, (float)a.cols, mean.d, a.eps), off = -mean.d * rs;
    for (uint32_t i = threadIdx.x; i < cols; i += 256) {
      float v = (ln_load(a.x, r * a.ldx + i, a.x_kind) - mu) * rs + off;
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
  const uint32_t cols = (uint32_t)a.cols;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float mu = a.mean[r], rs = a.rstd[r];
    float c1 = 0.f, c2 = 0.f;
    for (uint32_t i = threadIdx.x; i < cols; i += 256) {
      float g = ln_load(a.dy, r * a.lddy + i, a.y_kind);
      if (a.gamma) g *= ln_load(a.gamma, i, a.w_kind);
      c1 += g;
      c2 += g * ((ln_load(a.x, r * a.ldx + i, a.x_kind) - mu) * rs);
    }
    group_sum(c1, c2, s);
    c1 /= (float)a.cols;
    c2 /= (float)a.cols;
    for (uint32_t i = threadIdx.x; i < cols; i += 256) {
      float g = ln_load(a.dy, r * a.lddy + i, a.y_kind);
      if (a.gamma) g *= ln_load(a.gamma, i, a.w_kind);
      const float xh = (ln_load(a.x, r * a.ldx + i, a.x_kind) - mu) * rs;
      float v = rs * (g - c1 - xh * c2);
      if (a.dr) v += ln_load(a.dr, r * a.lddr + i, a.x_kind);
      ln_store(a.y, r * a.ldy + i, a.x_kind, v);
    }
  }
}

// Partial sums of dgamma and dbeta: a thread to eight columns, workgroup row y takes rows y,
// y + gridDim.y, ...
template <class X, class Y>
__global__ __launch_bounds__(256) void layernorm_dw_kernel(NormArgs a) {
  const int col = 8 * (blockIdx.x * 256 + threadIdx.x);
  if (col >= a.cols) return;
  const int nv = min(a.cols - col, 8);
  float dg[8] = {}, db[8] = {};
#pragma unroll 2
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    Raw8<X> x;
    Raw8<Y> d;
    raw_load(x, (const X*)a.x + r * a.ldx + col, nv);
    raw_load(d, (const Y*)a.dy + r * a.lddy + col, nv);
    const float mu = a.mean[r], rs = a.rstd[r];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dg[i] += d.get(i) * ((x.get(i) - mu) * rs);
      db[i] += d.get(i);
    }
  }
  const bool one = gridDim.y == 1;  // (the sums themselves)
  float* og = one ? a.dgamma : a.part + (int64_t)blockIdx.y * 2 * whole8(a.cols);
  float* ob = one ? a.dbeta : a.part + ((int64_t)blockIdx.y * 2 + 1) * whole8(a.cols);
  if (og) ep_store8<false>(og + col, one ? nv : 8, dg);
  if (ob) ep_store8<false>(ob + col, one ? nv : 8, db);
}

// Threads of a team for rows of `cols` columns at `cpt` chunks of 8 to a thread: whole waves, or
// as few lanes of one as do (8 at least).
unsigned team_threads(int64_t cols, int cpt) {
  const int64_t t = (cols + 8 * cpt - 1) / (8 * cpt);
  if (t > 32) return (unsigned)((t + 63) / 64) * 64;
  return t > 16 ? 32 : t > 8 ? 16 : 8;
}

template <class X, class Y, int CPT, int R, int MAXT>
hipError_t fwd(const NormArgs& a, hipStream_t s) {
  constexpr unsigned wg = 256, per_cu = 1024;
  const unsigned T = team_threads(a.cols, CPT);
  const unsigned teams = T < wg ? wg / T : 1;
  const int64_t need = (a.rows + (int64_t)teams * R - 1) / ((int64_t)teams * R);
  const int64_t most = 256 * (per_cu / (T * teams) ? per_cu / (T * teams) : 1);
  hipLaunchKernelGGL((layernorm_kernel<X, Y, CPT, R, MAXT>), dim3((unsigned)(need < most ? need : most)),
                     dim3(T, teams), 0, s, a);
  return hipGetLastError();
}

template <class X, class Y, int CPT, int R, int MAXT, bool SUMS>
hipError_t grad(const NormArgs& a, int max_parts, int* parts, hipStream_t s) {
  constexpr unsigned wg = 512;
  const unsigned T = team_threads(a.cols, CPT);
  unsigned teams = T < wg ? wg / T : 1;
  const bool few = SUMS && a.rows <= (int64_t)teams * R * 2;  // two rounds of one workgroup, no second launch
  // else spread the rows over the CUs (a workgroup stays whole waves); with sums of two chunks, one
  // workgroup to a CU, as long as that stays one round of them (1681 x 1488: 14.1 us, so 12.4)
  while (!few && teams > 1 && teams * T > 64 && (int64_t)teams * R * 256 > a.rows &&
         !(SUMS && CPT > 1 && (int64_t)((teams + 1) / 2) * R * 256 < a.rows))
    teams = (teams + 1) / 2;
  const int64_t need = (a.rows + (int64_t)teams * R - 1) / ((int64_t)teams * R);
  // With the weights' sums one workgroup to a CU: a partial row more per CU costs more (its
  // write and its read) than a second workgroup's overlap gains, 128.4 against 136.6 us at
  // 16384 x 5120 without a residual.  Narrow rows (one chunk a thread, no spills at 128 registers) take two.
  int64_t most = 256 * (SUMS && CPT > 1 ? 1 : 1024 / (T * teams) ? 1024 / (T * teams) : 1);
  if (SUMS && most > max_parts) most = max_parts;
  if (few) most = 1;
  const unsigned n = (unsigned)(need < most ? need : most);
  *parts = SUMS && n > 1 ? (int)n : 0;
  hipLaunchKernelGGL((layernorm_grad_kernel<X, Y, CPT, R, MAXT, SUMS>), dim3(n), dim3(T, teams), 0, s, a);
  return hipGetLastError();
}

// Chunks per thread, rows at a time, by width and rows (MI355X, bf16): at 16384 x 5120 two
// chunks (teams of 320 threads, three workgroups to a CU) take 59.6 us and one chunk 91.8-95;
// at 65536 x 768 two rows at a time 39.8, one 43.5.  A few rows finish sooner with more
// threads to each (1 x 5120: 3.4 against 3.9).
template <class X, class Y>
hipError_t fwd_xy(const NormArgs& a, hipStream_t s) {
  if (a.cols <= 8192) {
    if (a.rows <= 256) return fwd<X, Y, 1, 1, 1024>(a, s);
    return a.cols <= 1024 ? fwd<X, Y, 2, 2, 512>(a, s) : fwd<X, Y, 2, 1, 512>(a, s);
  }
  if (a.cols <= 16384) return fwd<X, Y, 2, 1, 1024>(a, s);
  if (a.cols <= 32768) return fwd<X, Y, 4, 1, 1024>(a, s);
  const unsigned g = (unsigned)(a.rows < 65536 ? a.rows : 65536);
  hipLaunchKernelGGL(layernorm_rows_kernel, dim3(g), dim3(256), 0, s, a);
  return hipGetLastError();
}

// The same for the gradient: at 16384 x 5120 two chunks and two rows at a time take 128.4 us (no residual)
// with the sum of the partials, one row 157, one chunk 137; at 65536 x 768 one chunk and two
// rows 109, two chunks 125.
template <class X, class Y, bool SUMS>
hipError_t grad_fit(const NormArgs& a, int max_parts, int* parts, hipStream_t s) {
  constexpr int kBytes = sizeof(X) + sizeof(Y);  // (R as far as the registers go)
  if (a.cols <= 1024) return grad<X, Y, 1, (kBytes > 4 ? 1 : 2), 1024, SUMS>(a, max_parts, parts, s);
  if (a.cols <= 8192) {
    if (a.rows <= 256) return grad<X, Y, 1, 1, 1024, SUMS>(a, max_parts, parts, s);
    return grad<X, Y, 2, (kBytes > 6 ? 1 : 2), 512, SUMS>(a, max_parts, parts, s);
  }
  return grad<X, Y, 2, 1, 1024, SUMS>(a, max_parts, parts, s);  // up to 16384
}

template <class X, class Y>
hipError_t grad_xy(const NormArgs& a, int max_parts, int* parts, hipStream_t s) {
  if (a.cols <= 16384)
    return a.part ? grad_fit<X, Y, true>(a, max_parts, parts, s) : grad_fit<X, Y, false>(a, 0, parts, s);
  // wider: dx and the weights' sums apart (the sums' registers would not fit beside the row)
  NormArgs d = a;
  d.part = nullptr;
  hipError_t e;
  if (a.cols <= 32768) {
    int none = 0;
    e = grad<X, Y, 4, 1, 1024, false>(d, 0, &none, s);
  } else {
    const unsigned g = (unsigned)(a.rows < 65536 ? a.rows : 65536);
    hipLaunchKernelGGL(layernorm_dx_kernel, dim3(g), dim3(256), 0, s, d);
    e = hipGetLastError();
  }
  *parts = 0;
  if (e != hipSuccess || !a.part) return e;
  const int64_t gx = (a.cols + 2047) / 2048;
  int64_t gy = 2048 / gx;
  if (gy > max_parts) gy = max_parts;
  if (gy > a.rows) gy = a.rows;
  if (gy < 1) gy = 1;
  *parts = gy > 1 ? (int)gy : 0;
  hipLaunchKernelGGL((layernorm_dw_kernel<X, Y>), dim3((unsigned)gx, (unsigned)gy), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layernorm(const NormArgs& a, hipStream_t s) {
  if (a.x_kind == T_F32)
    return a.y_kind == T_F32 ? fwd_xy<float, float>(a, s) : fwd_xy<float, uint16_t>(a, s);
  return a.y_kind == T_F32 ? fwd_xy<uint16_t, float>(a, s) : fwd_xy<uint16_t, uint16_t>(a, s);
}

hipError_t launch_layernorm_grad(const NormArgs& a, int max_parts, int* parts, hipStream_t s) {
  if (a.x_kind == T_F32)
    return a.y_kind == T_F32 ? grad_xy<float, float>(a, max_parts, parts, s)
                             : grad_xy<float, uint16_t>(a, max_parts, parts, s);
  return a.y_kind == T_F32 ? grad_xy<uint16_t, float>(a, max_parts, parts, s)
                           : grad_xy<uint16_t, uint16_t>(a, max_parts, parts, s);
}

}  // namespace dbgemm
