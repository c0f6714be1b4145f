// Products of a few rows with an epilogue: C = act(alpha A op(B) + bias) + beta R (or its
// gradient form) for A [M][K] of at most 64 rows, as a serving loop has them.
//
// Bound by the bytes of B, which is read once.  What counts is how many of them are in flight,
// that they are asked for in whole lines, and that one launch does it all:
//
//   * a workgroup takes BN columns over the whole of K; its waves take the K tiles in turn and
//     their sums meet in LDS, so no partial sums go through memory and no second launch adds
//     them up (the tiled kernels' split-K: 9.6 + 3.8 us at 1 x 4096 x 4096);
//   * every wave works alone, on a ring of LDS slots of its own, filled by direct-to-LDS loads:
//     the loads in flight cost no registers, and there is no barrier before the end;
//   * eight neighbouring lanes fetch one line of 128 bytes.  (B [N][K] straight into registers,
//     in the lanes that the MFMA wants, has neighbouring lanes on 16 different rows: 16.3 us
//     against 11.1 for the same bytes by lines, 13 x 5120 x 5120.)
//
// The gated operators' kernels are built from the same source (DBGEMM_GATED): two B as two
// sub-tiles of every slot, 8-bit integers whose sums meet as whole numbers.
#include "epilogue.h"
#include "mfma_common.h"
#ifdef DBGEMM_GATED
#include <cmath>

#include "gated_tile.h"
#endif

namespace dbgemm {
namespace {

#ifdef DBGEMM_GATED
using KernelArgs = GatedArgs;
#else
using KernelArgs = GemmEpArgs;
#endif

template <class C, int WAVES_>
struct Skinny {
  static constexpr int WAVES = WAVES_, THREADS = WAVES * 64, S = C::STAGES;
  static_assert(C::WM == 1 && C::WN == 1 && C::MT == 16 && (C::IN == IN_BF16 || C::IN == IN_E4M3_LDS || C::I8),
                "a wave's tile");
  static constexpr int SLOT = C::A_BYTES + C::B_BYTES;
  static_assert(C::A_BYTES % 1024 == 0 && C::SUB_BYTES % 1024 == 0, "whole 1 KiB copies");
  static constexpr int A_CP = C::A_BYTES / 1024, SUB_CP = C::SUB_BYTES / 1024, B_CP = SUB_CP * C::NSUB, CP = A_CP + B_CP;
  static_assert(S * CP <= 63, "vmcnt range");
  static constexpr int LDR = C::BN + 4;  // floats per row of a wave's sums
  static constexpr int RING = WAVES * S * SLOT, SUMS = WAVES * C::BM * LDR * 4;
  static constexpr int LDS_BYTES = RING > SUMS ? RING : SUMS;
  static_assert(LDS_BYTES <= 160 * 1024, "LDS of one CU");
};

template <int N, int FIRST, class O>
__device__ __forceinline__ void skinny_copies(uint32_t l, const O& o, __amdgpu_buffer_rsrc_t r) {
  if constexpr (FIRST < N) {
    constexpr int n = N - FIRST < 4 ? N - FIRST : 4;
    uint32_t v[n];
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = o(FIRST + i);
    pp_copies<n, false>(l + FIRST * 1024u, v, r);
    skinny_copies<N, FIRST + n>(l, o, r);
  }
}

// Workgroup id -> its columns, for B [K][N].  Each XCD (id b runs on XCD b % 8) should read
// whole lines of a row of B, and from all of its L2's channels: 256 bytes of addresses go to a
// channel, and rows of a multiple of 2 KiB repeat the pattern, so an XCD with one contiguous run
// of 1280 bytes of every row has 10 of 16 channels to read from (13 x 5120 x 5120: 16.6 us).
// So pairs of XCDs share a run of the row, its lines of 128 bytes to one and the other in turn.
// PER: workgroups to a line.
template <int PER>
__device__ __forceinline__ int line_remap(int b, int total) {
  const int lines = total / PER, runs = lines / 8 * 8;  // lines dealt out this way
  if (b >= runs * PER) return b;
  const int x = b & 7, j = b >> 3;
  return (2 * ((x >> 1) * (runs / 8) + j / PER) + (x & 1)) * PER + j % PER;
}

// OP: what a gated operator's kernel does with its sums.
template <class C, int WAVES, int OP = 0>
__global__ __launch_bounds__(WAVES * 64) void gemm_skinny_kernel(KernelArgs a) {
  using P = Skinny<C, WAVES>;
  __shared__ __attribute__((aligned(1024))) char lds[P::LDS_BYTES];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  // (B [N][K]: a run of columns to each XCD)
  const int tn = C::B_KC ? xcd_remap(blockIdx.x, gridDim.x, 8)
                         : line_remap<(128 > C::SUB_BN * C::ES ? 128 / (C::SUB_BN * C::ES) : 1)>(blockIdx.x, gridDim.x);
  const int n0 = tn * C::SUB_BN;

  // ---- the epilogue's operands: thread t < OUT takes eight columns of a row at the end
  constexpr int LPR = C::SUB_BN / 8, OUT = C::BM * LPR;
  static_assert(OUT <= P::THREADS, "one step");
  const int om = t / LPR, on = n0 + (t % LPR) * 8;
  const int nv = t < OUT && om < a.M && on < a.N ? 8 : 0;
#ifdef DBGEMM_GATED
  const GtCols<C::I8, OP> cols(a, on, nv);
  const GtRaw raw = gt_fetch8<false, C::I8, OP>(a, om, on, nv);
#else
  static_assert(LPR % 4 == 0, "whole blocks of 32 columns");
  float bias[8];
  ep_bias8(a, on, nv, bias);
  const EpRaw raw = !a.ep.grad                ? ep_fetch8<EP_FORWARD, false>(a, om, on, nv)
                    : a.ep.z_kind == Z_MX ? ep_fetch8<EP_GRAD_MX, false>(a, om, on, nv)
                                          : ep_fetch8<EP_GRAD_BF16, false>(a, om, on, nv);
#endif

  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, (uint32_t)(a.M * a.lda * C::ES));
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(a.B, (uint32_t)((C::B_KC ? (int64_t)a.N : (int64_t)a.K) * a.ldb * C::ES));
  const __amdgpu_buffer_rsrc_t rb2 =
      C::DUAL ? make_rsrc(a.B2, (uint32_t)((C::B_KC ? (int64_t)a.N : (int64_t)a.K) * a.ldb2 * C::ES)) : rb;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds0 + (uint32_t)(wave * P::S * P::SLOT));

  // ---- this lane's chunks: copy i of an operand fills LDS chunks 64 i .. + 63 of its tile, chunk
  // p = 64 i + lane being row p / CPR, physical chunk p % CPR, which holds logical chunk
  // (p % CPR) ^ swizzle(row).  Byte offset of it in K tile 0 (past every buffer for a row past
  // M or a column past N), and its K index within a tile.
  // (A second B has its sub-tile behind the first one's, and other offsets where its stride differs.)
  uint32_t a_off[P::A_CP], b_off[P::B_CP];
  int a_k[P::A_CP], b_k[P::B_CP];
#pragma unroll
  for (int i = 0; i < P::A_CP; ++i) {
    const int p = i * 64 + lane, r = p / C::A_CPR, c = (p % C::A_CPR) ^ pp_swz<C, true, C::A_CPR>(r);
    a_off[i] = r < a.M ? (uint32_t)((r * a.lda + c * C::VEC) * C::ES) : kOOB;
    a_k[i] = c * C::VEC;
  }
#pragma unroll
  for (int i = 0; i < P::B_CP; ++i) {
    const int p = i % P::SUB_CP * 64 + lane, r = p / C::SUB_CPR, c = (p % C::SUB_CPR) ^ pp_swz<C, C::B_KC, C::SUB_CPR>(r);
    const int64_t ldb = i < P::SUB_CP ? a.ldb : a.ldb2;
    if constexpr (C::B_KC) {
      b_off[i] = n0 + r < a.N ? (uint32_t)(((n0 + r) * ldb + c * C::VEC) * C::ES) : kOOB;
      b_k[i] = c * C::VEC;
    } else {
      b_off[i] = n0 + c * C::VEC < a.N ? (uint32_t)((r * ldb + n0 + c * C::VEC) * C::ES) : kOOB;
      b_k[i] = r;
    }
  }
  const uint32_t b_step = C::B_KC ? C::BK * C::ES : (uint32_t)(C::BK * a.ldb * C::ES);
  const uint32_t b2_step = C::B_KC ? C::BK * C::ES : (uint32_t)(C::BK * a.ldb2 * C::ES);
  // copies of this wave's tile number it (K tile wave + it * WAVES) into slot u; what lies past K
  // reads zeros and touches no memory
  auto copy_tile = [&](int it, int u) {
    const int kt = wave + it * WAVES, left = a.K - kt * C::BK;
    const uint32_t ao = (uint32_t)(kt * C::BK * C::ES), bo = (uint32_t)kt * b_step;
    const uint32_t l = __builtin_amdgcn_readfirstlane(ring + (uint32_t)(u * P::SLOT));
    skinny_copies<P::SUB_CP, 0>(
        l + C::A_BYTES, [&](int i) { return b_k[i] < left && b_off[i] != kOOB ? b_off[i] + bo : kOOB; }, rb);
    if constexpr (C::DUAL) {
      const uint32_t bo2 = (uint32_t)kt * b2_step;
      auto o = [&](int i) {
        return b_k[P::SUB_CP + i] < left && b_off[P::SUB_CP + i] != kOOB ? b_off[P::SUB_CP + i] + bo2 : kOOB;
      };
      skinny_copies<P::SUB_CP, 0>(l + C::A_BYTES + C::SUB_BYTES, o, rb2);
    }
    skinny_copies<P::A_CP, 0>(l, [&](int i) { return a_k[i] < left && a_off[i] != kOOB ? a_off[i] + ao : kOOB; }, ra);
  };

  constexpr int FSUB = C::FN / C::NSUB;
  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{};
  // fragment read h of the 16 rows or columns from x0 on, K step kk, of an operand at `base`
  auto frag = [&](auto kcc, auto rbc, uint32_t base, int x0, int kk) -> bf16x8 {
    constexpr bool KC = decltype(kcc)::value;
    constexpr int RB = decltype(rbc)::value;
    const uint32_t o0 = base + pp_frag_off<C, KC, RB>(x0, kk * C::KT, lane, 0);
    if constexpr (pp_e8<C>) {
      i32x2 v;
      if constexpr (KC)
        v = *(__attribute__((address_space(3))) i32x2*)(uintptr_t)o0;
      else
        v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(uintptr_t)o0);
      return pp_widen8(v);
    } else if constexpr (KC) {
      return *(__attribute__((address_space(3))) bf16x8*)(uintptr_t)o0;
    } else {
      return pp_read_tr<C>(o0, base + pp_frag_off<C, KC, RB>(x0, kk * C::KT, lane, 1));
    }
  };

  const int nk = (a.K + C::BK - 1) / C::BK;
  const int mine = wave < nk ? (nk - wave + WAVES - 1) / WAVES : 0;
  static_for<P::S>([&](auto uc) { copy_tile(decltype(uc)::value, decltype(uc)::value); });
  for (int it0 = 0; it0 < mine; it0 += P::S) {
    static_for<P::S>([&](auto uc) {
      constexpr int u = decltype(uc)::value;
      if (it0 + u < mine) {
        // this tile's copies have landed (those of the next S - 1 may still be on their way)
        asm volatile("s_waitcnt vmcnt(%0)" : : "n"((P::S - 1) * P::CP) : "memory");
        const uint32_t base = ring + (uint32_t)(u * P::SLOT);
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS; ++kk) {
          bf16x8 fa[C::FM], fb[C::FN];
#pragma unroll
          for (int i = 0; i < C::FM; ++i)
            fa[i] = frag(std::true_type{}, std::integral_constant<int, C::A_RB>{}, base, i * 16, kk);
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
            fb[j] = frag(std::bool_constant<C::B_KC>{}, std::integral_constant<int, C::SUB_RB>{},
                         base + C::A_BYTES + j / FSUB * C::SUB_BYTES, j % FSUB * 16, kk);
#pragma unroll
          for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) mma_of<C>(acc[i][j], fb[j], fa[i]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot has been read
        copy_tile(it0 + u + P::S, u);
      }
    });
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (the copies past K)
  __syncthreads();

  // ---- the waves' sums meet in LDS: a lane holds rows 16 i + lane % 16, columns 16 j +
  // 4 (lane / 16) .. + 3
  using Sum = std::conditional_t<C::I8, int, float>;
  Sum* sums = (Sum*)lds;
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
      *(f32x4*)(sums + (wave * C::BM + i * 16 + lane % 16) * P::LDR + j * 16 + (lane / 16) * 4) = acc[i][j];
  __syncthreads();
  for (int x = t; x < C::BM * C::BN; x += P::THREADS) {
    const int at = x / C::BN * P::LDR + x % C::BN;
    Sum v = sums[at];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += sums[w * C::BM * P::LDR + at];
    sums[at] = v;
  }
  __syncthreads();
#ifdef DBGEMM_GATED
  float cs[8] = {}, cs2[8] = {};
  if (nv) {
    float w[8], w2[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Sum* p = sums + om * P::LDR + (t % LPR) * 8 + i;
      w[i] = C::I8 ? (float)*p : a.alpha * (float)*p;
      if constexpr (C::DUAL) w2[i] = C::I8 ? (float)p[C::SUB_BN] : a.alpha * (float)p[C::SUB_BN];
    }
    ep_with_act(a.ep.act, [&](auto ac) EP_INLINE {
      gt_finish8<false, C::I8, OP, decltype(ac)::value>(a, w, w2, raw, cols, om, on, cs, cs2);
    });
  }
  if constexpr (OP == GT_GRAD) {  // every row is here: the column sums themselves
    constexpr int OW = (OUT + 63) / 64;  // waves that hold rows
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float* const out = k ? a.ep.sum2 : a.ep.sum1;
      if (!out) continue;
      float(&v)[8] = k ? cs2 : cs;
#pragma unroll
      for (int o = LPR; o < 64; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += __shfl_xor(v[i], o);
      __syncthreads();
      if (wave < OW && lane < LPR)
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[wave * C::BN + lane * 8 + i] = v[i];
      __syncthreads();
      if (t < C::BN && n0 + t < a.N) {
        float sum = sums[t];
#pragma unroll
        for (int w = 1; w < OW; ++w) sum += sums[w * C::BN + t];
        out[n0 + t] = sum;
      }
    }
  }
#else
  float cs[8] = {};
  if (t < OUT) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = a.alpha * sums[om * P::LDR + (t % LPR) * 8 + i];
    ep_dispatch(a.ep, [&](auto mc, auto ac) EP_INLINE {
      ep_finish8<false, decltype(mc)::value, decltype(ac)::value, false>(a, w, raw, bias, om, on, nv, cs);
    });
  }
  if (a.ep.grad && a.ep.colsum) {  // every row is here: the column sums themselves
    constexpr int OW = (OUT + 63) / 64;  // waves that hold rows
#pragma unroll
    for (int o = LPR; o < 64; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] += __shfl_xor(cs[i], o);
    __syncthreads();
    if (wave < OW && lane < LPR)
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[wave * C::BN + lane * 8 + i] = cs[i];
    __syncthreads();
    if (t < C::BN && n0 + t < a.N) {
      float v = sums[t];
#pragma unroll
      for (int w = 1; w < OW; ++w) v += sums[w * C::BN + t];
      a.ep.colsum[n0 + t] = v;
    }
  }
#endif
}

#ifdef DBGEMM_GATED

// The least columns of each B to a workgroup are the best where there are few workgroups or B is
// [N][K]; rows of B [K][N] are asked for in pieces of that many columns, and a line costs the same
// whatever is taken of it.
constexpr int kFewCols[] = {16, 32, 64};
constexpr int few_bm(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }
// The epilogue's one step; and for 64 rows of two B the least columns only, but for E4M3 B [N][K] (widens):
// of 200000 drawn products of 33 to 64 rows none was given more, since where more would be the better width
// the tiles take less time still.
constexpr bool few_fits(int bm, int sub, int nb, bool widens) {
  return bm * sub / 8 <= 256 && (bm < 64 || nb == 1 || sub == kFewCols[0] || widens);
}

// BM rows, SUB columns of each B, K tiles of 128 bytes of A, four waves of two slots each (three
// slots, or eight waves, measured alike or slower by up to 30 %)
template <int BM, int SUB, int IN, bool KC, int OP>
hipError_t launch(const GatedArgs& a, hipStream_t s) {
  constexpr bool DUAL = OP == GT_GATED;
  if constexpr (few_fits(BM, SUB, DUAL ? 2 : 1, IN == IN_E4M3_LDS && KC)) {
    using C = Cfg<BM, DUAL ? 2 * SUB : SUB, IN == IN_BF16 ? 64 : 128, 1, 1, 16, 2, IN, false, KC, 1, DUAL>;
    hipLaunchKernelGGL((gemm_skinny_kernel<C, 4, OP>), dim3((unsigned)((a.N + SUB - 1) / SUB)), dim3(256), 0, s, a);
    return hipGetLastError();
  } else {
    return hipErrorInvalidConfiguration;
  }
}

template <int SUB, int IN, bool KC, int OP>
hipError_t launch_bm(const GatedArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch<16, SUB, IN, KC, OP>(a, s);
  if (a.M <= 32) return launch<32, SUB, IN, KC, OP>(a, s);
  return launch<64, SUB, IN, KC, OP>(a, s);
}

template <int IN, bool KC, int OP>
hipError_t launch_rows(const GatedArgs& a, int cols, hipStream_t s) {
  if (cols == 16) return launch_bm<16, IN, KC, OP>(a, s);
  if (cols == 32) return launch_bm<32, IN, KC, OP>(a, s);
  return launch_bm<64, IN, KC, OP>(a, s);
}

template <int IN, bool KC>
hipError_t launch_op(const GatedArgs& a, int cols, hipStream_t s) {
  if (a.op == GT_GATED) return launch_rows<IN, KC, GT_GATED>(a, cols, s);
  return launch_rows<IN, KC, IN == IN_I8 ? GT_LINEAR : GT_GRAD>(a, cols, s);
}

#else

// BM rows, BN columns, K tiles of 128 bytes of A, S slots to a wave
template <int BM, int BN, int S, int WAVES, bool E8, bool KC>
hipError_t launch(const GemmEpArgs& a, hipStream_t s) {
  using C = Cfg<BM, BN, E8 ? 128 : 64, 1, 1, 16, S, E8 ? IN_E4M3_LDS : IN_BF16, false, KC>;
  hipLaunchKernelGGL((gemm_skinny_kernel<C, WAVES>), dim3((unsigned)((a.N + BN - 1) / BN)), dim3(WAVES * 64), 0, s, a);
  return hipGetLastError();
}

// Four waves with three slots each (72 KiB of LDS: two workgroups to a CU), against eight with
// two or three and four with six, measured alike within 5% (1 x 4096 x 4096, B [N][K]: 7.7 us;
// 13 x 5120 x 5120: 10.6, 4.9 TB/s); 64 columns to a workgroup 13.6.
template <bool E8, bool KC>
hipError_t launch_rows(const GemmEpArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch<16, 32, 3, 4, E8, KC>(a, s);
  if (a.M <= 32) return launch<32, 32, 3, 4, E8, KC>(a, s);
  return launch<64, 32, 2, 4, E8, KC>(a, s);
}

#endif

}  // namespace

#ifdef DBGEMM_GATED

// A workgroup's wave takes every fourth of the K tiles (128 bytes of K).  A K tile costs a wave what
// its lines (128 bytes, or the piece of one that a row of B [K][N] has in these columns) and its
// bytes take to be asked for; and all workgroups together need the CU's share of the memory's rate
// and of its line requests, whole workgroups to a CU (1 x 10944 x 4096, both B [N][K]: 39.3 us at 32
// columns, 342 workgroups, and 34.4 at 16, 684 of them).  Past what the CUs hold at once every further
// round starts and ends on its own (55 x 17840 x 272 of 8-bit integers, one workgroup of 64 rows to a CU,
// 16.7 us in five rounds; 8.3 on the tiles), and under half the CUs do not draw the memory's rate
// (13 x 8864 x 9056, both B [K][N], 8-bit: 57 us at 64 columns, 139 workgroups; 15 x 7760 x 8608 58, 122 of
// them, and 47 at 32 columns).  Fitted to 10500 products of 1 to 64 rows, N and K from 256 to 20480, in all
// kinds, layouts and the three widths, on 256 CUs: 14 % off in the mean square, its width 1.0 % behind the
// best of them in the mean.  Near ties it misses: 1 x 10944 x 4096 is given 64 columns, 35.6 us by the model
// and 36.3 at 16, and measures 37.4 there with its weights out of the caches.
double few_rows_us(int op, int in_kind, int transB, int64_t M, int64_t N, int64_t K, int cu_count, int* cols) {
  if (cu_count <= 0) cu_count = 256;
  const int bm = few_bm(M), nb = op == GT_GATED ? 2 : 1, es = in_kind == GT_BF16 ? 2 : 1;
  const double its = (double)((K * es + 127) / 128) / 4.0;
  double best = 0.0;
  *cols = 0;
  for (int sub : kFewCols) {
    if (!few_fits(bm, sub, nb, in_kind == GT_E4M3 && transB)) continue;
    const int64_t wgs = (N + sub - 1) / sub;
    const double whole = 0.85 * (double)((wgs + cu_count - 1) / cu_count), share = (double)wgs / cu_count;
    const double groups = wgs >= cu_count && whole > share ? whole : share;
    const double lines = nb * (transB ? sub : 128 / es) + bm, kb = nb * sub / 8.0;
    double wave = 0.00443 * lines + 0.0240 * kb;
    if (in_kind == GT_E4M3 && transB) wave *= 1.39;  // (the widening, where the lines do not hide it)
    const double all = 4.0 * (0.00114 * lines + 0.0349 * kb) * groups;
    const int held = 160 / (bm + nb * sub);  // workgroups that the LDS of a CU holds, 1 KiB to a row of A or B
    const int64_t at_once = (int64_t)cu_count * (held < 1 ? 1 : held > 8 ? 8 : held);
    const double more = (double)((wgs + at_once - 1) / at_once - 1), results = bm * sub * nb / 1024.0;
    double us = 2.75 + 0.696 * results + more * (0.874 + 0.689 * results) +
                its * std::sqrt(std::sqrt(wave * wave * wave * wave + all * all * all * all));
    if (sub == 64 && 2 * wgs < cu_count) us *= 1.2;
    if (*cols == 0 || us < best) {
      best = us;
      *cols = sub;
    }
  }
  return best;
}

hipError_t launch_gated_skinny(const GatedArgs& a, int cols, hipStream_t s) {
  if (a.M < 1 || a.M > 64 || a.N % 8 != 0) return hipErrorInvalidConfiguration;
  switch (a.in_kind * 2 + (a.transB != 0)) {
    case GT_BF16 * 2: return launch_op<IN_BF16, false>(a, cols, s);
    case GT_BF16 * 2 + 1: return launch_op<IN_BF16, true>(a, cols, s);
    case GT_E4M3 * 2: return launch_op<IN_E4M3_LDS, false>(a, cols, s);
    case GT_E4M3 * 2 + 1: return launch_op<IN_E4M3_LDS, true>(a, cols, s);
    case GT_I8 * 2: return launch_op<IN_I8, false>(a, cols, s);
    default: return launch_op<IN_I8, true>(a, cols, s);
  }
}

#else

// Where this kernel is the faster one: up to some K, past which a workgroup's waves walk too
// long and the tiled kernels' split of K wins.  Measured both ways on 24557 products of 1 to 64
// rows, N and K from 256 to 20480; time of the tiled kernels over this one's, N under / from 1500:
//
//                      K < 1024      1024-2048     2048-4096     4096-8192     8192 on
//   bf16 [N][K] M<=16  1.51 / 1.38   2.00 / 1.64   1.83 / 1.54   1.52 / 1.38   0.94 / 1.13
//               M<=32  1.52 / 1.28   1.81 / 1.37   1.55 / 1.29   1.20 / 1.11   0.68 / 0.89
//               M<=64  1.29 / 1.07   1.42 / 1.12   1.13 / 1.09   0.83 / 0.92   0.48 / 0.72
//   bf16 [K][N] M<=16  1.44 / 1.24   1.83 / 1.34   1.45 / 1.12   1.03 / 0.99   0.63 / 0.84
//               M<=32  1.38 / 1.05   1.60 / 1.18   1.18 / 1.04   0.77 / 0.88   0.50 / 0.74
//               M<=64  1.24 / 0.95   1.32 / 0.96   0.98 / 0.86   0.64 / 0.75   0.39 / 0.63
//   E4M3 [N][K] M<=16  1.42 / 1.38   1.80 / 1.71   1.74 / 1.74   1.50 / 1.69   1.09 / 1.47
//               M<=32  1.39 / 1.21   1.62 / 1.43   1.51 / 1.44   1.24 / 1.35   0.87 / 1.14
//               M<=64  1.20 / 0.99   1.28 / 1.11   1.09 / 1.05   0.82 / 0.98   0.54 / 0.84
//   E4M3 [K][N] M<=16  1.57 / 1.39   1.87 / 1.52   1.62 / 1.38   1.12 / 1.21   0.73 / 0.99
//               M<=32  1.47 / 1.15   1.66 / 1.29   1.38 / 1.16   0.99 / 1.05   0.64 / 0.88
//               M<=64  1.27 / 1.02   1.32 / 1.07   1.03 / 0.93   0.72 / 0.84   0.49 / 0.71
//
// (In B [K][N] an XCD finds its columns on some of its L2's channels only.)  With these limits the
// choice is 1.7 % slower than the better of the two in the mean.
bool skinny_serves(int in_fp8, int transA, int transB, int64_t M, int64_t K) {
  constexpr int64_t most[2][2][3] = {{{6144, 3072, 2048}, {12288, 8192, 4096}},   // bf16: B [K][N], [N][K]
                                     {{8192, 6144, 2560}, {20480, 12288, 5120}}};  // E4M3
  return !transA && M <= 64 && K <= most[in_fp8 != 0][transB != 0][M <= 16 ? 0 : M <= 32 ? 1 : 2];
}

hipError_t launch_skinny(const GemmEpArgs& a, hipStream_t s) {
  if (a.M < 1 || a.M > 64 || a.transA || a.N % 8 != 0) return hipErrorInvalidConfiguration;
  if (a.in_fp8) return a.transB ? launch_rows<true, true>(a, s) : launch_rows<true, false>(a, s);
  return a.transB ? launch_rows<false, true>(a, s) : launch_rows<false, false>(a, s);
}

#endif

}  // namespace dbgemm
