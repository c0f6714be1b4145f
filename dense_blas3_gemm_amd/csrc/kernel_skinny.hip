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
#include "epilogue.h"
#include "mfma_common.h"

namespace dbgemm {
namespace {

template <class C, int WAVES_>
struct Skinny {
  static constexpr int WAVES = WAVES_, THREADS = WAVES * 64, S = C::STAGES;
  static_assert(C::WM == 1 && C::WN == 1 && C::MT == 16 && (C::IN == IN_BF16 || C::IN == IN_E4M3_LDS), "a wave's tile");
  static constexpr int SLOT = C::A_BYTES + C::B_BYTES;
  static_assert(C::A_BYTES % 1024 == 0 && C::B_BYTES % 1024 == 0, "whole 1 KiB copies");
  static constexpr int A_CP = C::A_BYTES / 1024, B_CP = C::B_BYTES / 1024, CP = A_CP + B_CP;
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

template <class C, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void gemm_skinny_kernel(GemmEpArgs a) {
  using P = Skinny<C, WAVES>;
  __shared__ __attribute__((aligned(1024))) char lds[P::LDS_BYTES];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  // (B [N][K]: a run of columns to each XCD)
  const int tn = C::B_KC ? xcd_remap(blockIdx.x, gridDim.x, 8)
                         : line_remap<(128 > C::BN * C::ES ? 128 / (C::BN * C::ES) : 1)>(blockIdx.x, gridDim.x);
  const int n0 = tn * C::BN;

  // ---- the epilogue's operands: thread t < OUT takes eight columns of a row at the end
  constexpr int LPR = C::BN / 8, OUT = C::BM * LPR;
  static_assert(LPR % 4 == 0 && OUT <= P::THREADS, "whole blocks of 32 columns, one step");
  const int om = t / LPR, on = n0 + (t % LPR) * 8;
  const int nv = t < OUT && om < a.M && on < a.N ? 8 : 0;
  float bias[8];
  ep_bias8(a, on, nv, bias);
  const EpRaw raw = !a.ep.grad                ? ep_fetch8<EP_FORWARD, false>(a, om, on, nv)
                    : a.ep.z_kind == Z_MX ? ep_fetch8<EP_GRAD_MX, false>(a, om, on, nv)
                                          : ep_fetch8<EP_GRAD_BF16, false>(a, om, on, nv);

  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, (uint32_t)(a.M * a.lda * C::ES));
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(a.B, (uint32_t)((C::B_KC ? (int64_t)a.N : (int64_t)a.K) * a.ldb * C::ES));
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds0 + (uint32_t)(wave * P::S * P::SLOT));

  // ---- this lane's chunks: copy i of an operand fills LDS chunks 64 i .. + 63 of its tile, chunk
  // p = 64 i + lane being row p / CPR, physical chunk p % CPR, which holds logical chunk
  // (p % CPR) ^ swizzle(row).  Byte offset of it in K tile 0 (past every buffer for a row past
  // M or a column past N), and its K index within a tile.
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
    const int p = i * 64 + lane, r = p / C::B_CPR, c = (p % C::B_CPR) ^ pp_swz<C, C::B_KC, C::B_CPR>(r);
    if constexpr (C::B_KC) {
      b_off[i] = n0 + r < a.N ? (uint32_t)(((n0 + r) * a.ldb + c * C::VEC) * C::ES) : kOOB;
      b_k[i] = c * C::VEC;
    } else {
      b_off[i] = n0 + c * C::VEC < a.N ? (uint32_t)((r * a.ldb + n0 + c * C::VEC) * C::ES) : kOOB;
      b_k[i] = r;
    }
  }
  const uint32_t b_step = C::B_KC ? C::BK * C::ES : (uint32_t)(C::BK * a.ldb * C::ES);
  // copies of this wave's tile number it (K tile wave + it * WAVES) into slot u; what lies past K
  // reads zeros and touches no memory
  auto copy_tile = [&](int it, int u) {
    const int kt = wave + it * WAVES, left = a.K - kt * C::BK;
    const uint32_t ao = (uint32_t)(kt * C::BK * C::ES), bo = (uint32_t)kt * b_step;
    const uint32_t l = __builtin_amdgcn_readfirstlane(ring + (uint32_t)(u * P::SLOT));
    skinny_copies<P::B_CP, 0>(
        l + C::A_BYTES, [&](int i) { return b_k[i] < left && b_off[i] != kOOB ? b_off[i] + bo : kOOB; }, rb);
    skinny_copies<P::A_CP, 0>(l, [&](int i) { return a_k[i] < left && a_off[i] != kOOB ? a_off[i] + ao : kOOB; }, ra);
  };

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
      const uint32_t o1 = base + pp_frag_off<C, KC, RB>(x0, kk * C::KT, lane, 1);
      const u16x4 lo = __builtin_bit_cast(u16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                     (__attribute__((address_space(3))) s16x4*)(uintptr_t)o0));
      const u16x4 hi = __builtin_bit_cast(u16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                     (__attribute__((address_space(3))) s16x4*)(uintptr_t)o1));
      return __builtin_bit_cast(bf16x8, (ep_u16x8){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
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
            fb[j] = frag(std::bool_constant<C::B_KC>{}, std::integral_constant<int, C::B_RB>{}, base + C::A_BYTES,
                         j * 16, kk);
#pragma unroll
          for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) mma(acc[i][j], fb[j], fa[i]);
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
  float* sums = (float*)lds;
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
      *(f32x4*)(sums + (wave * C::BM + i * 16 + lane % 16) * P::LDR + j * 16 + (lane / 16) * 4) = acc[i][j];
  __syncthreads();
  for (int x = t; x < C::BM * C::BN; x += P::THREADS) {
    const int at = x / C::BN * P::LDR + x % C::BN;
    float v = sums[at];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += sums[w * C::BM * P::LDR + at];
    sums[at] = v;
  }
  __syncthreads();
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
}

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

}  // namespace

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

}  // namespace dbgemm
