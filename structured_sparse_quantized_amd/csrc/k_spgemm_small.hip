// Small tiles of the product with the general epilogue (gfx950 v_smfmac), for problems whose 256 x 128 tiles leave
// most of the chip idle. Deep reading of arXiv 2610.28947 (introduction; section 3.1: sparse W or sparse X).
//
// C[r][c] = sum_k A[r][k] B[c][k], A = the tiled compressed operand, B = the dense one, as in k_spgemm_tiled.hip,
// whose layout it reads and whose sums it repeats bit for bit (one accumulator per result, the steps in order).
//
// A workgroup of 4 waves (2 x 2) takes 64 A rows x 32 TJ B rows; a wave 32 x 16 TJ, 2 x TJ instructions a step. What
// bounds such a problem is the length of the reduction at one tile per CU, so the loads run far ahead: a ring of
// S stages of one 128-position step each (4 KB of compressed values, their index words, the B rows), every
// wave bringing the same number of pieces per stage by LDS DMA, so that "the next stage has landed" is a wait for a
// constant count. The fragments of step j + 1 are read while step j multiplies, before its loads set out (after them: 5% slower);
// one barrier a step. A step costs 0.14, 0.18 and 0.24 us at TJ = 1, 2 and 4: at TJ = 1 a CU takes in its 9 KB at 65 B/ns, at
// TJ = 2 and 4 at 74 and 90, so the L2s could give more: with 5 stages (46 KB) on their way it is the latency of 0.7 us that
// counts. A barrier per two steps measured the same at TJ = 1 and lost at TJ = 2 and 4, whose
// LDS holds too few stages for it. FP8, 4096 rows, 128 tokens: 8.6 us at K = 4096, 20.2 us at 14336, where the 256 x 128
// tiles take 20.8 and 51.8.
#include <type_traits>

#include "ss_device.h"
#include "ss_kernels.h"
#include "ss_mma.h"
#include "ss_store.h"

namespace ss {
namespace small {

using tiled::Meta;
using tiled::Mma;
using tiled::swz;
using tiled::v4i;
#define SS_LDS __attribute__((address_space(3)))

constexpr int NW = 4, BM = 64, S = 6;
constexpr int vm(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8); }  // s_waitcnt vmcnt(n)

template <int TJ> struct Shape {
  static constexpr int BN = 32 * TJ;
  static constexpr int A_BYTES = BM * 64, M_BYTES = BM / 16 * 256, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + M_BYTES + B_BYTES;
  static constexpr int LPW = 2 + TJ;  // loads per wave and stage: an A row block, its index words, TJ x 8 B rows
  static constexpr int LDS = S * STAGE;
};

template <int AB, bool SX, int TJ>
__global__ __launch_bounds__(64 * NW, 2) void small_kernel(int R, int C, int KS, const uint8_t* __restrict__ tv,
                                                            const uint8_t* __restrict__ tm, const uint8_t* __restrict__ bd,
                                                            int ldb, const float* __restrict__ sx,
                                                            const float* __restrict__ sw, void* __restrict__ Y, int ldy,
                                                            int tiles_r, Epilogue ep) {
  using SH = Shape<TJ>;
  using Acc = typename Mma<AB>::Acc;
  using MT = Meta<AB>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, r16 = lane & 15, jj = lane >> 4;
  const int tr = blockIdx.x % tiles_r, tc = blockIdx.x / tiles_r;
  const int r0 = tr * BM, c0 = tc * SH::BN;
  const int nrb = (R + 15) / 16, KS4 = (KS + 3) / 4, KSP = 4 * KS4;

  // Per-lane sources; rows past the end are clamped to the last row (block), their results are never stored.
  const int rb = min(r0 / 16 + wave, nrb - 1);
  const uint8_t* pa = tv + (int64_t)rb * KSP * 1024 + lane * 16;
  const uint8_t* pm = tm + (int64_t)rb * KS4 * MT::BLOCK + lane * (4 * MT::WB);
  const uint8_t* pb[TJ];
#pragma unroll
  for (int q = 0; q < TJ; ++q) {
    const int b = (wave + q * NW) * 8 + (lane >> 3);
    pb[q] = bd + (int64_t)min(c0 + b, C - 1) * (uint32_t)ldb + swz(lane & 7, b & 15) * 16;
  }
  // stage k into its slot; steps past the end re-read the last one (in bounds, never used), so that every wave's
  // count of loads stays the same
  auto issue = [&](int k) __attribute__((always_inline)) {
    SS_LDS uint8_t* base = (SS_LDS uint8_t*)smem + (k % S) * SH::STAGE;
    const int kk = min(k, KS - 1);
    __builtin_amdgcn_global_load_lds((const void*)(pa + (int64_t)kk * 1024), (SS_LDS void*)(base + wave * 1024), 16, 0, 0);
    // the 32-bit word with this step's index (bf16: two steps' halves)
    __builtin_amdgcn_global_load_lds((const void*)(pm + (int64_t)(kk >> 2) * MT::BLOCK + 4 * (AB == 2 ? (kk & 3) >> 1 : kk & 3)),
                                     (SS_LDS void*)(base + SH::A_BYTES + wave * 256), 4, 0, 0);
#pragma unroll
    for (int q = 0; q < TJ; ++q)
      __builtin_amdgcn_global_load_lds((const void*)(pb[q] + (int64_t)kk * 128),
                                       (SS_LDS void*)(base + SH::A_BYTES + SH::M_BYTES + (wave + q * NW) * 1024), 16, 0, 0);
  };

  Acc acc[2][TJ];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int u = 0; u < TJ; ++u) acc[t][u] = Acc{0, 0, 0, 0};
  struct Frag {
    v4i a[2], b[TJ][2];
    int m[2];
  };
  auto read = [&](Frag& f, int k) __attribute__((always_inline)) {
    const uint8_t* st = smem + (k % S) * SH::STAGE;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f.a[t] = *reinterpret_cast<const v4i*>(st + (wm * 2 + t) * 1024 + lane * 16);
      f.m[t] = *reinterpret_cast<const int*>(st + SH::A_BYTES + (wm * 2 + t) * 256 + lane * 4);
    }
#pragma unroll
    for (int u = 0; u < TJ; ++u) {
      const uint8_t* bb = st + SH::A_BYTES + SH::M_BYTES + ((wn * TJ + u) * 2 + (r16 >> 3)) * 1024 + (r16 & 7) * 128;
      f.b[u][0] = *reinterpret_cast<const v4i*>(bb + swz(jj, r16) * 16);
      f.b[u][1] = *reinterpret_cast<const v4i*>(bb + swz(4 + jj, r16) * 16);
    }
  };
  // step j, its fragments in `cur`: stage j + 1 landed for every wave, stage j + S - 1 set out (its slot held stage
  // j - 1, read before the barrier of step j - 1), fragments of j + 1 read, step j multiplied
  auto step = [&](int j, Frag& cur, Frag& nxt, auto half) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(vm((S - 3) * SH::LPW));
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's own reads
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(nxt, j + 1);
    __builtin_amdgcn_sched_barrier(0);
    issue(j + S - 1);
#pragma unroll
    for (int u = 0; u < TJ; ++u)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        acc[t][u] = Mma<AB>::template run<AB == 2 ? decltype(half)::value : 0>(cur.a[t], cur.b[u][0], cur.b[u][1], acc[t][u],
                                                                               cur.m[t]);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int k = 0; k < S - 1; ++k) issue(k);
  __builtin_amdgcn_s_waitcnt(vm((S - 2) * SH::LPW));  // stage 0
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  Frag f0, f1;
  read(f0, 0);
  for (int j = 0; j < KS; j += 2) {  // (KS is even: the operands' alignment)
    step(j, f0, f1, std::integral_constant<int, 0>{});
    step(j + 1, f1, f0, std::integral_constant<int, 1>{});
  }
  __builtin_amdgcn_s_waitcnt(vm(0));  // no load may outlive the workgroup
  __syncthreads();                    // the ring is idle

  // Epilogue: float32 rows of 32 (side X: tokens of A; side W: tokens of B) through the ring, as in the larger kernels.
  const float* sa = SX ? sx : sw;
  const float* sb = SX ? sw : sx;
  constexpr int CH = SX ? 16 * TJ : 32, ROWS = SX ? 32 : 16 * TJ, LD = CH + 4;  // staged channels, tokens of a wave
  float* stg = reinterpret_cast<float*>(smem) + wave * ROWS * LD;
  static_assert(NW * ROWS * LD * 4 <= SH::LDS, "staging fits the ring");
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float s_a[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) s_a[q] = sa ? sa[min(r0 + (wm * 2 + t) * 16 + 4 * jj + q, R - 1)] : 1.0f;
#pragma unroll
    for (int u = 0; u < TJ; ++u) {
      const float s_b = sb ? sb[min(c0 + (wn * TJ + u) * 16 + r16, C - 1)] : 1.0f;
      float y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)  // the token scale first, then the channel scale
        y[q] = __fmul_rn(__fmul_rn((float)acc[t][u][q], SX ? s_a[q] : s_b), SX ? s_b : s_a[q]);
      if constexpr (SX) {
#pragma unroll
        for (int q = 0; q < 4; ++q) stg[(t * 16 + 4 * jj + q) * LD + u * 16 + r16] = y[q];
      } else {
        *reinterpret_cast<float4*>(stg + (u * 16 + r16) * LD + t * 16 + 4 * jj) = make_float4(y[0], y[1], y[2], y[3]);
      }
    }
  }
  __builtin_amdgcn_wave_barrier();
  const int tok0 = SX ? r0 + wm * 32 : c0 + wn * 16 * TJ, ntok = SX ? R : C;
  const int ch0 = SX ? c0 + wn * 16 * TJ : r0 + wm * 32, nch = SX ? C : R;
  if (tok0 >= ntok) return;
  if (!aligned_rows(ep, ldy)) {
    leave_columns<CH>(stg, LD, ROWS, tok0, ntok, ch0, nch, Y, ldy, ep);
    return;
  }
  const int cpr = (CH / 8) >> ep.gated, rps = 64 / cpr, row0 = lane / cpr;
  const Leave out(ep, Y, ldy, lane % cpr, ch0, nch);
  if (row0 >= ROWS) return;
#pragma unroll 1
  for (int r = row0; r < ROWS; r += rps) {
    if (tok0 + r >= ntok) break;
    Leave::Res res;
    out.residual(res, tok0 + r);
    out.row(stg + r * LD, res, tok0 + r);
  }
}

template <int AB, bool SX, int TJ>
hipError_t launch(int R, int C, int KS, const uint8_t* tv, const uint8_t* tm, const uint8_t* bd, int ldb, const float* sx,
                  const float* sw, void* Y, int ldy, const Epilogue& ep, hipStream_t st) {
  auto kern = small_kernel<AB, SX, TJ>;
  constexpr int lds = Shape<TJ>::LDS;
  const hipError_t e = lds_limit((const void*)kern, lds);
  if (e != hipSuccess) return e;
  const int tr = (R + BM - 1) / BM, tc = (C + Shape<TJ>::BN - 1) / Shape<TJ>::BN;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tr * tc)), dim3(64 * NW), lds, st, R, C, KS, tv, tm, bd, ldb, sx, sw, Y, ldy, tr, ep);
  return hipGetLastError();
}

}  // namespace small

hipError_t launch_spgemm_small(int tj, bool side_x, int ab, int R, int C, int KS, const uint8_t* tv, const uint8_t* tm,
                               const uint8_t* bd, int ldb, const float* sx, const float* sw, void* Y, int ldy,
                               const Epilogue& ep, hipStream_t st) {
#define SS_SMALL(AB_, SX_)                                                                              \
  return tj == 1   ? small::launch<AB_, SX_, 1>(R, C, KS, tv, tm, bd, ldb, sx, sw, Y, ldy, ep, st)      \
         : tj == 2 ? small::launch<AB_, SX_, 2>(R, C, KS, tv, tm, bd, ldb, sx, sw, Y, ldy, ep, st)      \
                   : small::launch<AB_, SX_, 4>(R, C, KS, tv, tm, bd, ldb, sx, sw, Y, ldy, ep, st)
  if (side_x) {
    if (ab == 0) SS_SMALL(0, true);
    if (ab == 1) SS_SMALL(1, true);
    SS_SMALL(2, true);
  }
  if (ab == 0) SS_SMALL(0, false);
  if (ab == 1) SS_SMALL(1, false);
  SS_SMALL(2, false);
#undef SS_SMALL
}

}  // namespace ss
