// Attention over packed sequences (gfx950): o = softmax(scale q k^T + mask) v, grouped heads, causal or not.
//
// Mathematics. One pass over the keys with a running maximum and sum: for a query row, after keys 0..j,
//   m = max_i s_i, l = sum_i 2^(c s_i - m), O = sum_i 2^(c s_i - m) v_i  (s = q.k, c = scale * log2 e),
// and o = O / l. A new maximum m' multiplies l and O by 2^(m - m'). m only has to keep the powers in range,
// so it is raised only when a row's maximum passes it by more than kSlack, or (tiles of many rows) when 16 of its
// powers sum to more than kRise: the powers then stay below 2^8, their relative precision is the same, and O is left
// untouched on almost every tile. Scores, m, l and O are
// float32; the powers are rounded to bf16 (nearest even) for the second product, because the matrix
// instructions take bf16 there: with q, k, v in bf16 that adds one rounding of at most 2^-8 relative per
// key, independent over the keys (in all 0.0022 of a row against 0.0016 with float32 probabilities; what the rounding leaves as
// a second operand costs few_kernel 0-3% over long caches and up to 20% for chunks of tokens). l sums the powers before it.
//
// Rows. The query heads that share a key head read the same keys, so the rows of one (sequence, key head) are
// all its (token, head) pairs, r = token * G + head-in-group: a tile of rows covers fewer tokens than rows,
// which also wastes less at the causal edge.
//
// Matrix instructions (32x32x16 bf16, operands A: row l%32, positions 8(l/32)..+7; result: column l%32, rows
// 8(i/4) + 4(l/32) + i%4). Both products are taken transposed: S^T = K Q^T, so a lane holds 16 of 32 scores
// of one query row (its column) and the row's maximum needs one exchange with lane l^32; and O^T = V^T P^T,
// whose B operand takes the lane's own powers unmoved, because the order of the reduction is free: position
// 8h + j of a 16-key step stands for key 4h + j (j < 4) or 8 + 4h + j - 4 (j >= 4) of the step. V^T
// fragments come out of the row-major V tile in LDS by the transposing LDS read (64 bits per lane: 16 lanes
// read 4 rows of 16 values and each receives one column).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {
namespace attn {

#define SS_LDS __attribute__((address_space(3)))
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr float kSlack = 8.0f;     // in powers of two
constexpr float kRise = 256.0f;
constexpr int vm(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8); }  // s_waitcnt vmcnt(n)
constexpr float kLow = -3.402823466e38f;  // below every finite score's exponent, and finite: kLow - kLow = 0
// From this size of a maximum m on, the power's argument is the rounded product c s less m. Below it both come out of one
// fused step, whose exact product may pass the rounded maximum by half of a unit of m's last place: 2^7 at 2^31, a power that
// overflows (or, below m, a largest score whose power is 0).
constexpr float kBig = 16777216.0f;  // 2^24
__device__ __forceinline__ bool is_big(float m) { return m != kLow && fabsf(m) >= kBig; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
// The transposing LDS read, through a pointer that nothing else writes while it is read (the kernels' barriers and
// waits see to that). Said without it, the compiler lets every such read wait for all loads to LDS in flight,
// which exposed the latency of the next tile's load in every tile.
__device__ __forceinline__ v4s read_tr(const SS_LDS void* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((SS_LDS v4s*)p);
}

__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float unif(float x) { return __int_as_float(uni(__float_as_int(x))); }

// the value of this lane and of lane l ^ 32, combined
__device__ __forceinline__ float pair_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// One sequence's share of the call, all uniform. Bounds taken from device memory are clamped to the tensors,
// so whatever cu_q, cu_k and k_len hold, no access leaves q, k, v or o.
struct Seq {
  int64_t q0, k0;  // first query and key row
  int lq, lk;      // rows
};
__device__ __forceinline__ int64_t inside(int x, int64_t n) { return min(max((int64_t)x, (int64_t)0), n); }
__device__ __forceinline__ int64_t bound(const int32_t* cu, int i, int64_t n) {  // NULL: one sequence of all rows
  return cu ? inside(cu[i], n) : i == 0 ? 0 : n;
}
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  int64_t q0, q1, k0, k1;
  int len = 0x7FFFFFFF;
  if (a.cu_q && a.cu_k) {  // the five loads set out together (a call of few keys is a chain of such latencies)
    const int x0 = a.cu_q[b], x1 = a.cu_q[b + 1], y0 = a.cu_k[b], y1 = a.cu_k[b + 1], n = (a.k_len ? a.k_len : a.cu_q)[b];
    q0 = inside(x0, a.Tq), q1 = inside(x1, a.Tq), k0 = inside(y0, a.Tk), k1 = inside(y1, a.Tk);
    if (a.k_len) len = n;
  } else {
    q0 = bound(a.cu_q, b, a.Tq), q1 = bound(a.cu_q, b + 1, a.Tq), k0 = bound(a.cu_k, b, a.Tk), k1 = bound(a.cu_k, b + 1, a.Tk);
    if (a.k_len) len = a.k_len[b];
  }
  Seq s;
  s.q0 = q0;
  s.k0 = k0;
  s.lq = (int)(max(q1, q0) - q0);
  s.lk = min(max(len, 0), (int)(max(k1, k0) - k0));
  return s;
}

// Row tiles: sequence b's tiles of BM rows start at slot floor(cu_q[b] G / BM) + b. The slots between two
// starts are at least the tiles of the sequence (floor(x + n) - floor(x) + 1 >= ceil(n)), so a grid of
// floor(Tq G / BM) + B slots serves every split of Tq rows into B sequences without the host knowing it; a
// slot past its sequence's rows has nothing to do. Each wave finds its slot's sequence with one load of cu_q per lane
// and a ballot per factor of 64 in B. Returns false where there is no tile.
template <int BM> __device__ __forceinline__ bool find_tile(const AttnArgs& a, int slot, int& b, int& tile) {
  const int lane = threadIdx.x & 63;
  auto start = [&](int i) { return bound(a.cu_q, i, a.Tq) * a.G / BM + i; };
  int lo = 0, n = a.B;
  while (true) {
    const int step = (n + 63) / 64;
    const int i = lane * step;
    const bool in = i < n && start(lo + min(i, n - 1)) <= slot;
    const int cnt = __popcll(__ballot(in));
    if (cnt == 0) return false;
    lo += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
    if (step == 1) break;
  }
  b = uni(lo);
  tile = uni((int)(slot - start(b)));
  return tile >= 0;
}

// The tile and sequence of a slot; false where there is none.
template <int BM> __device__ __forceinline__ bool locate(const AttnArgs& a, int slot, Seq& s, int& tile) {
  if (a.B == 1) {
    s = load_seq(a, 0);
    tile = slot - (int)(s.q0 * a.G / BM);
  } else {
    int b;
    if (!find_tile<BM>(a, slot, b, tile)) return false;
    s = load_seq(a, b);
  }
  return tile >= 0 && tile * BM < s.lq * a.G;
}

// LDS tiles are row-major (DP values a row, in 16-byte chunks) with the chunks of a row permuted by an XOR, so
// that the fragment reads below spread over the banks: a K fragment reads one chunk column of 32 rows, a V
// fragment 4 chunks of 4 rows (rows of 64 values lie two to a turn of the banks, so pairs of rows share a place).
template <int DP> struct Lds {
  __device__ static int swk(int row) { return DP >= 128 ? row & 15 : (row >> 1) & 7; }
  __device__ static int swv(int row) { return DP >= 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2; }
};

// Under a causal mask a tile's keys go past what some of its rows see, or all of them (rows of one token, with 32 query heads
// and more to a key head: a tile is loaded up to the sequence's last key), and one product takes them all: a power of
// zero keeps a finite value of an unseen key out of a row, not an infinity or a NaN. Where a tile's values hold one, it is
// replaced by zero in the operand and added to the rows that see it by hand (its power is above zero, so the sum is v itself).
__device__ __forceinline__ uint32_t odd_bf16x2(uint32_t w) {  // bits 31, 15: that half is infinite or NaN
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t even_out(uint32_t w) {
  asm volatile("" : "+v"(w));  // (computed anew: its parts are not kept from the test)
  return w & ~((odd_bf16x2(w) >> 15) * 0xFFFFu);
}
// `vt`: 32 rows of values in LDS, of which row r of the lane sees the first `seen`
template <int DP> __device__ __forceinline__ void add_odd(v16f* O, const SS_LDS uint8_t* vt, int seen, int h) {
  asm volatile("" : "+v"(h), "+v"(seen));  // (nothing of this is kept in registers beside the loop that calls it)
#pragma unroll 1
  for (int k = 0; k < 32; ++k)
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const v2u w = *reinterpret_cast<const SS_LDS v2u*>(vt + k * DP * 2 + ((d * 4 + g) ^ Lds<DP>::swv(k)) * 16 + h * 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
          if (k < seen && !__builtin_isfinite(v)) O[d][4 * g + e] += v;
        }
      }
}

// What is computed from x is computed anew from here on (in the loops that have no registers to keep it in).
__device__ __forceinline__ void renew(uint32_t& x) { asm volatile("" : "+v"(x)); }

// ---- many rows: tiles of 4 waves x 32 rows, two workgroups per CU ----------------------------------------------
// The work of a wave is pipelined over stages of 32 keys (two to a tile of BK). Stage j, in program order:
//   the scores of stage j + 1, O += V P of stage j - 1, and between them the powers of stage j, step by step; a
//   fragment that has been used is read anew from LDS for the next stage at once;
//   where a lane's 16 powers sum to more than kRise (or overflow): the row's maximum found, l and O rescaled, the powers
//   taken again. Looking at the sum that is there anyway, after the fact, keeps 8 instructions and a branch
//   that waits for them out of every stage (1-3% for heads of 128, 6% for 64); the first stage's maximum is found ahead.
// So the matrix instructions have vector work of about the same length beside them that does not wait for
// them, and fragments are read a stage ahead of their use.
// Measured: one prompt of 8192 tokens, 32 heads of 128 over 8, causal: 470-507 us by the card, 1.09-1.17 PFLOP/s of the seen
// pairs (matrix cores busy 65% of the cycles, at the 1.8 GHz a card keeps under this load; its large bf16 product runs at
// 1.37); 9 packed prompts, 8001 tokens, 28 heads over 4: 84-88 us, 0.68-0.71 PFLOP/s. What bounds it is the vector work beside the matrix
// instructions, some 60 instructions per 16 scores a lane (the 16 powers at a quarter of the rate), about as long as
// the products themselves. Tried and not kept: 64 rows a wave (608 us for the first prompt, when this form took 537,
// the accumulators crowd the registers), 8 waves on one tile (561), stages not merged (557), deeper rings, the two
// chains of scores interleaved, waves' priorities, tiles in descending order of their keys (no gain or worse).
// With NS = 2 the workgroup has two such sets of waves, each with LDS of its own, for the first and the second half
// of the keys; the second set hands its O, m and l to the first through LDS at the end.
constexpr int NW = 4, BM = NW * 32;  // waves of a part, rows
constexpr int BK = 64;               // keys per tile

template <int DP, int NS>
__global__ __launch_bounds__(64 * NW * NS, 2) void prompt_kernel(AttnArgs a, int slots) {
  constexpr int CH = DP / 8, KST = DP / 16, DB = DP / 32;  // chunks a row, 16-value steps, 32-value blocks
  constexpr int KB = BK * DP * 2;                          // bytes of a K or V tile
  constexpr int LPW = KB / 1024 / NW, RPI = BK / LPW;      // 1 KB loads per wave and operand; rows between them
  constexpr int VRING = 2 * KB;                            // two slots for K tiles, two for V tiles
  extern __shared__ __align__(16) uint8_t smem_all[];
  const int lane = threadIdx.x & 63, part = NS > 1 ? uni(threadIdx.x >> 6) / NW : 0, wave = uni(threadIdx.x >> 6) % NW;
  const int l32 = lane & 31, h = lane >> 5;
  uint8_t* smem = smem_all + part * 4 * KB;

  // Workgroups go to the 8 XCDs round-robin: with the key head as the fast index, the tiles of a head meet in
  // one L2 (for 8 key heads; in few for other counts). The last rows, which see the most keys under a causal
  // mask, start first.
  const int kvh = blockIdx.x % a.Hkv, slot = slots - 1 - blockIdx.x / a.Hkv;
  int tile;
  Seq s;
  if (!locate<BM>(a, slot, s, tile)) return;
  const int nr = s.lq * a.G;  // rows of this sequence and key head

  // the keys row r sees: 0 .. lim(r) - 1
  auto lim = [&](int r) { return a.causal ? min(max(r / a.G + s.lk - s.lq + 1, 0), s.lk) : s.lk; };
  const int r0 = tile * BM + wave * 32;
  const int row = min(r0 + l32, nr - 1), row_lim = lim(row);
  v8bf qf[KST];
  {
    const uint16_t* p = a.q + (s.q0 + row / a.G) * a.sqt + (int64_t)(kvh * a.G + row % a.G) * a.sqh;
#pragma unroll
    for (int i = 0; i < KST; ++i) {
      const int c = 2 * i + h;
      v4u x = {0, 0, 0, 0};
      if (DP == a.D || c * 8 < a.D) x = *reinterpret_cast<const v4u*>(p + c * 8);
      qf[i] = __builtin_bit_cast(v8bf, x);
    }
  }
  const int kend = uni(lim(min(tile * BM + BM, nr) - 1));  // keys of the workgroup
  const int wmin = uni(r0 < nr ? lim(r0) : 0), wmax = uni(r0 < nr ? lim(min(r0 + 32, nr) - 1) : 0);
  const int all = (kend + BK - 1) / BK, nt = (all + NS - 1) / NS, t0 = part * nt;  // tiles; of a part; its first
  // this wave's tiles; those every row sees whole
  const int nw = min(max((wmax + BK - 1) / BK - t0, 0), nt), nfull = min(max(wmin / BK - t0, 0), nt);

  // DMA of a tile: load i of a wave brings rows RPI i + .. to byte 1024 (NW i + wave) + 16 lane of its slot; the rows
  // of a lane differ by RPI, a multiple of 16, so they share one place in the swizzle and one lane offset. The
  // buffer resource starts at the load's first row and ends behind the sequence's last key: what is read past it is
  // zero, so keys behind a sequence, whatever they hold, meet the product as zeros (rows wholly behind it: no
  // memory access). Resources move in 64 bits; lane offsets stay within a few rows.
  uint32_t ofk, ofv;
  {
    const int r = wave * (64 / CH) + lane / CH, ck = (lane % CH) ^ Lds<DP>::swk(r), cv = (lane % CH) ^ Lds<DP>::swv(r);
    static_assert(RPI % 16 == 0 && RPI == NW * (64 / CH), "rows of a lane share the swizzle");
    ofk = ck * 8 < a.D ? (uint32_t)r * (uint32_t)a.skt * 2u + ck * 16 : 0x80000000u;  // past every resource, also with the
    ofv = cv * 8 < a.D ? (uint32_t)r * (uint32_t)a.svt * 2u + cv * 16 : 0x80000000u;  // rows (below 2^31 bytes) added
  }
  const uint16_t* kp = a.k + s.k0 * a.skt + (int64_t)kvh * a.skh;
  const uint16_t* vp = a.v + s.k0 * a.svt + (int64_t)kvh * a.svh;
  // the tiles that are being brought in: where they start, and the keys from there to the sequence's end
  const uint32_t kr2 = (uint32_t)a.skt * 2u, vr2 = (uint32_t)a.svt * 2u;  // bytes from row to row
  const uint8_t *kb = reinterpret_cast<const uint8_t*>(kp) + (int64_t)t0 * BK * kr2,
                *vb = reinterpret_cast<const uint8_t*>(vp) + (int64_t)t0 * BK * vr2;
  int kleft = s.lk - t0 * BK, vleft = kleft;
  auto load_k = [&](int i, uint32_t to) __attribute__((always_inline)) {
    const int last = min(max(kleft, 0), BK) - 1;  // -1: nothing is left, a resource of no bytes
    const uint32_t n = ((uint32_t)last * kr2 + a.D * 2) & ~(uint32_t)(last >> 31);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(kb, n), (SS_LDS void*)((SS_LDS uint8_t*)smem + to + (NW * i + wave) * 1024), 16,
                                             ofk + (uint32_t)(i * RPI) * kr2, 0, 0, 0);
  };
  auto load_v = [&](int i, uint32_t to) __attribute__((always_inline)) {
    const int last = min(max(vleft, 0), BK) - 1;  // -1: nothing is left, a resource of no bytes
    const uint32_t n = ((uint32_t)last * vr2 + a.D * 2) & ~(uint32_t)(last >> 31);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(vb, n), (SS_LDS void*)((SS_LDS uint8_t*)smem + to + (NW * i + wave) * 1024), 16,
                                             ofv + (uint32_t)(i * RPI) * vr2, 0, 0, 0);
  };
  auto next_k = [&]() __attribute__((always_inline)) { kb += (int64_t)BK * kr2, kleft -= BK; };
  auto next_v = [&]() __attribute__((always_inline)) { vb += (int64_t)BK * vr2, vleft -= BK; };

  // this lane's places in a tile: K row l32 (chunk 2 i + h), V row 4 h + (lane % 16) / 4 of a 16-key step; the XOR
  // of the swizzle leaves KST addresses for K and DB for V, the rest are constant offsets
  const int vrow = 4 * h + ((lane & 15) >> 2), vcol = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1), vsub = (lane & 1) * 8;
  uint32_t ka[KST], va[DB];
#pragma unroll
  for (int i = 0; i < KST; ++i) ka[i] = l32 * DP * 2 + ((2 * i + h) ^ Lds<DP>::swk(l32)) * 16;
#pragma unroll
  for (int d = 0; d < DB; ++d) va[d] = vrow * DP * 2 + ((d * 4 + vcol) ^ Lds<DP>::swv(vrow)) * 16 + vsub;

  v16f O[DB], S0, S1;
  v8bf kf[KST], vf[2][DB], P[2];
  float m = kLow, l = 0.0f;
  float rise = kRise;  // below any sum while a row's maximum is big: every stage then takes its powers the careful way
#pragma unroll
  for (int d = 0; d < DB; ++d) {
    O[d] = v16f{};
    vf[0][d] = vf[1][d] = __builtin_bit_cast(v8bf, v4u{0, 0, 0, 0});
  }
  P[0] = P[1] = __builtin_bit_cast(v8bf, v4u{0, 0, 0, 0});

  auto read_k = [&](int i, uint32_t at) __attribute__((always_inline)) {
    kf[i] = *reinterpret_cast<const SS_LDS v8bf*>((const SS_LDS uint8_t*)smem + at + ka[i]);
  };
  auto read_v = [&](int kk, int d, uint32_t at) __attribute__((always_inline)) {  // 16 keys
    const SS_LDS uint8_t* p = (const SS_LDS uint8_t*)smem + at + va[d] + kk * 16 * DP * 2;
    const v4s x = read_tr(p), y = read_tr(p + 8 * DP * 2);
    vf[kk][d] = __builtin_bit_cast(v8bf, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  // one stage: `cur` holds its scores, `nxt` receives those of the next; kn: LDS offset of the keys of the stage after
  // the next, vc: of this stage's values; `side`: work beside it (loads)
  auto stage = [&](v16f& cur, v16f& nxt, uint32_t kn, uint32_t vc, int first, auto side, auto maskc) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(maskc)::value) {
      const int left = row_lim - first - 4 * h;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (8 * (i / 4) + i % 4 >= left) cur[i] = -INFINITY;
    }
    side();
    nxt = v16f{};
    v4u pk[2];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // a step of the scores' chain, a step of the values, two powers; then the fragments just used are read anew
#pragma unroll
      for (int j = i * KST / 8; j < (i + 1) * KST / 8; ++j) {
        nxt = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[j], qf[j], nxt, 0, 0, 0);
        read_k(j, kn);
      }
#pragma unroll
      for (int j = i * 2 * DB / 8; j < (i + 1) * 2 * DB / 8; ++j) {
        O[j % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[j / DB][j % DB], P[j / DB], O[j % DB], 0, 0, 0);
        read_v(j / DB, j % DB, vc);
      }
      const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(cur[2 * i], a.c, -m));
      const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(cur[2 * i + 1], a.c, -m));
      sum += x + y;
      pk[i / 4][i % 4] = pack_bf16x2(x, y);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (__builtin_expect(__any(sum > rise), 0)) {
      float mt = cur[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) mt = fmaxf(mt, cur[i]);
      const float mn = fmaxf(m, ceilf(pair_max(mt) * a.c)), f = __builtin_amdgcn_exp2f(m - mn);  // a power of two: exact
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[d][i] *= f;
      const bool big = is_big(m);
      rise = unif(__any(big) ? -1.0f : kRise);
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s0 = cur[2 * i], s1 = cur[2 * i + 1];
        const float x = __builtin_amdgcn_exp2f(big ? s0 * a.c - m : __builtin_fmaf(s0, a.c, -m));
        const float y = __builtin_amdgcn_exp2f(big ? s1 * a.c - m : __builtin_fmaf(s1, a.c, -m));
        sum += x + y;
        pk[i / 4][i % 4] = pack_bf16x2(x, y);
      }
    }
    l += sum;
    P[0] = __builtin_bit_cast(v8bf, pk[0]);
    P[1] = __builtin_bit_cast(v8bf, pk[1]);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(maskc)::value) {
      if (wmin < s.lk && first + 32 > wmin) {  // keys were loaded that some row does not see (its rows may be one token's)
        uint32_t odd = 0;
#pragma unroll
        for (int j = 0; j < 2 * DB; ++j) {
          const v4u w = __builtin_bit_cast(v4u, vf[j / DB][j % DB]);
#pragma unroll
          for (int i = 0; i < 4; ++i) odd |= odd_bf16x2(w[i]);
        }
        if (__builtin_expect(__any(odd != 0), 0)) {
#pragma unroll
          for (int j = 0; j < 2 * DB; ++j) {
            v4u w = __builtin_bit_cast(v4u, vf[j / DB][j % DB]);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = even_out(w[i]);
            vf[j / DB][j % DB] = __builtin_bit_cast(v8bf, w);
          }
          add_odd<DP>(O, (const SS_LDS uint8_t*)smem + vc, row_lim - first, h);
        }
      }
    }
  };

  // Iteration t reads K tile t + 1 and V tile t and brings in K tile t + 2 and V tile t + 1, into the slots of K tile t
  // and V tile t - 1, which were read in iteration t - 1: one wait and one barrier a tile.
  uint32_t k0 = 0, k1 = KB, v0 = VRING, v1 = VRING + KB;  // slots of tiles t, t + 1
  if (nt > 0) {
#pragma unroll
    for (int i = 0; i < LPW; ++i) load_k(i, k0);
    next_k();
#pragma unroll
    for (int i = 0; i < LPW; ++i) load_k(i, k1);
    next_k();
#pragma unroll
    for (int i = 0; i < LPW; ++i) load_v(i, v0);
    next_v();
    __builtin_amdgcn_s_waitcnt(vm(2 * LPW));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < KST; ++i) read_k(i, 0);
    S0 = v16f{};
#pragma unroll
    for (int i = 0; i < KST; ++i) S0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i], qf[i], S0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < KST; ++i) read_k(i, KB / 2);
    const int left = row_lim - t0 * BK - 4 * h;
    float mt = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (8 * (i / 4) + i % 4 < left) mt = fmaxf(mt, S0[i]);
    m = fmaxf(m, ceilf(pair_max(mt) * a.c));
    rise = unif(__any(is_big(m)) ? -1.0f : kRise);
  }
  auto turn = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x7 << 4);  // vmcnt(0), lgkmcnt(0): this wave's loads and LDS reads
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto rotate = [&]() __attribute__((always_inline)) {
    next_k();
    next_v();
    const uint32_t x = k0, y = v0;
    k0 = k1, k1 = x;
    v0 = v1, v1 = y;
  };
  auto tile_of = [&](int t, auto maskc) __attribute__((always_inline)) {
    turn();
    if constexpr (decltype(maskc)::value) renew(ofk), renew(ofv);
    stage(S0, S1, k1, v0, (t0 + t) * BK, [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < LPW; ++i) load_v(i, v1);
    }, maskc);
    stage(S1, S0, k1 + KB / 2, v0 + KB / 2, (t0 + t) * BK + 32, [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < LPW; ++i) load_k(i, k0);
    }, maskc);
    rotate();
  };
  int t = 0;
  for (; t < nfull; ++t) tile_of(t, std::false_type{});
  for (; t < nw; ++t) tile_of(t, std::true_type{});
#pragma unroll
  for (int j = 0; j < 2 * DB; ++j)  // the last stage's values
    O[j % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[j / DB][j % DB], P[j / DB], O[j % DB], 0, 0, 0);
  for (; t < nt; ++t) {  // the other waves' tiles
    turn();
#pragma unroll
    for (int i = 0; i < LPW; ++i) load_v(i, v1);
#pragma unroll
    for (int i = 0; i < LPW; ++i) load_k(i, k0);
    rotate();
  }
  __builtin_amdgcn_s_waitcnt(vm(0));  // no load may outlive the workgroup

  float lt = pair_sum(l);
  if constexpr (NS > 1) {  // the second part's results go through its LDS to the waves of the first
    static_assert(NS == 2, "two parts");
    typedef float v4f __attribute__((ext_vector_type(4)));
    __shared__ float red[2][64 * NW];
    SS_LDS v4f* to = (SS_LDS v4f*)(smem_all + 4 * KB) + wave * 64 + lane;
    __syncthreads();
    if (part == 1) {
      red[0][wave * 64 + lane] = m;
      red[1][wave * 64 + lane] = lt;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) to[(d * 4 + g) * NW * 64] = v4f{O[d][4 * g], O[d][4 * g + 1], O[d][4 * g + 2], O[d][4 * g + 3]};
    }
    __syncthreads();
    if (part == 1) return;
    const float m1 = red[0][wave * 64 + lane], mn = fmaxf(m, m1);
    const float f0 = __builtin_amdgcn_exp2f(m - mn), f1 = __builtin_amdgcn_exp2f(m1 - mn);
    m = mn;
    lt = lt * f0 + red[1][wave * 64 + lane] * f1;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const v4f x = to[(d * 4 + g) * NW * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) O[d][4 * g + e] = O[d][4 * g + e] * f0 + x[e] * f1;
      }
  }
  const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;  // a row that sees no key: zeros (of a NaN: NaN)
  const bool ok = r0 + l32 < nr;
  const int64_t tok = s.q0 + row / a.G;
  const int head = kvh * a.G + row % a.G;
  if (a.lse && ok && h == 0)
    a.lse[head * a.Tq + tok] = lt == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(lt)) * 0.69314718056f;
  uint16_t* op = a.o + tok * a.sot + head * a.soh;
#pragma unroll
  for (int d = 0; d < DB; ++d) {
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      // lane l holds values 8g + 4h .. +3 and 8(g+1) + 4h .. +3 of its row; exchanged with lane l ^ 32, the lower
      // lane has 8g .. 8g+7 and the upper 8(g+1) .. 8(g+1)+7
      uint32_t x[2], y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[e] = pack_bf16x2(O[d][4 * g + 2 * e] * inv, O[d][4 * g + 2 * e + 1] * inv);
        y[e] = pack_bf16x2(O[d][4 * g + 4 + 2 * e] * inv, O[d][4 * g + 5 + 2 * e] * inv);
      }
      const auto e0 = __builtin_amdgcn_permlane32_swap(x[0], y[0], false, false);
      const auto e1 = __builtin_amdgcn_permlane32_swap(x[1], y[1], false, false);
      const int col = d * 32 + 8 * (g + h);
      if (ok && (DP == a.D || col < a.D)) *reinterpret_cast<v4u*>(op + col) = v4u{e0[0], e1[0], e0[1], e1[1]};
    }
  }
}

// Two parts where a CU has few workgroups and a row many keys. Heads of 64: 12 of them, 14.2 against 15.6 us at 1000 causal
// tokens (96 workgroups), 43.0 / 49.3 at 4000 (384), 18.2 / 20.4 at 1500 without a mask; 8 of them, 86.8 / 99.1 at 8000 (504);
// 8.6 / 8.0 at 300, 11.3 / 11.5 at 600. Heads of 128: 8 of them, 31.1 / 33.6 at 2048 tokens (136), 55.1 / 60.7 at 4000
// (256), 22.1 / 22.7 at 1200 without a mask; 32 over 8, 15.5 / 14.3 at 512 tokens, 22.3 / 21.6 at 960 (248), 34.9 / 34.0 at
// 1536 (392); 12, no mask, 101.1 / 90.3 at 3500 (336).
template <int DP> hipError_t launch_prompt(const AttnArgs& a, hipStream_t st) {
  const int64_t slots = a.Tq * a.G / BM + a.B;
  auto go = [&](auto kern, int parts) -> hipError_t {
    const int lds = parts * 4 * BK * DP * 2;
    const hipError_t e = lds_limit((const void*)kern, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)(slots * a.Hkv)), dim3(64 * NW * parts), lds, st, a, (int)slots);
    return hipGetLastError();
  };
  const int64_t wgs = slots * a.Hkv, cus = num_cus_p();
  const bool two = DP <= 64 ? wgs <= 2 * cus && a.Tk >= 512 * (int64_t)a.B : wgs <= cus && a.Tk >= 1024 * (int64_t)a.B;
  return two ? go(prompt_kernel<DP, 2>, 2) : go(prompt_kernel<DP, 1>, 1);
}

// ---- few rows per sequence: the keys split over waves and workgroups ---------------------------------------------
// Single tokens over a cache read every key and value once for a handful of rows (HBM bound), so the work is cut
// along the keys: a tile has 32 rows, each wave takes every FW-th unit of 32 keys of its workgroup's share with a
// ring of its own in LDS (whole 1 KB DMA loads, no barrier in the loop: a wave waits for its own loads only),
// and gridDim.y workgroups share a tile's keys. The waves of a workgroup join through LDS, the workgroups through
// float32 parts (each normalised, with its row's log2 of the sum: maximum and sum in one float, exact to 2^-24 of the
// maximum, as the scores themselves are) that join_kernel adds in order.
// Measured: 64 caches of 4096 keys on average (32 heads of 128 over 8): 240 us, 5.0 TB/s, a large copy's rate on this card
// (4.9); one cache of 4000: 6.5 us here and 3 in the join, both chains of latencies (lengths, keys, LDS, parts).
// Short chunks of tokens over a long cache come here too, several tiles of 32 rows to a sequence (few_rows).
constexpr int FW = 2, FR = 2, FM = 32;  // waves, units in a wave's ring, rows
constexpr int kMaxParts = 32;           // workgroups that share a tile's keys

template <int DP, bool SPLIT>
__global__ __launch_bounds__(64 * FW, 2) void few_kernel(AttnArgs a, float* __restrict__ part) {
  constexpr int CH = DP / 8, KST = DP / 16, DB = DP / 32;
  constexpr int KB = 32 * DP * 2, UNIT = 2 * KB, RING = FR * UNIT;
  constexpr int LPU = KB / 1024;            // 1 KB loads per unit and operand
  constexpr int OST = DP * 4 + 16;          // bytes of a joined row, padded
  static_assert(FM * OST <= RING, "a wave's results fit its ring");
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[FW][2][FM];
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int kvh = blockIdx.x % a.Hkv, slot = blockIdx.x / a.Hkv;
  int tile;
  Seq s;
  if (!locate<FM>(a, slot, s, tile)) return;
  const int nr = s.lq * a.G;
  auto lim = [&](int r) { return a.causal ? min(max(r / a.G + s.lk - s.lq + 1, 0), s.lk) : s.lk; };
  const int r0 = tile * FM, rows = min(nr - r0, FM);
  const int r = min(r0 + l32, nr - 1);
  const int row_lim = lim(r);
  const int kend = uni(lim(r0 + rows - 1)), kmin = uni(lim(r0));
  const int units = (kend + 31) / 32;
  const int ulo = (int)((int64_t)units * blockIdx.y / gridDim.y), uhi = (int)((int64_t)units * (blockIdx.y + 1) / gridDim.y);

  uint32_t ofk[8], ofv[8];  // LPU of them
  static_assert(LPU <= 8, "loads per unit");
#pragma unroll
  for (int i = 0; i < LPU; ++i) {
    const int x = i * 64 + lane, row = x / CH, ck = (x % CH) ^ Lds<DP>::swk(row), cv = (x % CH) ^ Lds<DP>::swv(row);
    ofk[i] = ck * 8 < a.D ? (uint32_t)row * (uint32_t)a.skt * 2u + ck * 16 : 0xFFFFFF00u;
    ofv[i] = cv * 8 < a.D ? (uint32_t)row * (uint32_t)a.svt * 2u + cv * 16 : 0xFFFFFF00u;
  }
  const uint16_t* kp = a.k + s.k0 * a.skt + (int64_t)kvh * a.skh;
  const uint16_t* vp = a.v + s.k0 * a.svt + (int64_t)kvh * a.svh;
  SS_LDS uint8_t* ring = (SS_LDS uint8_t*)smem + wave * RING;
  auto issue = [&](int u, int at) {
    const int n = min(s.lk - u * 32, 32);  // >= 1
    const __amdgpu_buffer_rsrc_t rk = rsrc(kp + (int64_t)u * 32 * a.skt, (uint32_t)(n - 1) * (uint32_t)a.skt * 2u + a.D * 2),
                                 rv = rsrc(vp + (int64_t)u * 32 * a.svt, (uint32_t)(n - 1) * (uint32_t)a.svt * 2u + a.D * 2);
#pragma unroll
    for (int i = 0; i < LPU; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (SS_LDS void*)(ring + at + i * 1024), 16, ofk[i], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < LPU; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (SS_LDS void*)(ring + at + KB + i * 1024), 16, ofv[i], 0, 0, 0);
  };

  if (ulo + wave < uhi) issue(ulo + wave, 0);
  v8bf qf[KST];
  {
    const uint16_t* p = a.q + (s.q0 + r / a.G) * a.sqt + (int64_t)(kvh * a.G + r % a.G) * a.sqh;
#pragma unroll
    for (int i = 0; i < KST; ++i) {
      const int c = 2 * i + h;
      v4u x = {0, 0, 0, 0};
      if (DP == a.D || c * 8 < a.D) x = *reinterpret_cast<const v4u*>(p + c * 8);
      qf[i] = __builtin_bit_cast(v8bf, x);
    }
  }
  v16f O[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) O[d] = v16f{};
  float m = kLow, l = 0.0f;
  bool careful = false;  // some row's maximum is big
  const int vrow = 4 * h + ((lane & 15) >> 2), vcol = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1), vsub = (lane & 1) * 8;

  int at = 0;
  for (int u = ulo + wave; u < uhi; u += FW) {
    if (u + FW < uhi) {
      issue(u + FW, RING / FR - at);
      // unit u has landed when only the loads just issued are outstanding (loads complete in order)
      __builtin_amdgcn_s_waitcnt(((2 * LPU) & 0xF) | (((2 * LPU) >> 4) << 14) | (0x7 << 4) | (0xF << 8));
    } else {
      __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xF << 8));
    }
    __builtin_amdgcn_sched_barrier(0);
    const SS_LDS uint8_t* kt = ring + at;
    const SS_LDS uint8_t* vt = kt + KB;
    const int vo = at + KB;
    at = RING / FR - at;
    v16f S = v16f{};
#pragma unroll
    for (int i = 0; i < KST; ++i) {
      const v8bf kf = *reinterpret_cast<const SS_LDS v8bf*>(kt + l32 * DP * 2 + ((2 * i + h) ^ Lds<DP>::swk(l32)) * 16);
      S = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i], S, 0, 0, 0);
    }
    if (u * 32 + 32 > kmin) {
      const int left = row_lim - u * 32 - 4 * h;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (8 * (i / 4) + i % 4 >= left) S[i] = -INFINITY;
    }
    float mt = S[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) mt = fmaxf(mt, S[i]);
    if (__any(mt * a.c > m + kSlack)) {
      const float mn = fmaxf(m, pair_max(mt) * a.c), f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[d][i] *= f;
      careful = __any(is_big(m));
    }
    float pc = a.c, pm = m;  // a power is 2^(pc S - pm)
    if (__builtin_expect(careful, 0)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) S[i] = S[i] * a.c - m;
      pc = 1.0f, pm = 0.0f;
    }
    if (kmin < s.lk && u * 32 + 32 > kmin) {  // keys were loaded that some row does not see (the rows may be one token's)
      uint32_t odd = 0;
#pragma unroll
      for (int i = 0; i < LPU; ++i) {
        const v4u w = *reinterpret_cast<const SS_LDS v4u*>(vt + (i * 64 + lane) * 16);
        odd |= odd_bf16x2(w[0]) | odd_bf16x2(w[1]) | odd_bf16x2(w[2]) | odd_bf16x2(w[3]);
      }
      if (__builtin_expect(__any(odd != 0), 0)) {
        add_odd<DP>(O, vt, row_lim - u * 32, h);
#pragma unroll 1
        for (int i = 0; i < LPU; ++i) {
          SS_LDS v4u* p = (SS_LDS v4u*)(ring + vo + (i * 64 + lane) * 16);
          const v4u w = *p;
          *p = v4u{even_out(w[0]), even_out(w[1]), even_out(w[2]), even_out(w[3])};
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);
        asm volatile("" ::: "memory");  // the reads below stay below
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    v8bf P[2];
    {
      v4u pk[2];
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(S[i], pc, -pm));
        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(S[i + 1], pc, -pm));
        sum += x + y;
        pk[i / 8][(i % 8) / 2] = pack_bf16x2(x, y);
      }
      l += sum;
      P[0] = __builtin_bit_cast(v8bf, pk[0]);
      P[1] = __builtin_bit_cast(v8bf, pk[1]);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const int ra = kk * 16 + vrow, rb = ra + 8, c = d * 4 + vcol;
        const v4s x = read_tr((const SS_LDS uint8_t*)(vt + ra * DP * 2 + (c ^ Lds<DP>::swv(ra)) * 16 + vsub));
        const v4s y = read_tr((const SS_LDS uint8_t*)(vt + rb * DP * 2 + (c ^ Lds<DP>::swv(rb)) * 16 + vsub));
        const v8bf vf = __builtin_bit_cast(v8bf, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
        O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, P[kk], O[d], 0, 0, 0);
      }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this unit's LDS reads are done before its slot is filled again
    __builtin_amdgcn_sched_barrier(0);
  }

  // join the waves: a wave's O goes through its own ring, scaled to the workgroup's maximum
  if (h == 0) red[wave][0][l32] = m;
  const float lt = pair_sum(l);
  if (h == 0) red[wave][1][l32] = lt;
  __syncthreads();
  float M = red[0][0][l32];
#pragma unroll
  for (int w = 1; w < FW; ++w) M = fmaxf(M, red[w][0][l32]);
  if (l32 < rows) {
    const float f = __builtin_amdgcn_exp2f(m - M);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        typedef float v4f __attribute__((ext_vector_type(4)));
        *reinterpret_cast<SS_LDS v4f*>(ring + l32 * OST + (d * 32 + 8 * g + 4 * h) * 4) =
            v4f{O[d][4 * g] * f, O[d][4 * g + 1] * f, O[d][4 * g + 2] * f, O[d][4 * g + 3] * f};
      }
  }
  __syncthreads();
  const int quads = a.D / 4;
  for (int i = threadIdx.x; i < rows * quads; i += 64 * FW) {
    const int row = i / quads, c = (i - row * quads) * 4;
    float M2 = red[0][0][row], L = 0.0f;
#pragma unroll
    for (int w = 1; w < FW; ++w) M2 = fmaxf(M2, red[w][0][row]);
#pragma unroll
    for (int w = 0; w < FW; ++w) L += red[w][1][row] * __builtin_amdgcn_exp2f(red[w][0][row] - M2);
    float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < FW; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(smem + w * RING + row * OST + c * 4);
      o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int rr = r0 + row, head = kvh * a.G + rr % a.G;
    const int64_t tok = s.q0 + rr / a.G;
    const float lg = L == 0.0f ? -INFINITY : M2 + __builtin_amdgcn_logf(L);  // log2 of the row's sum
    if constexpr (SPLIT) {
      const int64_t Hq = (int64_t)a.Hkv * a.G, at_row = (blockIdx.y * a.Tq + tok) * Hq + head;
      *reinterpret_cast<float4*>(part + at_row * a.D + c) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      if (c == 0) part[(int64_t)gridDim.y * a.Tq * Hq * a.D + at_row] = lg;
    } else {
      *reinterpret_cast<uint2*>(a.o + tok * a.sot + head * a.soh + c) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (a.lse && c == 0) a.lse[head * a.Tq + tok] = lg * 0.69314718056f;
    }
  }
}

// o = sum_s w_s part_s, w_s = 2^(lg_s - max) / sum of them: one workgroup per (token, head), 16 bytes a thread,
// the parts dealt over groups of threads and joined in LDS in a fixed order. A launch this small is a chain of load
// latencies, so all parts (kMaxParts at most) set out together with the logarithms their weights need.
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, const float* __restrict__ part, int splits) {
  constexpr int kPre = kMaxParts / 8;  // parts a thread: D <= 128 leaves 8 groups or more
  __shared__ float4 acc[256];
  const int Hq = a.Hkv * a.G;
  const int64_t row = blockIdx.x, tok = row / Hq, n = a.Tq * Hq;
  const int head = (int)(row - tok * Hq);
  const float* lg = part + (int64_t)splits * n * a.D + row;
  const int lane = threadIdx.x & 63, last = splits - 1;
  const int quads = a.D / 4, groups = 256 / quads, g = threadIdx.x / quads, c = threadIdx.x % quads;
  auto at = [&](int s) { return *reinterpret_cast<const float4*>(part + (s * n + row) * a.D + c * 4); };
  const float l0 = lg[min(lane, last) * n];
  float lp[kPre];
  float4 xp[kPre];
#pragma unroll
  for (int i = 0; i < kPre; ++i) {
    lp[i] = lg[min(g + i * groups, last) * n];
    xp[i] = at(min(g + i * groups, last));
  }
  // rows of no sequence have no parts (what was read of them is not used)
  if (tok < bound(a.cu_q, 0, a.Tq) || tok >= bound(a.cu_q, a.B, a.Tq)) return;
  const float M = wave_max(l0);
  auto power = [&](float l) { return l == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(l - M); };  // (of a NaN: NaN)
  float sum = lane < splits ? power(l0) : 0.0f;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float4 o = make_float4(0, 0, 0, 0);
  auto add = [&](float l, const float4& x) {
    const float w = power(l) * inv;
    o.x += w * x.x; o.y += w * x.y; o.z += w * x.z; o.w += w * x.w;
  };
  if (g < groups) {
#pragma unroll
    for (int i = 0; i < kPre; ++i)
      if (g + i * groups < splits) add(lp[i], xp[i]);
  }
  acc[threadIdx.x] = o;
  __syncthreads();
  if (threadIdx.x < quads) {
    for (int k = 1; k < groups; ++k) {
      const float4 x = acc[k * quads + threadIdx.x];
      o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
    }
    *reinterpret_cast<uint2*>(a.o + tok * a.sot + head * a.soh + threadIdx.x * 4) =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[head * a.Tq + tok] = sum == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(sum)) * 0.69314718056f;
}

// Calls whose sequences have 32 rows or fewer on average go to few_kernel, and those whose tiles of 32 rows are few beside
// the keys (128 at most, and 40 keys or more for each): a chunk of tokens over a long cache, where the tiles of 128 rows would
// leave the chip idle. 16 tokens, 32 heads of 128 over 8 (16 tiles): 14.9 against 18.4 us over 1024 keys, 23.3 / 47.5 over
// 4096; 128 tokens (128 tiles): 24.0 / 20.1 over 1024, 36.2 / 49.6 over 4096, 78.9 / 170 over 16384; 4 chunks of 64 rows, 28
// heads over 4 (32 tiles): 22.0 / 18.7 over 1024, 24.8 / 28.7 over 2048.
inline bool few_rows(int64_t Tq, int64_t Tk, int64_t B, int64_t G, int64_t Hkv) {
  const int64_t tiles = (Tq * G + (FM - 1) * B) / FM * Hkv;
  return Tk > 0 && (Tq * G <= FM * B || (tiles <= 128 && tiles <= Tk / B / 40));
}
inline int64_t few_slots(int64_t Tq, int64_t B, int64_t G) { return Tq * G / FM + B; }
// Workgroups per tile. The chip holds two workgroups a CU (four for heads up to 64), and about as many in all is the
// best split: one cache of 4096 keys, 32 heads of 128 over 8: 10.4 us in 32 parts, 11.6 in 16, 12.0 in 64; 8 caches of 2048
// 19.6 in 8, 22.9 in 4, 22.5 in 16; 16 of 2048 29.7 in 4, 35.7 in 2, 31.7 in 8. Where the tiles alone fill it, up to 4 parts
// of 1024 keys even out lengths: 64 caches of 1 to 8192 keys 213 in 4, 274 whole (all of 8192: 384 / 393). The join costs 3
// us: below 512 keys a tile stays whole (9.8 in one, 9.7 in 3 at 384), below 1024 where it would be cut in few parts
// (16 caches of 512: 12.8 whole, 13.5 in 4).
// The lengths are in device memory, so both rules go by the mean of the room in k, and a call whose lengths are far from it
// runs by another's plan: 64 caches of 1024 keys in room for 8192 take 51.7 us, without the room 45.0; of 256 28.9 / 14.9;
// of 64 24.4 / 6.6; 16 tokens over 256 keys in room for 16384 19.3 / 8.6; one packed sequence of 8192 keys among 63 of 64
// 101 us (alone 10.6), where the same in room for 8192 each takes 49.
inline int splits(int64_t Tq, int64_t Tk, int64_t B, int64_t G, int64_t Hkv, int64_t D) {
  if (Tq * G * Hkv >= 1 << 24) return 1;  // join_kernel: 256 threads a row, fewer than 2^32 in a launch
  const int64_t tiles = std::max<int64_t>(B, Tq * G / FM) * Hkv, keys = Tk / B;
  int64_t n = std::min<int64_t>((D <= 64 ? 4 : 2) * (int64_t)num_cus_p() / tiles, kMaxParts);
  if (keys < (n < 8 ? 1024 : 512)) return 1;
  if (n < 4) n = std::max<int64_t>(n, std::min<int64_t>(keys / 1024, 4));
  return (int)std::min<int64_t>(n, keys / 64);
}

template <int DP> hipError_t launch_few(const AttnArgs& a, void* ws, hipStream_t st) {
  const int n = splits(a.Tq, a.Tk, a.B, a.G, a.Hkv, a.D);
  constexpr int lds = FW * FR * 2 * 32 * DP * 2;
  const dim3 grid((unsigned)(few_slots(a.Tq, a.B, a.G) * a.Hkv), (unsigned)n);
  auto go = [&](auto kern) -> hipError_t {
    const hipError_t e = lds_limit((const void*)kern, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, grid, dim3(64 * FW), lds, st, a, static_cast<float*>(ws));
    return hipGetLastError();
  };
  if (n == 1) return go(few_kernel<DP, false>);
  const hipError_t e = go(few_kernel<DP, true>);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)(a.Tq * a.Hkv * a.G)), dim3(256), 0, st, a, static_cast<const float*>(ws), n);
  return hipGetLastError();
}

}  // namespace attn

int64_t attn_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  const int64_t G = Hq / Hkv;
  if (!attn::few_rows(Tq, Tk, B, G, Hkv)) return 0;
  const int64_t n = attn::splits(Tq, Tk, B, G, Hkv, D);
  return n == 1 ? 0 : n * Tq * Hq * (D + 1) * 4;
}

// a launch holds fewer than 2^32 threads
bool attn_fits(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv) {
  const int64_t G = Hq / Hkv, few = attn::few_rows(Tq, Tk, B, G, Hkv);
  return (few ? attn::few_slots(Tq, B, G) * 64 * attn::FW : (Tq * G / attn::BM + B) * 64 * attn::NW) * Hkv <= 0xFFFFFFFFLL;
}

hipError_t launch_attn(const AttnArgs& a, void* ws, hipStream_t st) {
  if (attn::few_rows(a.Tq, a.Tk, a.B, a.G, a.Hkv)) return a.D <= 64 ? attn::launch_few<64>(a, ws, st) : attn::launch_few<128>(a, ws, st);
  return a.D <= 64 ? attn::launch_prompt<64>(a, st) : attn::launch_prompt<128>(a, st);
}

}  // namespace ss
