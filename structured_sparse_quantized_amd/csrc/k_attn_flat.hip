// Attention of few query rows a sequence over a paged cache, or over contiguous keys under a sliding window (gfx950):
//   o = softmax(scale q k^T + mask) v of the keys that a row sees: with position p (the last row of a sequence has its last
//   key), j <= p and, under a window w with s first tokens, j > p - w or j < s.
//
// Mathematics, matrix instructions and LDS tiles are those of the packed attention (k_attn.hip): tiles of 32 rows, the (token,
// head) pairs of a sequence that share a key head; units of 32 keys; one pass with a running maximum and sum. Scores, maxima,
// sums, results and parts are float32; the powers are rounded to bf16, which the second product's matrix instruction takes
// (their sum is of the unrounded ones): 2^-8 of each at most. A result's error is 0.0021-0.0023 of its size, 0.0016 of which is
// its own rounding.
//
// Split. Such calls read every seen key and value once for a handful of rows (HBM bound), and lengths differ from sequence to
// sequence. So the work is laid out flat: the units of all tiles one after the other, and each of the launch's workgroups (as
// many as the chip holds at once) takes an equal run of them, whatever tile that begins and ends in. The lengths are in device
// memory, so the workgroups find their runs themselves, by a sum over the sequences, 64 a step (one token each, all but 16 of
// 1024 empty: 63 us, the 16 alone 33; all but 2 of 2048: 78, alone 17; 1024 of 500 keys on average 439 us, 4.8 TB/s). A tile
// that lies whole in a run is finished there; of one that is cut, each workgroup leaves a part (float32, normalised, with its
// row's log2 of the sum), a run's first tile in one place and its last in another, and join_kernel adds the parts in order.
//
// Loads. A unit is loaded to registers while the unit before it is computed, and goes to LDS when that is done. (Loads to LDS
// without registers, from addresses of each lane, gave wrong parts now and then where the unit in flight was cut. Why was not
// found: the unit that was read had landed by then, for that loop waited for all loads, the table's among them, at its end. The
// packed attention's loads to LDS, by a resource and scalar places, differ in no call: tests/test_gpu_attn_repeat.py.) Each of
// 32 lanes looks up the page of one key, a unit ahead. A load covers 4 rows of heads of 128, or 8 of 64: where page sizes are
// multiples of that, its address is a scalar, where 32 divides them one for the unit; other sizes take addresses of each lane
// (16 times 30 instructions a unit more). Values of keys that no row of the tile sees (behind the end, outside the window, of
// entries that name no page) are replaced by zeros, so whatever they hold stays out of the product.
// Measured (32 heads of 128 over 8): 64 tokens over 262144 keys in pages of 16, lengths 1 to 8192: 193 us and 9 in the join,
// 5.3 TB/s; one token over 4000 keys 12 us and 4: the chain lengths, run, table, keys, parts, and instructions fetched cold. 4
// units at least to a run (one token 15.9 us a call; 2: 16.8, 8: 17.1), 4 workgroups a CU (64 caches 199 us; 3: 201, 2: 207, 8:
// 203; of heads of 64 a CU holds six: 64 of 500 keys 36.5 us in four, 29.8 in six, 1024 of 2000 792 / 774, 2 of 20000 23.5 /
// 25.0).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "ss_attn.h"

namespace ss {
namespace flat {

using namespace attn;
constexpr int FW = 2, FM = 32;          // waves, rows
constexpr int kMinUnits = 4;            // a workgroup's run, at least
constexpr int kMostWhole = 128;         // units of a tile that is left whole, at most
constexpr int kJoin = 8;                // workgroups that share a cut tile's rows (14 rows: 8.1 us; 4: 11.4)

__device__ const uint4 kZeros = {0, 0, 0, 0};

// Parts in the workspace: one record per workgroup, then log2 of the sums [workgroup][2][FM], then the parts
// [workgroup][2][rows][D].
struct Record {  // of the tile that begins in this workgroup's run and ends in a later one
  int parts;     // 0: none
  int slot, rows, kvh, r0, unused;
  int64_t q0;
};
static_assert(sizeof(Record) == 32, "workspace layout");
struct Parts {
  Record* rec;
  float* lg;
  float* part;
  int rows;  // room of a part
};
__host__ __device__ inline Parts parts_of(void* ws, int64_t wgs, int rows) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  return {reinterpret_cast<Record*>(p), reinterpret_cast<float*>(p + wgs * sizeof(Record)),
          reinterpret_cast<float*>(p + wgs * (sizeof(Record) + 2 * FM * 4)), rows};
}

// Where a unit's keys lie: rows of one tensor; pages, of sizes that 32, 16 or 8 divides (so many adjacent rows share a page); any
// pages.
constexpr int kRows = 0, kAnyPages = 1;  // and 32, 16, 8

struct Seq {
  int64_t q0, k0;  // first query row, first key row (contiguous keys)
  int lq, lk;
};
__device__ __forceinline__ int64_t inside(int x, int64_t n) { return min(max((int64_t)x, (int64_t)0), n); }
// Bounds from device memory are clamped to the tensors, so whatever they hold, no access leaves q, k, v or o.
template <int KEYS> __device__ __forceinline__ Seq load_seq(const FlatArgs& a, int b) {
  Seq s;
  int64_t q0 = 0, q1 = a.Tq, k0 = 0, k1 = a.Tk;
  int len = 0x7FFFFFFF;
  if (a.cu_q) {
    q0 = inside(a.cu_q[b], a.Tq), q1 = inside(a.cu_q[b + 1], a.Tq);
  } else if (a.B > 1) {  // one row a sequence
    q0 = min((int64_t)b, a.Tq), q1 = min((int64_t)b + 1, a.Tq);
  }
  if (KEYS != kRows) {
    k1 = min((int64_t)a.cols * a.page, (int64_t)0x7FFFFF00);
    len = a.k_len[b];
  } else {
    if (a.cu_k) k0 = inside(a.cu_k[b], a.Tk), k1 = inside(a.cu_k[b + 1], a.Tk);
    if (a.k_len) len = a.k_len[b];
  }
  s.q0 = q0;
  s.k0 = k0;
  s.lq = (int)(max(q1, q0) - q0);
  s.lk = min(max(len, 0), (int)min(max(k1, k0) - k0, (int64_t)0x7FFFFF00));
  return s;
}
__host__ __device__ inline int tiles_of(int lq, int G) { return (int)(((uint32_t)lq * (uint32_t)G + (FM - 1)) / FM); }
// units of a tile of the sequence, at most (at least one, so that rows without keys are written)
__host__ __device__ inline int units_of(int window, int sinks, int tokens, int lq, int lk) {
  uint32_t n = ((uint32_t)lk + 31) / 32;
  if (window) {  // the tile's tokens see window + tokens - 1 adjacent keys between them, and the first ones
    const uint32_t len = (uint32_t)window + (uint32_t)(tokens < lq ? tokens : lq) - 1;
    const uint32_t m = (len + 62) / 32 + ((uint32_t)sinks + 31) / 32;
    n = m < n ? m : n;
  }
  return n > 1 ? (int)n : 1;
}
__host__ __device__ inline int tokens_of(int G) { return (FM - 1 + G - 1) / G + 1; }  // of a tile, at most

// Sum over this lane and those below it, by the lanes' own exchange: each step adds what lies so many lanes down.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);   // 1 down, within rows of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);   // 2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);   // 4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);   // 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // a row's last lane to rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
  return x;
}

// The transposing LDS read of what the wave itself has written: LDS serves a wave in order.
__device__ __forceinline__ v4s read_columns(SS_LDS uint8_t* p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16((SS_LDS v4s*)p); }

// The address, or that of zeros, without a branch over what computes it.
__device__ __forceinline__ const uint16_t* pick(bool take, const uint16_t* p) {
  const uint64_t mask = take ? ~0ull : 0ull;
  return reinterpret_cast<const uint16_t*>(((uint64_t)p & mask) | ((uint64_t)&kZeros & ~mask));
}

// a wave's room in LDS holds a unit's keys and values, and at the end its rows' results
constexpr int lds_bytes(int DP) { return FW * (2 * 32 * DP * 2 > FM * (DP * 4 + 16) ? 2 * 32 * DP * 2 : FM * (DP * 4 + 16)); }

template <int DP, int KEYS>
__global__ __launch_bounds__(64 * FW, 2) void flat_kernel(FlatArgs a, Parts ws) {
  constexpr int CH = DP / 8, KST = DP / 16, DB = DP / 32;
  constexpr int KB = 32 * DP * 2;    // bytes of a unit's keys, and of its values
  constexpr int LPU = KB / 1024;     // 1 KB loads per unit and operand
  constexpr int RPL = 64 / CH;       // rows of a load
  constexpr int OST = DP * 4 + 16;   // bytes of a joined row, padded
  constexpr int RING = lds_bytes(DP) / FW;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[FW][2][FM];
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;

  // ---- this workgroup's run: 64 sequences at a time, one a lane ---------------------------------------------------
  Seq mine;
  auto weight = [&](int i) -> int {  // units of sequence i's tiles (plan() leaves tiles whole where all could pass 31 bits)
    mine = Seq{0, 0, 0, 0};
    if (i >= a.B) return 0;
    mine = load_seq<KEYS>(a, i);
    return tiles_of(mine.lq, a.G) * a.Hkv * (a.whole ? 1 : units_of(a.window, a.sinks, a.tokens, mine.lq, mine.lk));
  };
  int upto = 0, total = 0;
#pragma unroll 1
  for (int c = 0; c < a.B; c += 64) {
    upto = wave_scan(weight(c + lane));
    total += __builtin_amdgcn_readlane(upto, 63);
  }
  const int run = (int)max(a.by_wgs((uint32_t)total + gridDim.x - 1), (uint32_t)(a.whole ? 1 : kMinUnits));
  int s0 = (int)min((int64_t)blockIdx.x * run, (int64_t)0x7FFFFFFF);
  const int s1 = (int)min((int64_t)s0 + run, (int64_t)total);
  if (!a.whole && threadIdx.x == 0) ws.rec[blockIdx.x].parts = 0;
  if (s0 >= total) return;
  int b = 0, before = 0;  // the sequence, and the work before it
  Seq s;
#pragma unroll 1
  for (int c = 0;; c += 64) {  // (ends: the work of all sequences passes s0)
    if (a.B > 64) upto = wave_scan(weight(c + lane));
    const uint64_t past = __ballot(before + upto > s0);
    if (past || c + 64 >= a.B) {
      const int l = past ? __ffsll((unsigned long long)past) - 1 : 0;
      b = c + l;
      if (l > 0) before += __builtin_amdgcn_readlane(upto, l - 1);
      auto of = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
      auto of64 = [&](int64_t x) { return (int64_t)((uint64_t)(uint32_t)of((int)(x >> 32)) << 32 | (uint32_t)of((int)x)); };
      s = Seq{of64(mine.q0), of64(mine.k0), of(mine.lq), of(mine.lk)};
      break;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  int tiles = tiles_of(s.lq, a.G), un = a.whole ? 1 : units_of(a.window, a.sinks, a.tokens, s.lq, s.lk);
  int th = (int)((uint32_t)(s0 - before) / (uint32_t)un);  // tile and key head in the sequence, the head fastest
  int j0 = (int)((uint32_t)(s0 - before) - (uint32_t)th * (uint32_t)un);  // (0 .. un - 1, whatever the bounds hold)
  if ((uint32_t)th >= (uint32_t)(tiles * a.Hkv)) return;  // (bounds that decrease may overlap: more work than the host knows)

  SS_LDS uint8_t* ring = (SS_LDS uint8_t*)smem + wave * RING;
  // this lane's bytes of a load of RPL adjacent rows, whose chunks go to their places in LDS (the places repeat after NK loads)
  constexpr int NK = DP >= 128 ? 4 : 2;
  uint32_t lane_k[NK], lane_v;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int x = i * RPL + lane / CH, c = (lane % CH) ^ Lds<DP>::swk(x);
    lane_k[i] = c * 8 < a.D ? (uint32_t)(lane / CH) * a.skt * 2u + c * 16 : 0x80000000u;  // (past every resource)
  }
  {
    const int c = (lane % CH) ^ Lds<DP>::swv(lane / CH);
    lane_v = c * 8 < a.D ? (uint32_t)(lane / CH) * a.svt * 2u + c * 16 : 0x80000000u;
  }
  bool first = true;
#pragma unroll 1
  while (true) {
    const int take = min(un - j0, s1 - s0);
    const int tile = uni((int)a.by_Hkv(th)), kvh = uni(th - tile * a.Hkv);
    const int nr = s.lq * a.G, r0 = tile * FM, rows = min(nr - r0, FM);
    // what the rows of token t of the sequence see
    auto lim = [&](int t) { return a.causal ? min(max(t + s.lk - s.lq + 1, 0), s.lk) : s.lk; };
    auto low = [&](int t) {
      const int p = t + s.lk - s.lq;
      return a.window && p >= a.window ? p - a.window + 1 : 0;
    };
    const int t0 = uni((int)a.by_G(r0)), t1 = uni((int)a.by_G(r0 + rows - 1));  // tokens of the tile
    const int r = min(r0 + l32, nr - 1), t = (int)a.by_G(r), row_lim = lim(t), row_low = low(t);
    const int kend = uni(lim(t1)), kmin = uni(lim(t0)), klow = uni(low(t0)), khigh = uni(low(t1));
    const int sinks = a.window ? min(a.sinks, kend) : 0;
    const bool tokens = t0 != t1;  // more than one: rows that see different keys
    // the units that some row sees: those of the first tokens, then those of the windows
    const int su = (sinks + 31) / 32, wb = max(klow / 32, su), units = su + max((kend + 31) / 32 - wb, 0);
    const int j1 = a.whole ? units : j0 + take, je = min(j1, units);
    auto base = [&](int j) { return (j < su ? j : wb + j - su) * 32; };
    auto wanted = [&](int key) { return key < kend && (key >= klow || key < sinks); };
    // the page of this lane's key of unit j (a unit past the part: none)
    auto look = [&](int j) -> int {
      if (j >= je) return -1;
      const int key = base(j) + l32;
      if (!wanted(key)) return -1;
      if constexpr (KEYS != kRows) return a.table[b * a.ldt + a.by_page(key)];
      return 0;
    };
    const uint16_t* kb = a.k + s.k0 * (int64_t)a.skt + (int64_t)kvh * a.skh;
    const uint16_t* vb = a.v + s.k0 * (int64_t)a.svt + (int64_t)kvh * a.svh;
    // unit j on its way to registers; returns its keys that are there, a bit each
    v4u kr[LPU], vr[LPU];
    auto issue = [&](int j, int entry) __attribute__((always_inline)) -> uint32_t {
      const int first = base(j), key = first + l32;
      const bool ok = KEYS == kRows ? entry >= 0 : (uint32_t)entry < (uint32_t)a.pages;
      const uint32_t there = (uint32_t)__ballot(ok);
      const int row = KEYS == kRows ? key : key - (int)a.by_page(key) * a.page;
      if constexpr (KEYS == kAnyPages) {
#pragma unroll
        for (int i = 0; i < LPU; ++i) {
          const int x = i * RPL + lane / CH, ck = (lane % CH) ^ Lds<DP>::swk(x), cv = (lane % CH) ^ Lds<DP>::swv(x);
          const uint32_t page = (uint32_t)__shfl(entry, x, 64), place = (uint32_t)__shfl(row, x, 64);
          const uint64_t ofk = (uint64_t)page * a.skp + (uint64_t)place * a.skt;
          const uint64_t ofv = (uint64_t)page * a.svp + (uint64_t)place * a.svt;
          const bool in = there >> x & 1;
          kr[i] = *reinterpret_cast<const v4u*>(pick(in && ck * 8 < a.D, kb + ofk + ck * 8));
          vr[i] = *reinterpret_cast<const v4u*>(pick(in && cv * 8 < a.D, vb + ofv + cv * 8));
        }
      } else {
        // rows that share a page are adjacent: one resource each for their keys and values, which ends behind the sequence's last
        // key or, of pages, behind the last of them (a page's other rows are memory of the pool; an entry that names none leaves
        // no bytes)
        constexpr int PG = KEYS == kRows ? 32 : KEYS;
#pragma unroll
        for (int g = 0; g < 32 / PG; ++g) {
          uint64_t ofk, ofv;
          int n;
          if constexpr (KEYS == kRows) {
            ofk = (uint64_t)(uint32_t)first * a.skt, ofv = (uint64_t)(uint32_t)first * a.svt;
            n = there ? min(s.lk - first, 32) : 0;
          } else {
            const uint32_t some = PG == 32 ? there : there >> (g * PG) & ((1u << (PG & 31)) - 1);
            const uint32_t place = (uint32_t)__builtin_amdgcn_readlane(row, g * PG);
            const uint32_t page = (uint32_t)__builtin_amdgcn_readlane(entry, g * PG + (some ? __ffs(some) - 1 : 0));
            ofk = (uint64_t)page * a.skp + (uint64_t)place * a.skt, ofv = (uint64_t)page * a.svp + (uint64_t)place * a.svt;
            n = some ? PG : 0;
          }
          const auto rk = rsrc(kb + ofk, n ? (uint32_t)(n - 1) * a.skt * 2u + a.D * 2 : 0), rv = rsrc(vb + ofv, n ? (uint32_t)(n - 1) * a.svt * 2u + a.D * 2 : 0);
#pragma unroll
          for (int i = 0; i < PG / RPL; ++i) {
            const int x = g * (PG / RPL) + i;
            kr[x] = __builtin_amdgcn_raw_buffer_load_b128(rk, lane_k[x % NK] + (uint32_t)(i * RPL) * a.skt * 2u, 0, 0);
            vr[x] = __builtin_amdgcn_raw_buffer_load_b128(rv, lane_v + (uint32_t)(i * RPL) * a.svt * 2u, 0, 0);
          }
        }
      }
      return there;
    };

    int j = j0 + wave;
    int entry = look(j), ahead = look(j + FW);
    uint32_t there;
    there = issue(j, entry);  // (a unit past the part: no bytes)
    v8bf qf[KST];
    {
      const uint16_t* p = a.q + (s.q0 + t) * a.sqt + (int64_t)(kvh * a.G + r - t * a.G) * a.sqh;
#pragma unroll
      for (int i = 0; i < KST; ++i) {
        const int c = 2 * i + h;
        qf[i] = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u*>(pick(c * 8 < a.D, p + c * 8)));
      }
    }
    v16f O[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) O[d] = v16f{};
    float m = kLow, l = 0.0f;
    bool careful = false;  // some row's maximum is big

    SS_LDS uint8_t *kt = ring, *vt = ring + KB;
    // this lane's places in LDS, computed here, under the first loads (a call of few keys is a chain of latencies, and the
    // instructions themselves, each read once, are among them)
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int ll = ln & 31, hh = ln >> 5;
    const int vrow = 4 * hh + ((ln & 15) >> 2), vcol = ((ln >> 4) & 1) * 2 + ((ln & 3) >> 1), vsub = (ln & 1) * 8;
#pragma unroll 1
    for (; j < je; j += FW) {
#pragma unroll
      for (int i = 0; i < LPU; ++i) {
        *(SS_LDS v4u*)(ring + (i * 64 + lane) * 16) = kr[i];
        *(SS_LDS v4u*)(ring + KB + (i * 64 + lane) * 16) = vr[i];
      }
      if (KEYS != kAnyPages && uni(there) != -1) {  // values of keys that no row sees (their scores are replaced below)
#pragma unroll
        for (int i = 0; i < LPU; ++i)
          if (!(there >> (i * RPL + lane / CH) & 1)) *(SS_LDS v4u*)(ring + KB + (i * 64 + lane) * 16) = v4u{0, 0, 0, 0};
      }
      entry = ahead;
      ahead = look(j + 2 * FW);
      const uint32_t there_next = issue(j + FW, entry);
      v16f S = v16f{};
#pragma unroll
      for (int i = 0; i < KST; ++i) {
        const v8bf kf = *reinterpret_cast<const SS_LDS v8bf*>(kt + ll * DP * 2 + ((2 * i + hh) ^ Lds<DP>::swk(ll)) * 16);
        S = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i], S, 0, 0, 0);
      }
      const int k0 = base(j);
      const bool seen = uni(there) == -1 && k0 + 32 <= kmin && (k0 >= khigh || k0 + 32 <= sinks);  // by every row, whole
      if (!seen) {
        const uint32_t bits = (there & keys_between(row_low - k0, row_lim - k0, sinks - k0)) >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = where_seen(S[i], bits, 8 * (i / 4) + i % 4);
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
      if (tokens && !seen) {  // keys were loaded that some row does not see
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < LPU; ++i) {
          const v4u w = *reinterpret_cast<const SS_LDS v4u*>(vt + (i * 64 + lane) * 16);
          odd |= odd_bf16x2(w[0]) | odd_bf16x2(w[1]) | odd_bf16x2(w[2]) | odd_bf16x2(w[3]);
        }
        if (__builtin_expect(__any(odd != 0), 0)) {
          add_odd_between<DP>(O, vt, row_low - k0, row_lim - k0, sinks - k0, h);
#pragma unroll 1
          for (int i = 0; i < LPU; ++i) {
            SS_LDS v4u* p = (SS_LDS v4u*)(ring + KB + (i * 64 + lane) * 16);
            const v4u w = *p;
            *p = v4u{even_out(w[0]), even_out(w[1]), even_out(w[2]), even_out(w[3])};
          }
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
          const v4s x = read_columns((SS_LDS uint8_t*)(vt + ra * DP * 2 + (c ^ Lds<DP>::swv(ra)) * 16 + vsub));
          const v4s y = read_columns((SS_LDS uint8_t*)(vt + rb * DP * 2 + (c ^ Lds<DP>::swv(rb)) * 16 + vsub));
          const v8bf vf = __builtin_bit_cast(v8bf, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
          O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, P[kk], O[d], 0, 0, 0);
        }
      there = there_next;
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
    const bool cut = !a.whole && take < un;
    const int64_t slot = (int64_t)blockIdx.x * 2 + (first ? 0 : 1);
    if (cut && j0 == 0 && threadIdx.x == 0) {  // the tile begins here: who else has parts of it
      Record& rec = ws.rec[blockIdx.x];
      rec.slot = first ? 0 : 1;
      rec.rows = rows;
      rec.kvh = kvh;
      rec.r0 = r0;
      rec.q0 = s.q0;
      rec.parts = min(1 + (un - take + run - 1) / run, (int)(gridDim.x - blockIdx.x));
    }
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
      const float lg = L == 0.0f ? -INFINITY : M2 + __builtin_amdgcn_logf(L);  // log2 of the row's sum
      if (cut) {
        *reinterpret_cast<float4*>(ws.part + (slot * ws.rows + row) * a.D + c) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (c == 0) ws.lg[slot * FM + row] = lg;
      } else {
        const int rr = r0 + row, tr = (int)a.by_G(rr), head = kvh * a.G + rr - tr * a.G;
        const int64_t tok = s.q0 + tr;
        *reinterpret_cast<uint2*>(a.o + tok * a.sot + head * a.soh + c) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (a.lse && c == 0) a.lse[head * a.Tq + tok] = lg * 0.69314718056f;
      }
    }

    s0 += take;
    if (s0 >= s1) break;
    __syncthreads();  // the rings and sums are free again
    first = false;
    j0 = 0;
    if (++th == tiles * a.Hkv) {
      th = 0;
      do {
        if (++b >= a.B) return;
        s = load_seq<KEYS>(a, b);
        tiles = tiles_of(s.lq, a.G);
      } while (tiles == 0);
      un = a.whole ? 1 : units_of(a.window, a.sinks, a.tokens, s.lq, s.lk);
    }
  }
}

// o = sum_s w_s part_s, w_s = 2^(lg_s - max) / sum of them, for the tile that begins in workgroup blockIdx.x's run and
// ends in a later one: part 0 lies in the record's place, the others in the first places of the workgroups behind it. 16 bytes a
// thread, the parts dealt over groups of threads, in flight together, and added in LDS in a fixed order.
__global__ __launch_bounds__(256) void join_kernel(FlatArgs a, Parts ws) {
  constexpr int kPre = 4;
  __shared__ float4 acc[256];
  const Record rec = ws.rec[blockIdx.x];
  if (rec.parts == 0) return;
  const int lane = threadIdx.x & 63;
  const int quads = a.D / 4, groups = 256 / quads, g = threadIdx.x / quads, c = threadIdx.x % quads;
  auto slot = [&](int s) { return s == 0 ? (int64_t)blockIdx.x * 2 + rec.slot : ((int64_t)blockIdx.x + s) * 2; };
  for (int row = blockIdx.y; row < rec.rows; row += gridDim.y) {
    float lp[kPre];
    float4 xp[kPre];
    auto fetch = [&](int s0) {  // (behind the last part: that one again)
#pragma unroll
      for (int i = 0; i < kPre; ++i) {
        const int64_t at = slot(min(s0 + i * groups, rec.parts - 1));
        lp[i] = ws.lg[at * FM + row];
        xp[i] = *reinterpret_cast<const float4*>(ws.part + (at * ws.rows + row) * a.D + c * 4);
      }
    };
    const float l0 = ws.lg[slot(min(lane, rec.parts - 1)) * FM + row];
    fetch(g);
    float M = l0;
    for (int s = 64 + lane; s < rec.parts; s += 64) M = fmaxf(M, ws.lg[slot(s) * FM + row]);
    M = wave_max(M);
    auto power = [&](float l) { return l == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(l - M); };  // (of a NaN: NaN)
    float sum = lane < rec.parts ? power(l0) : 0.0f;
    for (int s = 64 + lane; s < rec.parts; s += 64) sum += power(ws.lg[slot(s) * FM + row]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    float4 o = make_float4(0, 0, 0, 0);
    if (g < groups) {
      for (int s0 = g; s0 < rec.parts; s0 += kPre * groups) {
        if (s0 != g) fetch(s0);
#pragma unroll
        for (int i = 0; i < kPre; ++i) {
          if (s0 + i * groups >= rec.parts) break;
          const float w = power(lp[i]) * inv;
          o.x += w * xp[i].x; o.y += w * xp[i].y; o.z += w * xp[i].z; o.w += w * xp[i].w;
        }
      }
    }
    acc[threadIdx.x] = o;
    __syncthreads();
    const int rr = rec.r0 + row, tr = (int)a.by_G(rr), head = rec.kvh * a.G + rr - tr * a.G;
    const int64_t tok = rec.q0 + tr;
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
    __syncthreads();
  }
}

// Workgroups of a call, and whether it leaves its tiles whole (then no workspace and one launch): rows over so few keys that
// a workgroup's least run holds them (or so many rows and keys that their units may pass 31 bits). The lengths are not known
// here: the rules go by the room for keys, the mean of the sequences' (contiguous keys: one of them may have `most` of them, all
// there are, and all the rows). By the mean alone one sequence of 100000 keys among 1023 of 8 was walked by a workgroup a
// tile (32 heads of 128 over 8, one token each: 3360 us, cut 223; one of 8000 among 80: 140 / 27, of 4000 among 40: 72 / 23);
// cut whenever one could be long, short ones pay for the join (64 of 60 keys 7.4 us whole, 12.0 cut; of 1 to 128 keys 8.6 / 25;
// 64 of 128 10.1 / 12.9, 256 of 60 28.2 / 22.8). So tiles stay whole while none can have more than kMostWhole units.
struct Plan {
  int64_t wgs;
  bool whole;
  int rows;
};
inline Plan plan(int64_t Tq, int64_t room, int64_t most, int64_t B, int64_t G, int64_t Hkv, int64_t D, int64_t window, int64_t sinks) {
  auto of = [&](int64_t keys) -> int64_t {
    return units_of((int)window, (int)sinks, tokens_of((int)G), (int)Tq, (int)std::min<int64_t>(keys, 0x7FFFFF00));
  };
  const int64_t units = of(room);
  const int64_t tiles = (Tq * G / FM + std::min(B, Tq)) * Hkv, fits = 4 * (int64_t)num_cus_p();
  const bool whole = (units <= kMinUnits && of(most) <= kMostWhole) || (double)tiles * of(most) >= 0x7FFF0000;
  const int64_t wgs = whole ? std::min<int64_t>(tiles, 4 * fits)
                            : std::min<int64_t>(fits, (int64_t)std::min<double>((double)tiles * units / kMinUnits + 1, 1e9));
  return {std::max<int64_t>(wgs, 1), whole, (int)std::min<int64_t>(FM, Tq * G)};
}

template <int DP, int KEYS> hipError_t launch(FlatArgs a, int64_t room, int64_t most, void* ws, hipStream_t st) {
  const Plan p = plan(a.Tq, room, most, a.B, a.G, a.Hkv, a.D, a.window, a.sinks);
  constexpr int lds = lds_bytes(DP);
  const hipError_t e = lds_limit((const void*)flat_kernel<DP, KEYS>, lds);
  if (e != hipSuccess) return e;
  a.whole = p.whole;
  a.tokens = tokens_of(a.G);
  a.by_G = FastDiv((uint32_t)a.G), a.by_Hkv = FastDiv((uint32_t)a.Hkv), a.by_wgs = FastDiv((uint32_t)p.wgs);
  a.by_page = FastDiv((uint32_t)std::max(a.page, 1));
  const Parts parts = parts_of(ws, p.wgs, p.rows);
  hipLaunchKernelGGL((flat_kernel<DP, KEYS>), dim3((unsigned)p.wgs), dim3(64 * FW), lds, st, a, parts);
  if (const hipError_t f = hipGetLastError(); f != hipSuccess || p.whole) return f;
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)p.wgs, (unsigned)std::min(p.rows, kJoin)), dim3(256), 0, st, a, parts);
  return hipGetLastError();
}

}  // namespace flat

int64_t flat_workspace_bytes(int64_t Tq, int64_t room, int64_t most, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t window,
                             int64_t sinks) {
  const flat::Plan p = flat::plan(Tq, room, most, B, Hq / Hkv, Hkv, D, window, sinks);
  return p.whole ? 0 : p.wgs * ((int64_t)sizeof(flat::Record) + 2 * flat::FM * 4 + 2 * p.rows * D * 4);
}

bool flat_fits(int64_t Tq, int64_t B, int64_t Hq, int64_t Hkv) {
  return (double)(Tq * (Hq / Hkv) / flat::FM + std::min(B, Tq)) * Hkv < 0x7FFF0000;
}

hipError_t launch_flat(const FlatArgs& a, int64_t room, int64_t most, void* ws, hipStream_t st) {
  auto go = [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    if (!a.paged) return flat::launch<DP, flat::kRows>(a, room, most, ws, st);
    if (a.page % 32 == 0) return flat::launch<DP, 32>(a, room, most, ws, st);
    if (a.page % 16 == 0) return flat::launch<DP, 16>(a, room, most, ws, st);
    return a.page % 8 == 0 ? flat::launch<DP, 8>(a, room, most, ws, st) : flat::launch<DP, flat::kAnyPages>(a, room, most, ws, st);
  };
  return a.D <= 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace ss
