// New tokens into a paged cache (gfx950): rotary positions on their queries and keys, and keys and values to their places,
// page table[sequence][pos / page], row pos % page, in one pass (the angle: k_rotary.hip).
//
// Bound: HBM, every value is read and written once; for a few tokens the launch. Threads are laid out as in the rotary kernel: a
// thread computes the angles of one chunk of pairs once and applies them to several heads of its token, query heads
// first, then key heads, then value heads (which are copied). The places of a workgroup's tokens are looked up once, into LDS.
// Measured: 8192 tokens of 9 prompts, 28 query and 4 key heads of 128: 31 us, 4.8 TB/s; 4 tokens, 32 and 8 heads: 3.8 us.
#include <algorithm>

#include "ss_rotary.h"

namespace ss {
namespace paged {

using rotary::Turn;
using rotary::v4u;
constexpr int kNoPlace = -1, kNoSequence = -2;

// Page and row of a token's place. Tokens of no sequence have kNoSequence; a place outside the table, or an entry that names no
// page, gives kNoPlace: whatever pos, cu and table hold, no access leaves the cache.
__device__ __forceinline__ int2 place_of(const StoreArgs& a, int64_t tok) {
  int64_t b = tok;  // without bounds: one token a sequence
  if (a.cu) {
    if (tok < a.cu[0] || tok >= a.cu[a.B]) return make_int2(kNoSequence, 0);
    int64_t lo = 0, hi = a.B;  // cu[lo] <= tok < cu[hi]
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (a.cu[mid] <= tok) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  const int pos = a.pos[tok];
  const int i = pos / a.page;
  if (pos < 0 || i >= a.cols) return make_int2(kNoPlace, 0);
  const int entry = a.table[b * a.ldt + i];
  return make_int2(entry >= 0 && entry < a.pages ? entry : kNoPlace, pos - i * a.page);
}

struct Head {
  const uint16_t* from;
  uint16_t* to;  // NULL: not stored
  bool turned;
};
__device__ __forceinline__ Head head_of(const StoreArgs& a, int64_t tok, int hd, const int2& at) {
  if (hd < a.Hq) return {a.q + tok * a.sqt + hd * a.sqh, a.qo + tok * a.sot + hd * a.soh, true};
  hd -= a.Hq;
  if (hd < a.Hkv)
    return {a.k + tok * a.skt + hd * a.skh, at.x < 0 ? nullptr : a.kc + at.x * a.kp + at.y * a.kt + hd * a.kh, true};
  hd -= a.Hkv;
  return {a.v + tok * a.svt + hd * a.svh, at.x < 0 ? nullptr : a.vc + at.x * a.vp + at.y * a.vt + hd * a.vh, false};
}

// Items (token, head group, chunk), the chunk fastest. VEC: a chunk is one 16-byte vector of first halves and one of second
// halves (HALF), or one of adjacent pairs, and from `pairs` on one vector of the values behind rot; else one pair or one value.
constexpr int NB = 4;
template <bool HALF, bool VEC> __global__ __launch_bounds__(256) void store_kernel(StoreArgs a, int pairs, int chunks, int groups) {
  constexpr int N = VEC ? 8 : 1, NP = VEC && !HALF ? 4 : N;
  __shared__ int2 place[258];  // a workgroup's items belong to 256 / per + 2 tokens at most
  const int per = groups * chunks, heads = a.Hq + 2 * a.Hkv;
  const int64_t first = (int64_t)blockIdx.x * 256, items = a.T * per, t0 = first / per;  // (tokens of this launch)
  if (a.cu) {
    const int tokens = (int)(min(first + 255, items - 1) / per - t0) + 1;
    for (int i = threadIdx.x; i < tokens; i += 256) place[i] = place_of(a, a.first + t0 + i);
    __syncthreads();
  }
  const int64_t it = first + threadIdx.x;
  if (it >= items) return;
  const int64_t in = it / per, tok = a.first + in;
  const int rest = (int)(it - in * per), hg = rest / chunks, ch = rest - hg * chunks;
  // (without a search for the sequence every thread looks its token's place up, under the loads of the values)
  const int2 at = a.cu ? place[in - t0] : place_of(a, tok);
  if (at.x == kNoSequence) return;
  const bool pair = ch < pairs;
  const int second = !pair ? 0 : HALF ? a.rot / 2 : VEC ? 0 : 1;  // from a chunk's first part to its second; 0: one part
  const int col = !pair ? a.rot + (ch - pairs) * N : HALF || VEC ? ch * N : 2 * ch;
  Turn t[NP];
  if (pair) {
    const int32_t p = a.pos[tok];
#pragma unroll
    for (int i = 0; i < NP; ++i) t[i] = rotary::turn(p, a.steps[ch * NP + i], a.mscale, a.mscale);
  }
  for (int h0 = hg; h0 < heads; h0 += NB * groups) {
    if constexpr (VEC) {
      v4u x[NB], y[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int hd = h0 + j * groups;
        if (hd >= heads) break;
        const uint16_t* p = head_of(a, tok, hd, at).from + col;
        x[j] = *reinterpret_cast<const v4u*>(p);
        if (second) y[j] = *reinterpret_cast<const v4u*>(p + second);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int hd = h0 + j * groups;
        if (hd >= heads) break;
        const Head h = head_of(a, tok, hd, at);
        if (!h.to) continue;
        if (pair && h.turned) {
          float f[8], g[8];
          rotary::Vec<uint16_t>::get(x[j], f);
          if constexpr (HALF) {
            rotary::Vec<uint16_t>::get(y[j], g);
#pragma unroll
            for (int i = 0; i < NP; ++i) rotary::apply(f[i], g[i], t[i]);
            y[j] = rotary::Vec<uint16_t>::put(g);
          } else {
#pragma unroll
            for (int i = 0; i < NP; ++i) rotary::apply(f[2 * i], f[2 * i + 1], t[i]);
          }
          x[j] = rotary::Vec<uint16_t>::put(f);
        }
        *reinterpret_cast<v4u*>(h.to + col) = x[j];
        if (second) *reinterpret_cast<v4u*>(h.to + col + second) = y[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int hd = h0 + j * groups;
        if (hd >= heads) break;
        const Head h = head_of(a, tok, hd, at);
        if (!h.to) continue;
        uint16_t x = h.from[col], y = h.from[col + second];
        if (pair && h.turned) {
          float f = bf16_to_f32(x), g = bf16_to_f32(y);
          rotary::apply(f, g, t[0]);
          x = (uint16_t)pack_bf16x2(f, 0.0f);
          y = (uint16_t)pack_bf16x2(g, 0.0f);
        }
        h.to[col] = x;
        if (second) h.to[col + second] = y;
      }
    }
  }
}

}  // namespace paged

hipError_t launch_paged_store(const StoreArgs& a, hipStream_t st) {
  auto vec = [](const void* p, int64_t s0, int64_t s1) { return ((uintptr_t)p & 15) == 0 && s0 % 8 == 0 && s1 % 8 == 0; };
  const int np = a.half ? 8 : 4;
  const bool v = a.rot / 2 % np == 0 && (a.D - a.rot) % 8 == 0 && vec(a.k, a.skt, a.skh) && vec(a.v, a.svt, a.svh) &&
                 (a.Hq == 0 || (vec(a.q, a.sqt, a.sqh) && vec(a.qo, a.sot, a.soh)));
  const int pairs = v ? a.rot / 2 / np : a.rot / 2, chunks = pairs + (a.D - a.rot) / (v ? 8 : 1);
  const int heads = a.Hq + 2 * a.Hkv;
  // heads per thread: as many as leave the chip 8 waves per SIMD or so (more heads share one angle), else one
  const int64_t full = (int64_t)num_cus_p() * 2048;
  const int per = (int)std::max<int64_t>(1, std::min<int64_t>(2 * paged::NB, a.T * heads * chunks / full));
  const int groups = (heads + per - 1) / per;
  // launches of fewer than 2^32 threads: many tokens go in several
  const int64_t most = std::max<int64_t>(1, (int64_t)0x7FFFFF00 / ((int64_t)groups * chunks));
  for (int64_t t = 0; t < a.T; t += most) {
    StoreArgs b = a;
    b.first = t;
    b.T = std::min(most, a.T - t);
    const dim3 grid((unsigned)((b.T * groups * chunks + 255) / 256));
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, b, pairs, chunks, groups); };
    if (v && a.half) go(paged::store_kernel<true, true>);
    else if (v) go(paged::store_kernel<false, true>);
    else if (a.half) go(paged::store_kernel<true, false>);
    else go(paged::store_kernel<false, false>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace ss
