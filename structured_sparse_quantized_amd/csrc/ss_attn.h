// Device helpers shared by the attention kernels (internal to the library): types of the matrix instructions, buffer
// resources, the lane exchange of a row's two halves, the layout of key and value tiles in LDS, and what keeps infinities and
// NaN of unseen values out of a row.
#pragma once
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
// The same under a window: `vt`: 32 rows of values in LDS; row r of the lane sees those below hi that are not below lo, and those below sk
template <int DP> __device__ __forceinline__ void add_odd_between(v16f* O, const SS_LDS uint8_t* vt, int lo, int hi, int sk, int h) {
  asm volatile("" : "+v"(h), "+v"(hi), "+v"(lo));  // (nothing of this is kept in registers beside the loop that calls it)
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
          if (k < hi && (k >= lo || k < sk) && !__builtin_isfinite(v)) O[d][4 * g + e] += v;
        }
      }
}

// The keys of a unit of 32 that a row sees, a bit each: those below hi that are not below lo, and those below sk; and a score, or
// -infinity where its key's bit is not set (two instructions: the bit over a word, and a choice of bits).
__device__ __forceinline__ uint32_t keys_below(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1; }
__device__ __forceinline__ uint32_t keys_between(int lo, int hi, int sk) { return keys_below(hi) & (~keys_below(lo) | keys_below(sk)); }
__device__ __forceinline__ float where_seen(float score, uint32_t bits, int key) {
  const uint32_t m = (uint32_t)__builtin_amdgcn_sbfe((int)bits, key, 1);
  return __uint_as_float((m & __float_as_uint(score)) | (~m & 0xFF800000u));
}

}  // namespace attn
}  // namespace ss
