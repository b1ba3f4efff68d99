// Rotary positions (gfx950): each pair (a, b) of a head's first rot_dim values is turned by the angle of its
// token, u = a cos t - b sin t, v = b cos t + a sin t, t = pos * f(pair); cos and sin carry the factor mscale,
// the inverse turns by -t.
//
// Angle. pos * f in float32 is off by pos * f * 2^-24 radians, which at position 10^6 is a visible angle. Here
// a pair's frequency is a 64-bit fraction of a turn per position, step = round(f / 2 pi * 2^64), so
// pos * step modulo 2^64 is the token's place within the turn, exact to pos * 2^-65 turns at any 32-bit
// position (one wrapping integer multiply), and whole turns drop out by themselves. The nearest quarter turn is taken
// out in integers too, and the 32 bits below it go to sin and cos of pi x as a float: it rounds by 2^-28 turns at most, and
// next to every zero of sin and cos by 2^-24 of the distance from it.
//
// Bound: every value is read and written once (HBM). No cos/sin table is read: a thread computes the angles
// of its pairs once and applies them to several heads of the token; it loads a batch of heads before it
// stores the first, so that several loads are in flight also where the output is the input.
// Measured: 16384 tokens, 40 heads of 128, bf16: 67 us, 5.0 TB/s (a large copy: 4.9); 777 tokens, 14 heads of 80 of which
// 32 turn, float32: 4.1 us; one token, 40 heads: 2.5 us, which is what a launch takes. Sizes that vectors do not divide go by
// elements of 2 or 4 bytes: 2000 tokens, 40 heads of 100 of which 74 turn, bf16: 15.4 us, 2.1 TB/s.
#include <algorithm>

#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {
namespace rotary {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

struct Turn {
  float c, s;
};
__device__ __forceinline__ Turn turn(int32_t pos, uint64_t step, float cscale, float sscale) {
  const uint64_t phase = (uint64_t)(int64_t)pos * step;
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);        // the nearest
  const float f = (float)(int32_t)(uint32_t)(phase >> 30) * 0x1p-33f;       // half turns from it, [-1/4, 1/4]
  // sin(pi f) = f (pi + f^2 p(f^2)), pi in two floats, and cos(pi f) = 1 + f^2 q(f^2): polynomials fitted to the least relative
  // error on [-1/4, 1/4] (4e-9 and 5e-11), both within 1.4 x 2^-24 of the value as evaluated.
  const float u = f * f;
  float p = __builtin_fmaf(-0.589418776f, u, 2.54980521f);
  p = __builtin_fmaf(p, u, -5.16770904f);
  p = __builtin_fmaf(p, u, -8.74227801e-8f);
  const float s = __builtin_fmaf(f, 3.14159274f, f * p);
  float q = __builtin_fmaf(0.231429548f, u, -1.33505846f);
  q = __builtin_fmaf(q, u, 4.0587079f);
  q = __builtin_fmaf(q, u, -4.93480217f);
  const float c = __builtin_fmaf(q, u, 1.0f);
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  return {((quarter + 1) & 2 ? -x : x) * cscale, (quarter & 2 ? -y : y) * sscale};
}
__device__ __forceinline__ void apply(float& a, float& b, const Turn& t) {
  const float u = __builtin_fmaf(a, t.c, -(b * t.s));
  b = __builtin_fmaf(b, t.c, a * t.s);
  a = u;
}

// 16 bytes of a row as floats and back
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void get(const v4u& x, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(x[i]);
  }
  __device__ static v4u put(const float* f) {
    return v4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};
template <> struct Vec<uint16_t> {
  static constexpr int N = 8;
  __device__ static void get(const v4u& x, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(x[i] << 16);
      f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
    }
  }
  __device__ static v4u put(const float* f) {
    return v4u{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  }
};

// Items (token, head group, chunk), the chunk fastest: a thread turns one chunk of pairs of the heads hg,
// hg + groups, .. of its token, so the lanes of a wave cover whole heads side by side. A chunk is one 16-byte
// vector of first halves and one of second halves (HALF), or one 16-byte vector of adjacent pairs; the chunks
// from `pairs` on are the values behind rot_dim, copied (only when the output is another buffer).
template <typename T, bool HALF, int NB>
__global__ __launch_bounds__(256) void vec_kernel(RotaryArgs a, int pairs, int chunks, int groups) {
  constexpr int N = Vec<T>::N, NP = HALF ? N : N / 2;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  const int per = groups * chunks;
  const int64_t items = a.T * per;
  for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
    const int64_t tok = items <= 0x7FFFFFFF ? (int64_t)((uint32_t)it / (uint32_t)per) : it / per;
    const int rest = (int)(it - tok * per), hg = rest / chunks, ch = rest - hg * chunks;
    const T* xt = x + tok * a.sxt;
    T* yt = y + tok * a.syt;
    if (ch >= pairs) {  // behind rot_dim
      const int col = a.rot + (ch - pairs) * N;
      for (int hd = hg; hd < a.H; hd += groups)
        *reinterpret_cast<v4u*>(yt + hd * a.syh + col) = *reinterpret_cast<const v4u*>(xt + hd * a.sxh + col);
      continue;
    }
    const int32_t p = a.pos[tok];
    const int col = ch * N, off = a.rot / 2;
    Turn t[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) t[i] = turn(p, a.steps[ch * NP + i], a.cscale, a.sscale);
    for (int h0 = hg; h0 < a.H; h0 += NB * groups) {
      v4u va[NB], vb[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int hd = h0 + j * groups;
        if (hd < a.H) {
          va[j] = *reinterpret_cast<const v4u*>(xt + hd * a.sxh + col);
          if constexpr (HALF) vb[j] = *reinterpret_cast<const v4u*>(xt + hd * a.sxh + col + off);
        }
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int hd = h0 + j * groups;
        if (hd >= a.H) break;
        float f[N], g[N];
        Vec<T>::get(va[j], f);
        if constexpr (HALF) {
          Vec<T>::get(vb[j], g);
#pragma unroll
          for (int i = 0; i < N; ++i) apply(f[i], g[i], t[i]);
          *reinterpret_cast<v4u*>(yt + hd * a.syh + col + off) = Vec<T>::put(g);
        } else {
#pragma unroll
          for (int i = 0; i < NP; ++i) apply(f[2 * i], f[2 * i + 1], t[i]);
        }
        *reinterpret_cast<v4u*>(yt + hd * a.syh + col) = Vec<T>::put(f);
      }
    }
  }
}

// Sizes, strides or pointers that 16-byte vectors do not divide: one pair (or one copied value) per item.
template <typename T> __device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(*p);
  else return *p;
}
template <typename T> __device__ __forceinline__ void store1(T* p, float f) {
  if constexpr (sizeof(T) == 2) *p = (uint16_t)pack_bf16x2(f, 0.0f);
  else *p = f;
}
template <typename T>
__global__ __launch_bounds__(256) void pair_kernel(RotaryArgs a, int pairs, int chunks, int groups) {
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  const int per = groups * chunks;
  const int64_t items = a.T * per;
  for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
    const int64_t tok = it / per;
    const int rest = (int)(it - tok * per), hg = rest / chunks, ch = rest - hg * chunks;
    const T* xt = x + tok * a.sxt;
    T* yt = y + tok * a.syt;
    if (ch >= pairs) {
      const int col = a.rot + ch - pairs;
      for (int hd = hg; hd < a.H; hd += groups) yt[hd * a.syh + col] = xt[hd * a.sxh + col];
      continue;
    }
    const Turn t = turn(a.pos[tok], a.steps[ch], a.cscale, a.sscale);
    const int ca = a.half ? ch : 2 * ch, cb = a.half ? ch + a.rot / 2 : 2 * ch + 1;
    for (int hd = hg; hd < a.H; hd += groups) {
      float u = load1(xt + hd * a.sxh + ca), v = load1(xt + hd * a.sxh + cb);
      apply(u, v, t);
      store1(yt + hd * a.syh + ca, u);
      store1(yt + hd * a.syh + cb, v);
    }
  }
}

constexpr int NB = 4;

template <typename T> hipError_t launch(const RotaryArgs& a, hipStream_t st) {
  constexpr int N = Vec<T>::N;
  const int np = a.half ? N : N / 2, half = a.rot / 2;
  auto vec = [&](const void* p, int64_t s0, int64_t s1) {
    return ((uintptr_t)p & 15) == 0 && s0 % N == 0 && s1 % N == 0;
  };
  const bool v = half % np == 0 && (a.D - a.rot) % N == 0 && vec(a.x, a.sxt, a.sxh) && vec(a.y, a.syt, a.syh);
  const int pairs = v ? half / np : half;
  const int chunks = pairs + (a.x == a.y ? 0 : (a.D - a.rot) / (v ? N : 1));
  // heads per thread: as many as leave the chip 8 waves per SIMD or so (more heads share one angle), else one
  const int64_t full = (int64_t)num_cus_p() * 2048;
  const int per = (int)std::max<int64_t>(1, std::min<int64_t>(2 * NB, a.T * a.H * chunks / full));
  const int groups = (a.H + per - 1) / per;
  const int64_t blocks = (a.T * groups * chunks + 255) / 256;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 22));
  if (!v) hipLaunchKernelGGL((pair_kernel<T>), grid, dim3(256), 0, st, a, pairs, chunks, groups);
  else if (a.half) hipLaunchKernelGGL((vec_kernel<T, true, NB>), grid, dim3(256), 0, st, a, pairs, chunks, groups);
  else hipLaunchKernelGGL((vec_kernel<T, false, NB>), grid, dim3(256), 0, st, a, pairs, chunks, groups);
  return hipGetLastError();
}

}  // namespace rotary

hipError_t launch_rotary(bool bf16, const RotaryArgs& a, hipStream_t st) {
  return bf16 ? rotary::launch<uint16_t>(a, st) : rotary::launch<float>(a, st);
}

}  // namespace ss
