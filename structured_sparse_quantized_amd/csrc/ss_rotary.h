// The turn of a pair of values by its token's angle, and 16-byte vectors of a row (internal to the library; the mathematics
// stands in k_rotary.hip).
#pragma once
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

}  // namespace rotary
}  // namespace ss
