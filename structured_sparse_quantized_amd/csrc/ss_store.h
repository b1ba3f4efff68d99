// Epilogue store shared by the product kernels (internal to the library).
#pragma once
#include <type_traits>

#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {

// Store one lane's 4 results: rows ar..ar+3 of the sparse operand, one dense row bc.
template <int YT, bool SIDE_X>
__device__ __forceinline__ void store_out(void* Y, int64_t ldy, int64_t ar, int64_t bc, int64_t R, const float* y,
                                          const int32_t* yi) {
  if (!SIDE_X && (ldy & 3) == 0 && ar + 3 < R) {  // Y[bc][ar .. ar+3] is one aligned vector
    if constexpr (YT == 0) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(Y) + bc * ldy + ar) =
          make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    } else if constexpr (YT == 1) {
      *reinterpret_cast<float4*>(static_cast<float*>(Y) + bc * ldy + ar) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
      *reinterpret_cast<int4*>(static_cast<int32_t*>(Y) + bc * ldy + ar) = make_int4(yi[0], yi[1], yi[2], yi[3]);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (ar + q >= R) break;
    const int64_t off = SIDE_X ? (ar + q) * ldy + bc : bc * ldy + ar + q;
    if constexpr (YT == 0) static_cast<uint16_t*>(Y)[off] = f32_to_bf16(y[q]);
    else if constexpr (YT == 1) static_cast<float*>(Y)[off] = y[q];
    else static_cast<int32_t*>(Y)[off] = yi[q];
  }
}

// ---- the general epilogue (YT == 3) ---------------------------------------------
// The kernels take an Epilogue where YT is 3 and nothing otherwise.
struct NoEpilogue {};
template <int YT> using EpilogueOf = typename std::conditional<YT == 3, Epilogue, NoEpilogue>::type;

// The activations in float32. 1 / (1 + exp(-z)) takes the chip's power and reciprocal instructions where the
// result is rounded to bf16 (their error and that of the exponent, |z| 2^-23, vanish in its 2^-8), the exact
// functions for float32 results. tanh(u) enters as 2 / (1 + exp(-2u)) - 1, which makes the tanh form of GELU
// z / (1 + exp(-2u)).
__device__ __forceinline__ float over_1p_exp(float num, float z, bool f32) {  // num / (1 + exp(-z))
  if (f32) return num / (1.0f + expf(-z));
  return num * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * z));
}
// erfc(a), a >= 0, for results rounded to bf16, with the chip's reciprocal and power: e^(-a^2) times a polynomial in
// t = 1 / (1 + a / 2) without a constant term, fitted so that neither 10^7 times the absolute error nor 10^5 times the
// relative one passes 0.8 up to a = 9.4, where the power ends; evaluated in float32: 3.4e-7 and 1.2e-5 (7e-7 with the
// chip's instructions a unit off). Relative too, because GELU's negative tail is z/2 erfc itself, where 1 + erf cancels.
__device__ __forceinline__ float erfc_short(float a) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, a, 1.0f));
  float p = __builtin_fmaf(0.087252283f, t, -0.350759044f);
  p = __builtin_fmaf(p, t, 0.376597889f);
  p = __builtin_fmaf(p, t, 0.0502277593f);
  p = __builtin_fmaf(p, t, 0.275517803f);
  p = __builtin_fmaf(p, t, 0.278945086f);
  p = __builtin_fmaf(p, t, 0.282218303f);
  return p * t * __builtin_amdgcn_exp2f(-1.44269504088896340736f * a * a);
}
// SHORT: for bf16 results only (f32 is false).
template <int N, bool SHORT = false> __device__ __forceinline__ void activate_n(float* z, int act, bool f32) {
  if constexpr (SHORT) f32 = false;
  if (act == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];  // (a NaN stays)
  } else if (act == 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = z[i] * -0.70710678118654752440f;
      if (f32) {
        z[i] = 0.5f * z[i] * erfcf(x);
      } else {
        const float q = erfc_short(fabsf(x));
        z[i] = 0.5f * z[i] * (z[i] < 0.0f ? q : 2.0f - q);
      }
    }
  } else if (act == 3) {  // the tanh form: u = sqrt(8 / pi) (z + 0.044715 z^3)
#pragma unroll
    for (int i = 0; i < N; ++i)
      z[i] = over_1p_exp(z[i], 1.59576912160573071176f * __builtin_fmaf(0.044715f * z[i] * z[i], z[i], z[i]), f32);
  } else if (act == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = over_1p_exp(z[i], z[i], f32);
  }
}
__device__ __forceinline__ float load_res(const Epilogue& e, int64_t at) {
  return e.f32 ? static_cast<const float*>(e.res)[at] : bf16_to_f32(static_cast<const uint16_t*>(e.res)[at]);
}
__device__ __forceinline__ void store_one(void* Y, int64_t at, float v, bool f32) {
  if (f32) static_cast<float*>(Y)[at] = v;
  else static_cast<uint16_t*>(Y)[at] = (uint16_t)pack_bf16x2(v, 0.0f);
}
// The few-token kernels (weight-sparse side): a lane's 4 results are channels ar .. ar+3 of token bc. Their residuals (of the
// 4 columns, or with a gate the 2, clamped into the row) are loaded under the product, long before the stores: the
// residual may be Y, so no load could move over one.
__device__ __forceinline__ void load_residual(float* r, int64_t ar, int64_t bc, int64_t R, const Epilogue& e) {
  if (!e.res) return;
  const int n = e.gated ? 2 : 4;
  const int64_t col = e.gated ? ar >> 1 : ar, cols = e.gated ? R >> 1 : R;
  if (n == 4 && !e.f32 && (e.ldr & 3) == 0 && col + 4 <= cols) {
    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(e.res) + bc * e.ldr + col);
    r[0] = __uint_as_float(x.x << 16);
    r[1] = __uint_as_float(x.x & 0xFFFF0000u);
    r[2] = __uint_as_float(x.y << 16);
    r[3] = __uint_as_float(x.y & 0xFFFF0000u);
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q < n) r[q] = load_res(e, bc * e.ldr + min(col + q, cols - 1));
}
// The finished values (gated: y[0], y[1]) plus their residuals, stored.
__device__ __forceinline__ void store_epilogue(void* Y, int64_t ldy, int64_t ar, int64_t bc, int64_t R, float* y,
                                               const float* r, const Epilogue& e) {
  if (e.res) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < 2 || !e.gated) y[q] += r[q];
  }
  const int n = e.gated ? 2 : 4;
  const int64_t col = e.gated ? ar >> 1 : ar, cols = e.gated ? R >> 1 : R;
  if (n == 4 && !e.f32 && (ldy & 3) == 0 && col + 4 <= cols) {  // 8-byte vectors
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(Y) + bc * ldy + col) =
        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q >= n || col + q >= cols) break;
    store_one(Y, bc * ldy + col + q, y[q], e.f32);
  }
}

// Their epilogue, of the scaled sums.
__device__ __forceinline__ void finish_and_store(void* Y, int64_t ldy, int64_t ar, int64_t bc, int64_t R, float* y,
                                                 const float* r, const Epilogue& e) {
  if (e.bias) {
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] += e.bias[min(ar + q, R - 1)];
  }
  if (e.gated) {
    float g[2] = {y[0], y[2]};
    activate_n<2>(g, e.act, e.f32);
    y[0] = g[0] * y[1];
    y[1] = g[1] * y[3];
  } else {
    activate_n<4>(y, e.act, e.f32);
  }
  store_epilogue(Y, ldy, ar, bc, R, y, r, e);
}

// Whether rows of Y and of the residual start on 16 bytes (their pointers do).
__device__ __forceinline__ bool aligned_rows(const Epilogue& e, int64_t ldy) {
  const int per16 = e.f32 ? 3 : 7;  // elements of 16 bytes, less one
  return (ldy & per16) == 0 && (!e.res || (e.ldr & per16) == 0);
}

// Eight columns of one row of Y from a staged row of scaled sums (channels ch0, ch0 + 1, ..; nch of them in all):
// piece i holds 8 channels, or with a gate the 16 channels of 8 pairs.
struct Leave {
  typedef float v4fl __attribute__((ext_vector_type(4)));
  typedef uint32_t v4ul __attribute__((ext_vector_type(4)));
  struct Res {
    v4ul a, b;  // 8 bf16 in a, or 8 f32
  };
  const Epilogue& e;
  void* Y;
  int64_t ldy;
  int piece, first, nch, col, ncol;
  bool vec;        // this lane's piece is whole
  float bias[16];  // of this lane's piece

  __device__ __forceinline__ Leave(const Epilogue& ep, void* y, int64_t ld, int pc, int ch0, int nc)
      : e(ep), Y(y), ldy(ld), piece(pc), nch(nc) {
    first = ch0 + (piece << (3 + e.gated));
    col = (ch0 >> e.gated) + piece * 8;
    ncol = nch >> e.gated;
    vec = col + 8 <= ncol;
#pragma unroll
    for (int i = 0; i < 16; ++i) bias[i] = e.bias && (i < 8 || e.gated) ? e.bias[min(first + i, nch - 1)] : 0.0f;
  }
  __device__ __forceinline__ void residual(Res& r, int64_t tok) const {
    if (!e.res || !vec) return;
    if (e.f32) {
      const v4ul* p = reinterpret_cast<const v4ul*>(static_cast<const float*>(e.res) + tok * e.ldr + col);
      r.a = p[0];
      r.b = p[1];
    } else {
      r.a = *reinterpret_cast<const v4ul*>(static_cast<const uint16_t*>(e.res) + tok * e.ldr + col);
    }
  }
  __device__ __forceinline__ void row(const float* staged, const Res& r, int64_t tok) const {
    if (first >= nch) return;
    float f[16], g[8];
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      if (i >= 8 && !e.gated) break;
      const float4 x = *reinterpret_cast<const float4*>(staged + (piece << (3 + e.gated)) + i);
      f[i] = x.x, f[i + 1] = x.y, f[i + 2] = x.z, f[i + 3] = x.w;
    }
    if (e.bias) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < 8 || e.gated) f[i] = f[i] + bias[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = e.gated ? f[2 * i] : f[i];
    activate_n<8>(g, e.act, e.f32);
    if (e.gated) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= f[2 * i + 1];
    }
    if (vec && e.f32) {
      if (e.res) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] += __uint_as_float(r.a[i]);
          g[4 + i] += __uint_as_float(r.b[i]);
        }
      }
      v4fl* d = reinterpret_cast<v4fl*>(static_cast<float*>(Y) + tok * ldy + col);
      __builtin_nontemporal_store(v4fl{g[0], g[1], g[2], g[3]}, d);
      __builtin_nontemporal_store(v4fl{g[4], g[5], g[6], g[7]}, d + 1);
    } else if (vec) {
      if (e.res) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[2 * i] += __uint_as_float(r.a[i] << 16);
          g[2 * i + 1] += __uint_as_float(r.a[i] & 0xFFFF0000u);
        }
      }
      const v4ul v{pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7])};
      __builtin_nontemporal_store(v, reinterpret_cast<v4ul*>(static_cast<uint16_t*>(Y) + tok * ldy + col));
    } else {
      int c = col;
      asm volatile("" : "+v"(c));  // addresses made here, not kept for the whole tile
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i >= ncol) break;
        store_one(Y, tok * ldy + c + i, e.res ? g[i] + load_res(e, tok * e.ldr + c + i) : g[i], e.f32);
      }
    }
  }
};

// The same for rows that do not start on 16 bytes: a lane per column, so that a wave's loads and stores are runs of
// adjacent elements, and narrow rows side by side over the 64 lanes; 4 rows a lane at a time, the residuals of the next 4
// on their way while these are finished. (Pieces of 16 bytes from where each row first meets one measured 20-50% slower:
// every wave has ends of rows, which go by elements, in every step.) COLS staged channels a row, a power of two.
template <int COLS>
__device__ __forceinline__ void leave_columns(const float* stg, int ld, int rows, int64_t tok0, int64_t ntok, int ch0, int nch,
                                              void* Y, int64_t ldy, const Epilogue& e) {
  const int lane = threadIdx.x & 63, wide = COLS >> e.gated, col0 = ch0 >> e.gated, ncol = nch >> e.gated;
  const int have = (int)min((int64_t)rows, ntok - tok0);  // rows of Y
  const int beside = wide < 64 ? 64 / wide : 1, first = lane / wide;  // rows next to each other, and this lane's first
  const int es = e.f32 ? 4 : 2, shift = e.f32 ? 0 : 16;
#pragma unroll 1
  for (int c = lane & (min(wide, 64) - 1); c < wide; c += 64) {
    if (col0 + c >= ncol) break;
    const int at = c << e.gated;
    const float b0 = e.bias ? e.bias[ch0 + at] : 0.0f, b1 = e.bias && e.gated ? e.bias[ch0 + at + 1] : 0.0f;
    const uint8_t* rp = static_cast<const uint8_t*>(e.res) + (tok0 * e.ldr + col0 + c) * es;
    uint8_t* yp = static_cast<uint8_t*>(Y) + (tok0 * ldy + col0 + c) * es;
    const int64_t rstep = e.ldr * es, ystep = ldy * es;
    uint32_t next[4] = {0, 0, 0, 0};  // residuals as they lie in memory
    auto fetch = [&](int r) __attribute__((always_inline)) {  // the type's branch outside, so the four are in flight together
      if (e.res && e.f32) {
#pragma unroll
        for (int x = 0; x < 4; ++x) next[x] = *reinterpret_cast<const uint32_t*>(rp + min(r + x * beside, have - 1) * rstep);
      }
      if (e.res && !e.f32) {
#pragma unroll
        for (int x = 0; x < 4; ++x) next[x] = *reinterpret_cast<const uint16_t*>(rp + min(r + x * beside, have - 1) * rstep);
      }
    };
    fetch(first);
#pragma unroll 1
    for (int r = first; r < have; r += 4 * beside) {
      uint32_t res[4];
      float z[4], up[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) res[x] = next[x];
      fetch(r + 4 * beside);  // (behind the last row: the last one again)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float* p = stg + min(r + x * beside, have - 1) * ld + at;
        z[x] = p[0] + b0;
        up[x] = p[e.gated] + b1;
      }
      activate_n<4>(z, e.act, e.f32);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = r + x * beside;
        if (row >= have) break;
        float v = e.gated ? z[x] * up[x] : z[x];
        if (e.res) v += __uint_as_float(res[x] << shift);
        if (e.f32) *reinterpret_cast<float*>(yp + row * ystep) = v;
        else *reinterpret_cast<uint16_t*>(yp + row * ystep) = (uint16_t)pack_bf16x2(v, 0.0f);
      }
    }
  }
}

}  // namespace ss
