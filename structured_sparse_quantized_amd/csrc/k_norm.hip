// Root-mean-square norm of token rows, with the residual's addition before it and the quantisation and lift of the next
// product's activations behind it, in one pass over the rows:
//   r = x + residual (rounded to the stream's type and written: it is the next residual),
//   rs = fl32(1 / sqrt(mean(r^2) + eps)), z = fl32(fl32(r rs) w),
//   y = z rounded to bf16, or codes of the row z with one scale, lifted to K'.
//
// The mean is summed in float64: squares of float32 are exact there, so the order of a sum moves rs by 2^-52 and its rounding to
// float32 is the same for every order (but for one row in 10^8), which keeps the INT8 codes those of the definition, bit for
// bit. It costs two instructions of half rate a value.
//
// Bound: HBM. A row stays in registers between its three passes (squares, absmax, codes), so x and the residual are read
// once, r and the codes written once. A workgroup per row, or 4 or 16 short rows to one (655360 rows of 128 to bf16: 115 us, a
// workgroup of one wave each 242); a row's two sums go through LDS where it has several waves.
// Measured: 16384 x 4096 bf16 with residual to FP8 75-80 us, 5.9-6.3 TB/s (a large copy: 5.2); 6:8 INT8 79; 4096 x 14336 70; one row of
// 3584 3.5, which is a launch and three chains of latencies.
#include <algorithm>

#include "ss_device.h"
#include "ss_kernels.h"

namespace ss {
namespace norm {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <typename T> struct Vec;
template <> struct Vec<uint16_t> {  // 8 bf16 of 16 bytes
  static constexpr int E = 8;
  __device__ static float get(const v4u& v, int i) {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
  }
  __device__ static float load(const uint16_t* p) { return bf16_to_f32(*p); }
  __device__ static void store(uint16_t* p, float f) { *p = (uint16_t)pack_bf16x2(f, 0.0f); }
  __device__ static float round(float f) { return bf16_to_f32((uint16_t)pack_bf16x2(f, 0.0f)); }
  __device__ static v4u add(const v4u& a, const v4u& b) {
    v4u r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(get(a, 2 * i) + get(b, 2 * i), get(a, 2 * i + 1) + get(b, 2 * i + 1));
    return r;
  }
};
template <> struct Vec<float> {  // 4 floats
  static constexpr int E = 4;
  __device__ static float get(const v4u& v, int i) { return __uint_as_float(v[i]); }
  __device__ static float load(const float* p) { return *p; }
  __device__ static void store(float* p, float f) { *p = f; }
  __device__ static float round(float f) { return f; }
  __device__ static v4u add(const v4u& a, const v4u& b) {
    v4u r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(get(a, i) + get(b, i));
    return r;
  }
};

// Sum and maximum over the BT threads of a row (16, or whole waves).
template <int BT> __device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = BT < 64 ? BT / 2 : 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (BT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    lds_barrier();
    v = red[0];
#pragma unroll
    for (int i = 1; i < BT / 64; ++i) v += red[i];
  }
  return v;
}
// (the greater one; a NaN where either is one, unlike fmaxf)
__device__ __forceinline__ float greater(float a, float b) { return __builtin_elementwise_maximum(a, b); }
template <int BT> __device__ __forceinline__ float block_top(float v, float* red) {
#pragma unroll
  for (int o = BT < 64 ? BT / 2 : 32; o >= 1; o >>= 1) v = greater(v, __shfl_xor(v, o, 64));
  if constexpr (BT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    lds_barrier();
    v = red[0];
#pragma unroll
    for (int i = 1; i < BT / 64; ++i) v = greater(v, red[i]);
  }
  return v;
}
// 1 / sqrt(mean + eps), float32's largest number where it is beyond that, or 0 for a row of zeros without eps (its z are zeros,
// not 0 * infinity). Of a NaN: NaN; of an infinity: 0, so z is NaN there.
__device__ __forceinline__ float inverse_root(double sum, int64_t K, double eps) {
  const double m = sum / (double)K + eps, r = 1.0 / sqrt(m);
  return m == 0.0 ? 0.0f : r > 3.4028234663852886e38 ? 3.4028234663852886e38f : (float)r;
}
// The scale of a row whose largest |z| is `top`, and what z is multiplied with (two roundings: the header). A row with a NaN or an
// infinity among its z has codes of zero and that scale, so that its products are NaN and not those of an empty row.
template <typename Qz> struct Scale {
  bool zero;  // all codes are
  float inv, sx;
  __device__ explicit Scale(float top) {
    zero = !(top > 0.0f && top < INFINITY);
    inv = zero ? 0.0f : 1.0f / top * Qz::Q;
    sx = top == 0.0f ? 0.0f : top / Qz::Q;
  }
};

// The lift of a row of codes staged in LDS (zero behind K): whole periods of its byte pattern per thread.
template <int N, int BT> __device__ __forceinline__ void lift_row(const uint8_t* codes, uint8_t* out, int Kc, int tid) {
  using LP = LiftPeriod<N>;
  const int nchunk = Kc / 16, nper = (nchunk + LP::PC - 1) / LP::PC;
  const uint32_t* l32 = reinterpret_cast<const uint32_t*>(codes);
  for (int p = tid; p < nper; p += BT) {
    uint32_t s[LP::SW], o[4 * LP::PC];
#pragma unroll
    for (int i = 0; i < LP::SW; ++i) s[i] = l32[p * LP::SW + i];
    LP::emit(s, o);
#pragma unroll
    for (int h = 0; h < LP::PC; ++h)
      if (p * LP::PC + h < nchunk)
        *reinterpret_cast<uint4*>(out + (p * LP::PC + h) * 16) = make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
  }
}
// source bytes that the lift of n reads for Kc output bytes
__host__ __device__ inline int staged_bytes(int n, int Kc) {
  auto of = [&](int pc, int sb) { return (Kc / 16 + pc - 1) / pc * sb; };
  switch (n) {
    case 3: return of(LiftPeriod<3>::PC, LiftPeriod<3>::SB);
    case 4: return of(LiftPeriod<4>::PC, LiftPeriod<4>::SB);
    case 5: return of(LiftPeriod<5>::PC, LiftPeriod<5>::SB);
    case 6: return of(LiftPeriod<6>::PC, LiftPeriod<6>::SB);
    case 7: return of(LiftPeriod<7>::PC, LiftPeriod<7>::SB);
    default: return of(LiftPeriod<8>::PC, LiftPeriod<8>::SB);
  }
}
template <int BT> __device__ __forceinline__ void lift_any(int n, const uint8_t* codes, uint8_t* out, int Kc, int tid) {
  switch (n) {
    case 3: lift_row<3, BT>(codes, out, Kc, tid); break;
    case 4: lift_row<4, BT>(codes, out, Kc, tid); break;
    case 5: lift_row<5, BT>(codes, out, Kc, tid); break;
    case 6: lift_row<6, BT>(codes, out, Kc, tid); break;
    case 7: lift_row<7, BT>(codes, out, Kc, tid); break;
    default: lift_row<8, BT>(codes, out, Kc, tid); break;
  }
}

// T: the stream's type; TW: the weights'; OUT: 0 int8, 1 fp8, 2 bf16; BT threads of VPT vectors each hold a row, short rows
// several to a workgroup.
template <int BT> constexpr int rows_of() { return BT < 256 ? 256 / BT : 1; }
template <typename T, typename TW, int OUT, int BT, int VPT>
__global__ __launch_bounds__(BT * rows_of<BT>()) void row_kernel(NormArgs a) {
  using V = Vec<T>;
  constexpr int E = V::E;
  using Qz = Quant<OUT == 1>;
  constexpr int R = rows_of<BT>();
  extern __shared__ __align__(16) uint8_t all_codes[];  // of each row, where the lift gathers from LDS
  __shared__ double red_sum[R > 1 ? 1 : BT / 64];
  __shared__ float red_top[R > 1 ? 1 : BT / 64];
  const int tid = threadIdx.x % BT, sub = threadIdx.x / BT, K = (int)a.K;
  const int64_t row = a.first + (int64_t)blockIdx.x * R + sub;
  if (row >= a.last) return;  // (of a workgroup with several rows, whose only barrier waits for the waves that are left)
  const int nvec = K / E, tail = nvec * E + tid;  // a last part of a vector goes by elements, one a thread
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = static_cast<const T*>(a.res) + row * a.ldr;
  T* sum = static_cast<T*>(a.sum) + row * a.lds;
  const TW* w = static_cast<const TW*>(a.w);

  v4u r[VPT];
  float rt = 0.0f;
  {
    v4u b[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vi = tid + i * BT;
      r[i] = b[i] = v4u{0, 0, 0, 0};
      if (vi < nvec) {
        r[i] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(x) + vi);
        if (a.res) b[i] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(res) + vi);
      }
    }
    if (tail < K) {
      rt = V::load(x + tail);
      if (a.res) rt = V::round(rt + V::load(res + tail));
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int vi = tid + i * BT;
        r[i] = V::add(r[i], b[i]);
        if (vi < nvec) reinterpret_cast<v4u*>(sum)[vi] = r[i];
      }
      if (tail < K) V::store(sum + tail, rt);
    }
  }
  double s0 = (double)rt * rt, s1 = 0.0;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const double u = V::get(r[i], e), v = V::get(r[i], e + 1);
      s0 = __builtin_fma(u, u, s0);
      s1 = __builtin_fma(v, v, s1);
    }
  const float rs = inverse_root(block_sum<BT>(s0 + s1, red_sum), K, a.eps);

  float z[VPT * E], zt = rt * rs;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vi = tid + i * BT;
#pragma unroll
    for (int e = 0; e < E; ++e) z[i * E + e] = V::get(r[i], e) * rs;
    if (w && vi < nvec) {
      constexpr int EW = Vec<TW>::E;
#pragma unroll
      for (int p = 0; p < E / EW; ++p) {
        const v4u c = reinterpret_cast<const v4u*>(w)[vi * (E / EW) + p];
#pragma unroll
        for (int e = 0; e < EW; ++e) z[i * E + p * EW + e] *= Vec<TW>::get(c, e);
      }
    }
  }
  if (w && tail < K) zt *= Vec<TW>::load(w + tail);

  if constexpr (OUT == 2) {
    uint16_t* y = static_cast<uint16_t*>(a.y) + row * a.ldy;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vi = tid + i * BT;
      if (vi >= nvec) break;
      if constexpr (E == 8) {
        reinterpret_cast<uint4*>(y)[vi] = make_uint4(pack_bf16x2(z[i * 8], z[i * 8 + 1]), pack_bf16x2(z[i * 8 + 2], z[i * 8 + 3]),
                                                     pack_bf16x2(z[i * 8 + 4], z[i * 8 + 5]), pack_bf16x2(z[i * 8 + 6], z[i * 8 + 7]));
      } else {
        reinterpret_cast<uint2*>(y)[vi] = make_uint2(pack_bf16x2(z[i * 4], z[i * 4 + 1]), pack_bf16x2(z[i * 4 + 2], z[i * 4 + 3]));
      }
    }
    if (tail < K) y[tail] = (uint16_t)pack_bf16x2(zt, 0.0f);
  } else {
    float top = fabsf(zt);
#pragma unroll
    for (int i = 0; i < VPT * E; ++i) top = greater(top, fabsf(z[i]));
    const Scale<Qz> scale(block_top<BT>(top, red_top));
    const bool zero = scale.zero;
    const float inv = scale.inv;
    if (tid == 0) a.sx[row] = scale.sx;
    auto four = [&](int i) -> uint32_t { return zero ? 0u : Qz::pack4(z[i], z[i + 1], z[i + 2], z[i + 3], inv); };
    uint8_t* q = static_cast<uint8_t*>(a.y) + row * a.ldy;
    const int Kc = (int)a.Kc, n = a.n;
    if (n == 4 && E == 8 && (K & 7) == 0) {
      // 6:8 with whole groups: a vector is one group of 8, its windows bytes 0-3, 2-5 and 4-7 of the codes
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int vi = tid + i * BT;
        if (vi >= nvec) break;
        const uint32_t lo = four(i * E), hi = four(i * E + 4);
        uint32_t* p = reinterpret_cast<uint32_t*>(q) + vi * 3;
        p[0] = lo;
        p[1] = lo >> 16 | hi << 16;
        p[2] = hi;
      }
      for (int c = nvec * 12 + tid; c < Kc; c += BT) q[c] = 0;
    } else {
      uint8_t* codes = all_codes + sub * ((staged_bytes(n, Kc) + 15) / 16 * 16);
      uint8_t* to = n == 2 ? q : codes;
      const int end = n == 2 ? Kc : staged_bytes(n, Kc);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int vi = tid + i * BT;
        if (vi >= nvec) break;
        if constexpr (E == 8) *reinterpret_cast<uint2*>(to + vi * 8) = make_uint2(four(i * 8), four(i * 8 + 4));
        else *reinterpret_cast<uint32_t*>(to + vi * 4) = four(i * 4);
      }
      if (tail < K) to[tail] = zero ? 0 : Qz::code(zt, inv);
      for (int c = K + tid; c < end; c += BT) to[c] = 0;
      if (n != 2) {
        __syncthreads();
        lift_any<BT>(n, codes, q, Kc, tid);
      }
    }
  }
}

// Rows longer than the registers of a workgroup hold: the same steps, each over the row in memory. What a pass reads of r
// another thread of the workgroup may have written in the one before: the barriers between them order that.
template <typename T, typename TW, int OUT> __global__ __launch_bounds__(1024) void long_kernel(NormArgs a) {
  using V = Vec<T>;
  using Qz = Quant<OUT == 1>;
  constexpr int BT = 1024;
  __shared__ double red_sum[BT / 64];
  __shared__ float red_top[BT / 64];
  const int tid = threadIdx.x;
  const int64_t row = a.first + blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = static_cast<const T*>(a.res) + row * a.ldr;
  T* sum = static_cast<T*>(a.sum) + row * a.lds;
  const TW* w = static_cast<const TW*>(a.w);
  double s = 0.0;
  for (int64_t k = tid; k < a.K; k += BT) {
    float f = V::load(x + k);
    if (a.res) {
      f = V::round(f + V::load(res + k));
      V::store(sum + k, f);
    }
    s = __builtin_fma((double)f, (double)f, s);
  }
  const float rs = inverse_root(block_sum<BT>(s, red_sum), a.K, a.eps);
  __syncthreads();
  const T* r = a.res ? sum : x;
  auto z = [&](int64_t k) { return w ? V::load(r + k) * rs * Vec<TW>::load(w + k) : V::load(r + k) * rs; };
  if constexpr (OUT == 2) {
    uint16_t* y = static_cast<uint16_t*>(a.y) + row * a.ldy;
    for (int64_t k = tid; k < a.K; k += BT) y[k] = (uint16_t)pack_bf16x2(z(k), 0.0f);
  } else {
    float top = 0.0f;
    for (int64_t k = tid; k < a.K; k += BT) top = greater(top, fabsf(z(k)));
    const Scale<Qz> scale(block_top<BT>(top, red_top));
    const bool zero = scale.zero;
    const float inv = scale.inv;
    if (tid == 0) a.sx[row] = scale.sx;
    uint8_t* q = static_cast<uint8_t*>(a.y) + row * a.ldy;
    const int64_t gb = 4 * (a.n - 1);  // output bytes per group of 2n
    for (int64_t c = tid; c < a.Kc; c += BT) {
      const int64_t g = c / gb, rem = c - g * gb, src = a.n == 2 ? c : 2 * a.n * g + 2 * (rem >> 2) + (rem & 3);
      q[c] = src < a.K && !zero ? Qz::code(z(src), inv) : 0;
    }
  }
}

constexpr int64_t kSlab = 1 << 21;
template <typename T, typename TW, int OUT> hipError_t launch(const NormArgs& a, hipStream_t st) {
  constexpr int E = Vec<T>::E;
  const int64_t nvec = (a.K + E - 1) / E;
  const bool gathers = OUT != 2 && nvec <= 4096 && a.n != 2 && !(a.n == 4 && E == 8 && a.K % 8 == 0);
  const int64_t lds = !gathers ? 0 : (staged_bytes(a.n, (int)a.Kc) + 15) / 16 * 16;
  auto go = [&](auto kern, int threads, int rows = 1) -> hipError_t {
    const hipError_t e = lds_limit((const void*)kern, (int)(lds * rows));
    if (e != hipSuccess) return e;
    for (int64_t m = 0; m < a.M; m += kSlab) {  // launches of fewer than 2^32 threads
      NormArgs b = a;
      b.first = m;
      b.last = std::min(m + kSlab, a.M);
      hipLaunchKernelGGL(kern, dim3((unsigned)((b.last - m + rows - 1) / rows)), dim3(threads), (unsigned)(lds * rows), st, b);
      if (const hipError_t f = hipGetLastError(); f != hipSuccess) return f;
    }
    return hipSuccess;
  };
  if (nvec <= 16) return go(row_kernel<T, TW, OUT, 16, 1>, 256, 16);
  if (nvec <= 64) return go(row_kernel<T, TW, OUT, 64, 1>, 256, 4);
  if (nvec <= 256) return go(row_kernel<T, TW, OUT, 256, 1>, 256);
  if (nvec <= 512) return go(row_kernel<T, TW, OUT, 256, 2>, 256);
  if (nvec <= 1024) return go(row_kernel<T, TW, OUT, 256, 4>, 256);
  if (nvec <= 2048) return go(row_kernel<T, TW, OUT, 512, 4>, 512);
  if (nvec <= 4096) return go(row_kernel<T, TW, OUT, 1024, 4>, 1024);
  return go(long_kernel<T, TW, OUT>, 1024);
}
template <typename T, typename TW> hipError_t launch_out(int out, const NormArgs& a, hipStream_t st) {
  return out == 0 ? launch<T, TW, 0>(a, st) : out == 1 ? launch<T, TW, 1>(a, st) : launch<T, TW, 2>(a, st);
}

}  // namespace norm

hipError_t launch_rmsnorm(bool x_bf16, bool w_bf16, int out, const NormArgs& a, hipStream_t st) {
  if (!x_bf16) return norm::launch_out<float, float>(out, a, st);
  return w_bf16 ? norm::launch_out<uint16_t, uint16_t>(out, a, st) : norm::launch_out<uint16_t, float>(out, a, st);
}

}  // namespace ss
