// Host-callable launchers of the gfx950 kernels (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ss {

// Compute units of the current device (cached).
int num_cus_p();
// Raise a kernel's dynamic-LDS limit to `bytes` on the current device (the runtime call runs once per device,
// kernel and larger size).
hipError_t lds_limit(const void* kern, int bytes);
// Resident workgroups per CU (cached per device, kernel, block size and LDS bytes; at least 1).
int occupancy_p(const void* kern, int block, size_t lds);

hipError_t launch_quant_lift(bool x_bf16, bool fp8, const void* X, int64_t ldx, int64_t M, int64_t K, int n,
                             void* Xq, int64_t ldq, int64_t Kc, float* sx, hipStream_t st);

// out: 0 = int8, 1 = fp8, 2 = bf16
hipError_t launch_prune24(bool in_bf16, int out, const void* X, int64_t ldx, int64_t M, int64_t K, void* vals,
                          int64_t ldv_bytes, uint8_t* meta, int64_t ldm, int64_t Kc, float* scale, hipStream_t st);

hipError_t launch_slide(bool in_bf16, int out, const void* W, int64_t ldw, int64_t rows, int64_t K, int n, void* vals,
                        int64_t ldv_bytes, uint8_t* meta, int64_t ldm, int64_t Kc, float* scale, hipStream_t st);

// ab: 0 = int8, 1 = fp8, 2 = bf16; yt: 0 = bf16, 1 = f32, 2 = i32
hipError_t launch_spgemm(bool side_x, int ab, int yt, int64_t R, int64_t C, int64_t Kc, const void* av,
                         int64_t lda_bytes, const uint8_t* am, int64_t ldm, const void* bd, int64_t ldb_bytes,
                         const float* sx, const float* sw, void* Y, int64_t ldy, hipStream_t st);

// Online 2:4 prune of bf16 activations written in the tiled layout (out: 0 = int8, 1 = fp8, 2 = bf16).
hipError_t launch_prune24_act_tiled(int out, const void* X, int64_t ldx, int64_t M, int64_t K, int64_t Kc, void* tv,
                                    uint8_t* tm, float* sx, hipStream_t st);

// Weight preparation written in the tiled layout: 2:4 (F32 / BF16 input) and the (2n-2):2n decomposition.
hipError_t launch_prune24_tiled(bool in_bf16, int out, const void* W, int64_t ldw, int64_t rows, int64_t K, int64_t Kc,
                                void* tv, uint8_t* tm, float* scale, hipStream_t st);
hipError_t launch_slide_tiled(bool in_bf16, int out, const void* W, int64_t ldw, int64_t rows, int64_t K, int n,
                              int64_t Kc, void* tv, uint8_t* tm, float* scale, hipStream_t st);

// What the general epilogue of a product (yt = 3) does after the scales: z = scaled + bias[n]; act(z), or with
// `gated` act(z[2j]) * z[2j + 1] as column j; + residual; rounded to f32 or bf16.
struct Epilogue {
  const float* bias;  // [N] or NULL
  const void* res;    // type of Y, or NULL
  int64_t ldr;
  int act;    // ss_act
  int gated;
  int f32;    // Y and the residual are f32, else bf16
};

// Tiled sparse operand and the product that reads it. es = value bytes (1: int8/fp8, 2: bf16).
int64_t tiled_vals_bytes(int64_t rows, int64_t Kc, int es);
int64_t tiled_meta_bytes(int64_t rows, int64_t Kc, int es);
hipError_t launch_pack_tiled(int es, const uint8_t* vals, int64_t ldv_bytes, const uint8_t* meta, int64_t ldm,
                             int64_t rows, int64_t Kc, uint8_t* tv, uint8_t* tm, hipStream_t st);
// ab: 0 = int8, 1 = fp8, 2 = bf16; yt: 0 = bf16, 1 = f32, 2 = i32, 3 = the general epilogue `ep`
// ws: workspace of spgemm_tiled_workspace_bytes bytes, or NULL (no split-K path)
hipError_t launch_spgemm_tiled(bool side_x, int ab, int yt, int64_t R, int64_t C, int64_t Kc, const uint8_t* tv,
                               const uint8_t* tm, const void* bd, int64_t ldb_bytes, const float* sx, const float* sw,
                               void* Y, int64_t ldy, void* ws, const Epilogue& ep, hipStream_t st);
int64_t spgemm_tiled_workspace_bytes(bool side_x, int ab, int64_t R, int64_t C, int64_t Kc);
// The prefill kernel of k_spgemm_wide.hip with 256 x bn tiles (bn = 256: one workgroup per CU, weight-sparse
// side only, eight waves for reductions of at most 64 steps and four beyond; bn = 128: two workgroups of four
// waves); R = rows of the sparse operand, C = rows of the dense one, KS = steps of 64 value bytes, ldb in
// bytes; launch_spgemm_tiled routes the larger prefill problems to it.
hipError_t launch_spgemm_wide(int bn, bool side_x, int ab, int yt, int R, int C, int KS, const uint8_t* tv,
                              const uint8_t* tm, const uint8_t* bd, int ldb, const float* sx, const float* sw, void* Y,
                              int ldy, const Epilogue& ep, hipStream_t st);

// The small-tile kernel of k_spgemm_small.hip (general epilogue): 64 x 32 tj tiles, tj = 1, 2 or 4; arguments as above.
hipError_t launch_spgemm_small(int tj, bool side_x, int ab, int R, int C, int KS, const uint8_t* tv, const uint8_t* tm,
                               const uint8_t* bd, int ldb, const float* sx, const float* sw, void* Y, int ldy,
                               const Epilogue& ep, hipStream_t st);

// A batch of same-shaped tiled products (one launch; blockIdx.y = problem); strides in bytes for the tiled
// operand and the dense operand, in elements for the scales and Y.
hipError_t launch_spgemm_tiled_batched(bool side_x, int ab, int yt, int64_t batch, int64_t R, int64_t C, int64_t Kc,
                                       const uint8_t* tv, int64_t s_tv, const uint8_t* tm, int64_t s_tm, const void* bd,
                                       int64_t ldb_bytes, int64_t s_bd, const float* sx, int64_t s_sx, const float* sw,
                                       int64_t s_sw, void* Y, int64_t ldy, int64_t s_y, hipStream_t st);

// Few-token quant+lift fused into the weight-sparse row-block product (ab: 0 = int8, 1 = fp8; yt as above).
bool quant_lift_spgemm_fits(bool x_bf16, int64_t M, int64_t K, int64_t Kc);
hipError_t launch_quant_lift_spgemm(bool x_bf16, int ab, int yt, const void* X, int64_t ldx, int64_t M, int64_t K, int n,
                                    int64_t N, int64_t Kc, const uint8_t* tv, const uint8_t* tm, const float* sw,
                                    void* Y, int64_t ldy, float* sx_out, hipStream_t st);

// Prefill with the per-token quantisation inside the product (2:4 weights, K % 128 == 0, bf16 X): absmax
// into sx, the product coding X into its LDS stages, then sx = a / Q. ab: 0 = int8, 1 = fp8; yt: 0 = bf16,
// 1 = f32.
hipError_t launch_quant_spgemm_prefill(int ab, int yt, const uint16_t* X, int64_t ldx, int64_t M, int64_t K,
                                       const uint8_t* tv, const uint8_t* tm, const float* sw, int64_t N, void* Y,
                                       int64_t ldy, float* sx, hipStream_t st);

// Block-scaled FP8 (128 x 128 weight blocks, per-token groups of 128; 2:4 weights, K' = K = Kc):
// weight prep into the tiled operand with scales [ceil(rows / 128)][Kc / 128], activation codes [M][Kc] with
// scales [M][Kc / 128], and the weight-sparse product (yt: 0 = bf16, 1 = f32).
hipError_t launch_prune24_block(bool in_bf16, const void* W, int64_t ldw, int64_t rows, int64_t K, int64_t Kc,
                                void* tv, uint8_t* tm, float* sw, hipStream_t st);
hipError_t launch_quant_group(bool x_bf16, const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq, int64_t ldq,
                              int64_t Kc, float* sx, hipStream_t st);
hipError_t launch_spgemm_tiled_block(int yt, int64_t R, int64_t C, int64_t Kc, const uint8_t* tv, const uint8_t* tm,
                                     const void* bd, int64_t ldb_bytes, const float* sx, const float* sw, void* Y,
                                     int64_t ldy, hipStream_t st);

// Attention over packed sequences. Strides in elements (t: token, h: head); q, k, v, o are bf16.
struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  float* lse;  // [Hq][Tq] or NULL
  const int32_t *cu_q, *cu_k, *k_len;
  int64_t sqt, sqh, skt, skh, svt, svh, sot, soh;
  int64_t Tq, Tk;
  int B, Hkv, G, D;  // G = query heads per key head
  float c;           // scale * log2 e
  int causal, window, sinks;  // window 0: none
};
int64_t attn_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t window, int64_t sinks);
bool attn_fits(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t window, int64_t sinks);  // (a launch's threads)
hipError_t launch_attn(const AttnArgs& a, void* ws, hipStream_t st);

// Rotary positions on [T][H][D] views (strides in elements, t: token, h: head); y may be x (same strides).
struct RotaryArgs {
  const void* x;
  void* y;
  const int32_t* pos;     // [T]
  const uint64_t* steps;  // [rot / 2] turns per position * 2^64
  int64_t T, sxt, sxh, syt, syh;
  int H, D, rot;
  int half;  // pairs (i, i + rot / 2), else (2 i, 2 i + 1)
  float cscale, sscale;
};
hipError_t launch_rotary(bool bf16, const RotaryArgs& a, hipStream_t st);

// Norm of token rows with the residual's addition; out: 0 = int8, 1 = fp8 (codes lifted by n, scales sx), 2 = bf16.
struct NormArgs {
  const void *x, *res, *w;  // res, w: or NULL
  void *sum, *y;            // sum: where res is given
  float* sx;
  int64_t M, first, last, K, Kc, ldx, ldr, lds, ldy;  // first, last: the launch's rows
  double eps;
  int n;
};
hipError_t launch_rmsnorm(bool x_bf16, bool w_bf16, int out, const NormArgs& a, hipStream_t st);

// Rotary positions on queries and keys, keys and values into the pages of a cache (bf16; strides in elements).
struct StoreArgs {
  const uint16_t *q, *k, *v;
  uint16_t *qo, *kc, *vc;
  const int32_t *pos, *cu, *table;  // cu: or NULL (one token a sequence)
  const uint64_t* steps;
  int64_t T, first, B, ldt;  // first: of the launch's tokens
  int64_t sqt, sqh, skt, skh, svt, svh, sot, soh;
  int64_t kp, kt, kh, vp, vt, vh;  // cache: page, row, head
  int Hq, Hkv, D, rot, half, cols, pages, page;
  float mscale;
};
hipError_t launch_paged_store(const StoreArgs& a, hipStream_t st);

// Division of 0 .. 2^31 - 1 by a number known on the host: with 2^s the next power of two from d on, m = floor(2^(31+s) / d) + 1
// is (2^(31+s) + e) / d with 0 < e <= 2^s, so n m / 2^(31+s) passes n / d by less than 1 / d.
struct FastDiv {
  uint32_t m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    for (s = 0; (1ull << s) < d; ++s) {}
    m = (uint32_t)((1ull << (31 + s)) / d + 1);
  }
#ifdef __HIPCC__
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return __umulhi(n << 1, m) >> s; }
#endif
};

// Attention of few rows a sequence over a paged cache, or over contiguous keys under a window.
struct FlatArgs {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  float* lse;  // [Hq][Tq] or NULL
  const int32_t *cu_q, *cu_k, *k_len, *table;  // table: paged; cu_k: contiguous keys
  int64_t sqt, sqh, sot, soh, skh, svh;
  uint32_t skp, skt, svp, svt;  // page, key
  int64_t Tq, Tk, ldt;
  int B, Hkv, G, D, pages, page, cols;
  FastDiv by_G, by_Hkv, by_page, by_wgs;  // (set by the launch)
  float c;  // scale * log2 e
  int causal, window, sinks;  // window 0: none
  int paged;  // by table, else contiguous keys
  int whole, tokens;  // (set by the launch)
};
// room: the keys that a sequence has room for, on average; most: that any of them can have
int64_t flat_workspace_bytes(int64_t Tq, int64_t room, int64_t most, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t window,
                             int64_t sinks);
bool flat_fits(int64_t Tq, int64_t B, int64_t Hq, int64_t Hkv);  // (tiles within 31 bits)
hipError_t launch_flat(const FlatArgs& a, int64_t room, int64_t most, void* ws, hipStream_t st);

}  // namespace ss
