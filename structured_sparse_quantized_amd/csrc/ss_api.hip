// C ABI of the library: host-side argument validation, then one kernel launch
// per call on the caller's stream. Nothing is enqueued when validation fails.
#include <hip/hip_runtime.h>
#include <stdarg.h>

#include <atomic>
#include <cmath>
#include <stdio.h>
#include <string.h>

#include "ss.h"
#include "ss_kernels.h"

namespace {

thread_local char g_err[512] = "";

ss_status fail(ss_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return s;
}

ss_status ok() {
  g_err[0] = 0;
  return SS_OK;
}

ss_status hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(SS_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

int esize(ss_dtype t) {
  switch (t) {
    case SS_F32: case SS_I32: return 4;
    case SS_BF16: return 2;
    case SS_I8: case SS_FP8E4M3: return 1;
  }
  return 0;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Row starts of a [rows x cols] matrix with leading dimension ld (elements).
ss_status check_mat(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
  if (!p) return fail(SS_ERR_NULL, "%s is NULL", name);
  if (ld < cols) return fail(SS_ERR_SHAPE, "%s: leading dimension %lld < %lld columns", name, (long long)ld, (long long)cols);
  if (!aligned16(p)) return fail(SS_ERR_ALIGN, "%s is not 16-byte aligned", name);
  if (rows > 1 && (ld * es) % 16 != 0)
    return fail(SS_ERR_ALIGN, "%s: row stride of %lld bytes is not a multiple of 16", name, (long long)(ld * es));
  return SS_OK;
}

int out_code(ss_dtype t) { return t == SS_I8 ? 0 : t == SS_FP8E4M3 ? 1 : 2; }

}  // namespace

extern "C" {

int64_t ss_lifted_k_logical(int64_t K, int n) {
  if (K < 0 || n < 2 || n > 8) return -1;
  return (K + 2 * n - 1) / (2 * n) * 4 * (n - 1);
}

int64_t ss_lifted_k(int64_t K, int n) {
  const int64_t k = ss_lifted_k_logical(K, n);
  if (k < 0) return -1;
  return (k + SS_KALIGN - 1) / SS_KALIGN * SS_KALIGN;
}

const char* ss_status_string(int s) {
  switch (s) {
    case SS_OK: return "SS_OK";
    case SS_ERR_NULL: return "SS_ERR_NULL";
    case SS_ERR_SHAPE: return "SS_ERR_SHAPE";
    case SS_ERR_ALIGN: return "SS_ERR_ALIGN";
    case SS_ERR_DTYPE: return "SS_ERR_DTYPE";
    case SS_ERR_PATTERN: return "SS_ERR_PATTERN";
    case SS_ERR_UNSUPPORTED: return "SS_ERR_UNSUPPORTED";
    case SS_ERR_HIP: return "SS_ERR_HIP";
  }
  return "unknown status";
}

const char* ss_last_error(void) { return g_err; }
int ss_version(void) { return SS_VERSION; }

static ss_status check_weight_prep(const void* W, ss_dtype w_dt, int64_t rows, int64_t K, int64_t ldw,
                                   ss_dtype out_dt, void* vals, int64_t ldv, uint8_t* meta, int64_t ldm,
                                   float* scale, int64_t Kc) {
  if (w_dt != SS_F32 && w_dt != SS_BF16) return fail(SS_ERR_DTYPE, "input must be F32 or BF16");
  if (out_dt != SS_I8 && out_dt != SS_FP8E4M3 && out_dt != SS_BF16)
    return fail(SS_ERR_DTYPE, "output must be I8, FP8E4M3 or BF16");
  if (rows < 0 || K < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (rows > 0x7FFFFFFF) return fail(SS_ERR_SHAPE, "too many rows");
  if (rows == 0 || K == 0) return SS_OK;
  ss_status s;
  if ((s = check_mat("input", W, rows, K, ldw, esize(w_dt))) != SS_OK) return s;
  if ((s = check_mat("vals", vals, rows, Kc / 2, ldv, esize(out_dt))) != SS_OK) return s;
  if ((s = check_mat("meta", meta, rows, Kc / 8, ldm, 1)) != SS_OK) return s;
  if (out_dt == SS_BF16) {
    if (scale) return fail(SS_ERR_DTYPE, "BF16 output takes no scale (pass NULL)");
  } else if (!scale) {
    return fail(SS_ERR_NULL, "scale is NULL");
  }
  return SS_OK;
}

ss_status ss_prune24(const void* W, ss_dtype w_dt, int64_t rows, int64_t K, int64_t ldw, ss_dtype out_dt,
                     void* vals, int64_t ldv, uint8_t* meta, int64_t ldm, float* scale, void* stream) {
  if (K % 4 != 0) return fail(SS_ERR_SHAPE, "K=%lld is not a multiple of 4", (long long)K);
  const int64_t Kc = ss_lifted_k(K, 2);
  ss_status s = check_weight_prep(W, w_dt, rows, K, ldw, out_dt, vals, ldv, meta, ldm, scale, Kc);
  if (s != SS_OK) return s;
  if (rows == 0 || K == 0) return ok();
  return hip_status(ss::launch_prune24(w_dt == SS_BF16, out_code(out_dt), W, ldw, rows, K, vals, ldv * esize(out_dt),
                                       meta, ldm, Kc, scale, (hipStream_t)stream),
                    "ss_prune24 launch");
}

ss_status ss_slide_decompose(const void* W, ss_dtype w_dt, int64_t rows, int64_t K, int64_t ldw, int n,
                             ss_dtype out_dt, void* vals, int64_t ldv, uint8_t* meta, int64_t ldm, float* scale,
                             void* stream) {
  if (n < 2 || n > 8) return fail(SS_ERR_PATTERN, "n=%d outside 2..8", n);
  const int64_t Kc = ss_lifted_k(K, n);
  ss_status s = check_weight_prep(W, w_dt, rows, K, ldw, out_dt, vals, ldv, meta, ldm, scale, Kc);
  if (s != SS_OK) return s;
  if (rows == 0 || K == 0) return ok();
  return hip_status(ss::launch_slide(w_dt == SS_BF16, out_code(out_dt), W, ldw, rows, K, n, vals, ldv * esize(out_dt),
                                     meta, ldm, Kc, scale, (hipStream_t)stream),
                    "ss_slide_decompose launch");
}

ss_status ss_quant_lift_act(const void* X, ss_dtype x_dt, int64_t M, int64_t K, int64_t ldx, int n, ss_dtype q_dt,
                            void* Xq, int64_t ldq, float* sx, void* stream) {
  if (n < 2 || n > 8) return fail(SS_ERR_PATTERN, "n=%d outside 2..8", n);
  if (x_dt != SS_F32 && x_dt != SS_BF16) return fail(SS_ERR_DTYPE, "input must be F32 or BF16");
  if (q_dt != SS_I8 && q_dt != SS_FP8E4M3) return fail(SS_ERR_DTYPE, "output must be I8 or FP8E4M3");
  if (M < 0 || K < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (M > 0x7FFFFFFF) return fail(SS_ERR_SHAPE, "too many rows");
  if (M == 0 || K == 0) return ok();
  const int64_t Kc = ss_lifted_k(K, n);
  ss_status s;
  if ((s = check_mat("X", X, M, K, ldx, esize(x_dt))) != SS_OK) return s;
  if ((s = check_mat("Xq", Xq, M, Kc, ldq, 1)) != SS_OK) return s;
  if (!sx) return fail(SS_ERR_NULL, "sx is NULL");
  return hip_status(ss::launch_quant_lift(x_dt == SS_BF16, q_dt == SS_FP8E4M3, X, ldx, M, K, n, Xq, ldq, Kc, sx,
                                          (hipStream_t)stream),
                    "ss_quant_lift_act launch");
}

ss_status ss_prune24_act(const void* X, ss_dtype x_dt, int64_t M, int64_t K, int64_t ldx, ss_dtype out_dt, void* vals,
                         int64_t ldv, uint8_t* meta, int64_t ldm, float* sx, void* stream) {
  if (x_dt != SS_BF16) return fail(SS_ERR_DTYPE, "activations must be BF16");
  if (K % 4 != 0) return fail(SS_ERR_SHAPE, "K=%lld is not a multiple of 4", (long long)K);
  const int64_t Kc = ss_lifted_k(K, 2);
  ss_status s = check_weight_prep(X, x_dt, M, K, ldx, out_dt, vals, ldv, meta, ldm, sx, Kc);
  if (s != SS_OK) return s;
  if (M == 0 || K == 0) return ok();
  return hip_status(ss::launch_prune24(true, out_code(out_dt), X, ldx, M, K, vals, ldv * esize(out_dt), meta, ldm, Kc,
                                       sx, (hipStream_t)stream),
                    "ss_prune24_act launch");
}

ss_status ss_spgemm(ss_side side, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt, const void* sp_vals, int64_t ldsv,
                    const uint8_t* sp_meta, int64_t ldsm, const void* dense, int64_t ldd, const float* sx,
                    const float* sw, ss_dtype y_dt, void* Y, int64_t ldy, void* stream) {
  if (side != SS_SPARSE_W && side != SS_SPARSE_X) return fail(SS_ERR_SHAPE, "bad side");
  if (ab_dt != SS_I8 && ab_dt != SS_FP8E4M3 && ab_dt != SS_BF16)
    return fail(SS_ERR_DTYPE, "operands must be I8, FP8E4M3 or BF16");
  if (y_dt != SS_BF16 && y_dt != SS_F32 && y_dt != SS_I32) return fail(SS_ERR_DTYPE, "output must be BF16, F32 or I32");
  if (y_dt == SS_I32 && ab_dt != SS_I8) return fail(SS_ERR_DTYPE, "I32 output needs I8 operands");
  if (M < 0 || N < 0 || Kc < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (Kc % SS_KALIGN != 0) return fail(SS_ERR_SHAPE, "Kc=%lld is not a multiple of %d", (long long)Kc, SS_KALIGN);
  if (M > 0x7FFFFFFFLL * 128 || N > 0x7FFFFFFFLL * 128) return fail(SS_ERR_SHAPE, "too many rows");
  if (M == 0 || N == 0) return ok();
  const bool sx_side = (side == SS_SPARSE_X);
  const int64_t R = sx_side ? M : N, C = sx_side ? N : M;
  const int es = esize(ab_dt);
  ss_status s;
  if ((s = check_mat("sp_vals", sp_vals, R, Kc / 2, ldsv, es)) != SS_OK) return s;
  if ((s = check_mat("sp_meta", sp_meta, R, Kc / 8, ldsm, 1)) != SS_OK) return s;
  if ((s = check_mat("dense", dense, C, Kc, ldd, es)) != SS_OK) return s;
  // Y needs only an aligned base; rows are stored with vector writes when
  // ldy % 4 == 0 and element by element otherwise
  if ((s = check_mat("Y", Y, 1, N, ldy, esize(y_dt))) != SS_OK) return s;
  if (ab_dt != SS_BF16 && y_dt != SS_I32 && (!sx || !sw))
    return fail(SS_ERR_NULL, "INT8/FP8 products need both scales");
  const int ab = ab_dt == SS_I8 ? 0 : ab_dt == SS_FP8E4M3 ? 1 : 2;
  const int yt = y_dt == SS_BF16 ? 0 : y_dt == SS_F32 ? 1 : 2;
  return hip_status(ss::launch_spgemm(sx_side, ab, yt, R, C, Kc, sp_vals, ldsv * es, sp_meta, ldsm, dense, ldd * es,
                                      y_dt == SS_I32 ? nullptr : sx, y_dt == SS_I32 ? nullptr : sw, Y, ldy,
                                      (hipStream_t)stream),
                    "ss_spgemm launch");
}

int64_t ss_tiled_vals_bytes(int64_t rows, int64_t Kc, ss_dtype dt) {
  if (rows < 0 || Kc < 0 || Kc % SS_KALIGN != 0 || (dt != SS_I8 && dt != SS_FP8E4M3 && dt != SS_BF16)) return -1;
  return ss::tiled_vals_bytes(rows, Kc, esize(dt));
}

int64_t ss_tiled_meta_bytes(int64_t rows, int64_t Kc, ss_dtype dt) {
  if (rows < 0 || Kc < 0 || Kc % SS_KALIGN != 0 || (dt != SS_I8 && dt != SS_FP8E4M3 && dt != SS_BF16)) return -1;
  return ss::tiled_meta_bytes(rows, Kc, esize(dt));
}

ss_status ss_pack_sparse(int64_t rows, int64_t Kc, ss_dtype dt, const void* vals, int64_t ldv, const uint8_t* meta,
                         int64_t ldm, void* tvals, uint8_t* tmeta, void* stream) {
  if (dt != SS_I8 && dt != SS_FP8E4M3 && dt != SS_BF16) return fail(SS_ERR_DTYPE, "values must be I8, FP8E4M3 or BF16");
  if (rows < 0 || Kc < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (Kc % SS_KALIGN != 0) return fail(SS_ERR_SHAPE, "Kc=%lld is not a multiple of %d", (long long)Kc, SS_KALIGN);
  if (rows > 0x7FFFFFF0LL || Kc / 64 > 0x7FFFFFF0LL) return fail(SS_ERR_SHAPE, "too large");
  if (rows == 0 || Kc == 0) return ok();
  const int es = esize(dt);
  ss_status s;
  if ((s = check_mat("vals", vals, rows, Kc / 2, ldv, es)) != SS_OK) return s;
  if ((s = check_mat("meta", meta, rows, Kc / 8, ldm, 1)) != SS_OK) return s;
  if (!tvals || !tmeta) return fail(SS_ERR_NULL, "tiled outputs are NULL");
  if (!aligned16(tvals) || !aligned16(tmeta)) return fail(SS_ERR_ALIGN, "tiled outputs are not 16-byte aligned");
  return hip_status(ss::launch_pack_tiled(es, static_cast<const uint8_t*>(vals), ldv * es, meta, ldm, rows, Kc,
                                          static_cast<uint8_t*>(tvals), tmeta, (hipStream_t)stream),
                    "ss_pack_sparse launch");
}

ss_status ss_prune24_act_tiled(const void* X, ss_dtype x_dt, int64_t M, int64_t K, int64_t ldx, ss_dtype out_dt,
                               void* tvals, uint8_t* tmeta, float* sx, void* stream) {
  if (x_dt != SS_BF16) return fail(SS_ERR_DTYPE, "activations must be BF16");
  if (out_dt != SS_I8 && out_dt != SS_FP8E4M3 && out_dt != SS_BF16) return fail(SS_ERR_DTYPE, "bad output type");
  if (M < 0 || K < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (K % 4 != 0) return fail(SS_ERR_SHAPE, "K=%lld is not a multiple of 4", (long long)K);
  if (M > 0x7FFFFFF0LL || K > 0x3FFFFFF0LL) return fail(SS_ERR_SHAPE, "too large");
  if (M == 0 || K == 0) return ok();
  ss_status s;
  if ((s = check_mat("X", X, M, K, ldx, 2)) != SS_OK) return s;
  if (!tvals || !tmeta) return fail(SS_ERR_NULL, "tiled outputs are NULL");
  if (!aligned16(tvals) || !aligned16(tmeta)) return fail(SS_ERR_ALIGN, "tiled outputs are not 16-byte aligned");
  if (out_dt == SS_BF16 && sx) return fail(SS_ERR_DTYPE, "BF16 output takes no scale");
  if (out_dt != SS_BF16 && !sx) return fail(SS_ERR_NULL, "quantised output needs sx");
  const int64_t Kc = ss_lifted_k(K, 2);
  return hip_status(ss::launch_prune24_act_tiled(out_code(out_dt), X, ldx, M, K, Kc, tvals, tmeta, sx,
                                                 (hipStream_t)stream),
                    "ss_prune24_act_tiled launch");
}

ss_status ss_slide_decompose_tiled(const void* W, ss_dtype w_dt, int64_t rows, int64_t K, int64_t ldw, int n,
                                   ss_dtype out_dt, void* tvals, uint8_t* tmeta, float* scale, void* stream) {
  if (n < 2 || n > 8) return fail(SS_ERR_PATTERN, "n=%d outside 2..8", n);
  if (w_dt != SS_F32 && w_dt != SS_BF16) return fail(SS_ERR_DTYPE, "input must be F32 or BF16");
  if (out_dt != SS_I8 && out_dt != SS_FP8E4M3 && out_dt != SS_BF16)
    return fail(SS_ERR_DTYPE, "output must be I8, FP8E4M3 or BF16");
  if (rows < 0 || K < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (rows > 0x7FFFFFF0LL || K > 0x3FFFFFF0LL) return fail(SS_ERR_SHAPE, "too large");
  if (rows == 0 || K == 0) return ok();
  ss_status s;
  if ((s = check_mat("input", W, rows, K, ldw, esize(w_dt))) != SS_OK) return s;
  if (!tvals || !tmeta) return fail(SS_ERR_NULL, "tiled outputs are NULL");
  if (!aligned16(tvals) || !aligned16(tmeta)) return fail(SS_ERR_ALIGN, "tiled outputs are not 16-byte aligned");
  if (out_dt == SS_BF16 && scale) return fail(SS_ERR_DTYPE, "BF16 output takes no scale (pass NULL)");
  if (out_dt != SS_BF16 && !scale) return fail(SS_ERR_NULL, "scale is NULL");
  const int64_t Kc = ss_lifted_k(K, n);
  return hip_status(ss::launch_slide_tiled(w_dt == SS_BF16, out_code(out_dt), W, ldw, rows, K, n, Kc, tvals, tmeta,
                                           scale, (hipStream_t)stream),
                    "ss_slide_decompose_tiled launch");
}

// Checks shared by ss_spgemm_tiled and ss_spgemm_tiled_ws; sets *run = false for an empty problem.
static ss_status check_spgemm_tiled(ss_side side, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt, const void* tvals,
                                    const uint8_t* tmeta, const void* dense, int64_t ldd, const float* sx,
                                    const float* sw, ss_dtype y_dt, void* Y, int64_t ldy, bool* run,
                                    bool half_width = false) {
  *run = false;
  if (side != SS_SPARSE_W && side != SS_SPARSE_X) return fail(SS_ERR_SHAPE, "bad side");
  if (ab_dt != SS_I8 && ab_dt != SS_FP8E4M3 && ab_dt != SS_BF16)
    return fail(SS_ERR_DTYPE, "operands must be I8, FP8E4M3 or BF16");
  if (y_dt != SS_BF16 && y_dt != SS_F32 && y_dt != SS_I32) return fail(SS_ERR_DTYPE, "output must be BF16, F32 or I32");
  if (y_dt == SS_I32 && ab_dt != SS_I8) return fail(SS_ERR_DTYPE, "I32 output needs I8 operands");
  if (M < 0 || N < 0 || Kc < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (Kc % SS_KALIGN != 0) return fail(SS_ERR_SHAPE, "Kc=%lld is not a multiple of %d", (long long)Kc, SS_KALIGN);
  if (M == 0 || N == 0) return SS_OK;
  if (Kc == 0) return fail(SS_ERR_SHAPE, "Kc must be positive");
  const bool sx_side = (side == SS_SPARSE_X);
  const int64_t R = sx_side ? M : N, C = sx_side ? N : M;
  if (R > 0x7FFFFFF0LL || C > 0x7FFFFFF0LL || ldy > 0x7FFFFFFFLL || Kc / 64 > 0x7FFFFFF0LL)
    return fail(SS_ERR_SHAPE, "too large");
  const int es = esize(ab_dt);
  ss_status s;
  if ((s = check_mat("dense", dense, C, Kc, ldd, es)) != SS_OK) return s;
  // the kernel addresses the dense operand with 32-bit byte offsets
  if ((uint64_t)(C - 1) * (uint64_t)ldd * es + (uint64_t)Kc * es > 0xFFFFFFFFull)
    return fail(SS_ERR_UNSUPPORTED, "dense operand spans more than 4 GiB");
  if ((s = check_mat("Y", Y, 1, half_width ? N / 2 : N, ldy, esize(y_dt))) != SS_OK) return s;
  if (!tvals || !tmeta) return fail(SS_ERR_NULL, "tiled operand is NULL");
  if (!aligned16(tvals) || !aligned16(tmeta)) return fail(SS_ERR_ALIGN, "tiled operand is not 16-byte aligned");
  if (ab_dt != SS_BF16 && y_dt != SS_I32 && (!sx || !sw)) return fail(SS_ERR_NULL, "INT8/FP8 products need both scales");
  *run = true;
  return SS_OK;
}

static ss_status run_spgemm_tiled(ss_side side, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt, const void* tvals,
                                  const uint8_t* tmeta, const void* dense, int64_t ldd, const float* sx,
                                  const float* sw, ss_dtype y_dt, void* Y, int64_t ldy, void* ws, void* stream,
                                  const ss::Epilogue* ep = nullptr) {
  const bool sx_side = (side == SS_SPARSE_X);
  const int64_t R = sx_side ? M : N, C = sx_side ? N : M;
  const int ab = ab_dt == SS_I8 ? 0 : ab_dt == SS_FP8E4M3 ? 1 : 2;
  const int yt = ep ? 3 : y_dt == SS_BF16 ? 0 : y_dt == SS_F32 ? 1 : 2;
  return hip_status(ss::launch_spgemm_tiled(sx_side, ab, yt, R, C, Kc, static_cast<const uint8_t*>(tvals), tmeta, dense,
                                            ldd * esize(ab_dt), y_dt == SS_I32 ? nullptr : sx,
                                            y_dt == SS_I32 ? nullptr : sw, Y, ldy, ws, ep ? *ep : ss::Epilogue{},
                                            (hipStream_t)stream),
                    "ss_spgemm_tiled launch");
}

ss_status ss_spgemm_tiled(ss_side side, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt, const void* tvals,
                          const uint8_t* tmeta, const void* dense, int64_t ldd, const float* sx, const float* sw,
                          ss_dtype y_dt, void* Y, int64_t ldy, void* stream) {
  bool run = false;
  const ss_status s = check_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy, &run);
  if (s != SS_OK) return s;
  if (!run) return ok();
  return run_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy, nullptr, stream);
}

int64_t ss_spgemm_tiled_workspace_bytes(ss_side side, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt) {
  if (side != SS_SPARSE_W && side != SS_SPARSE_X) return -1;
  if (ab_dt != SS_I8 && ab_dt != SS_FP8E4M3 && ab_dt != SS_BF16) return -1;
  if (M < 0 || N < 0 || Kc < 0 || Kc % SS_KALIGN != 0) return -1;
  if (M == 0 || N == 0 || Kc == 0 || M > 0x7FFFFFF0LL || N > 0x7FFFFFF0LL) return 0;
  const bool sx_side = (side == SS_SPARSE_X);
  const int ab = ab_dt == SS_I8 ? 0 : ab_dt == SS_FP8E4M3 ? 1 : 2;
  return ss::spgemm_tiled_workspace_bytes(sx_side, ab, sx_side ? M : N, sx_side ? N : M, Kc);
}

// The allocation-free variant's split-K workspace: a static array in the code object (one copy per GPU), and
// its device address per GPU, looked up once with that GPU current. Host code must use the looked-up
// address: the array's name on the host is only a stand-in for the symbol.
static __device__ __align__(256) uint8_t scratch[SS_NOALLOC_SCRATCH_BYTES];
namespace {
constexpr int kMaxDevices = 64;
std::atomic<void*> g_scratch[kMaxDevices];

ss_status scratch_ptr(void** out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(SS_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(SS_ERR_UNSUPPORTED, "device %d beyond the %d the library tracks", dev,
                                                 kMaxDevices);
  void* p = g_scratch[dev].load(std::memory_order_acquire);
  if (!p) {
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || !p) return fail(SS_ERR_HIP, "hipGetSymbolAddress(scratch): %s", hipGetErrorString(e));
    g_scratch[dev].store(p, std::memory_order_release);
  }
  *out = p;
  return SS_OK;
}
}  // namespace

ss_status ss_spgemm_tiled_noalloc(ss_side side, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt, const void* tvals,
                                  const uint8_t* tmeta, const void* dense, int64_t ldd, const float* sx,
                                  const float* sw, ss_dtype y_dt, void* Y, int64_t ldy, void* stream) {
  bool run = false;
  ss_status s = check_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy, &run);
  if (s != SS_OK) return s;
  if (!run) return ok();
  const int64_t need = ss_spgemm_tiled_workspace_bytes(side, M, N, Kc, ab_dt);
  if (need > SS_NOALLOC_SCRATCH_BYTES)
    return fail(SS_ERR_UNSUPPORTED, "workspace of %lld bytes exceeds the %d-byte static scratch", (long long)need,
                SS_NOALLOC_SCRATCH_BYTES);
  void* ws = nullptr;
  if (need > 0 && (s = scratch_ptr(&ws)) != SS_OK) return s;
  return run_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy, ws, stream);
}

ss_status ss_quant_spgemm_prefill(const void* X, ss_dtype x_dt, int64_t M, int64_t K, int64_t ldx, ss_dtype q_dt,
                                  const void* tvals, const uint8_t* tmeta, const float* sw, int64_t N, ss_dtype y_dt,
                                  void* Y, int64_t ldy, float* sx, void* stream) {
  if (x_dt != SS_BF16) return fail(SS_ERR_DTYPE, "X must be BF16");
  if (q_dt != SS_I8 && q_dt != SS_FP8E4M3) return fail(SS_ERR_DTYPE, "codes must be I8 or FP8E4M3");
  if (y_dt != SS_BF16 && y_dt != SS_F32) return fail(SS_ERR_DTYPE, "output must be BF16 or F32");
  if (M < 0 || N < 0 || K < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (K % 128 != 0) return fail(SS_ERR_SHAPE, "K=%lld is not a multiple of 128", (long long)K);
  if (M == 0 || N == 0) return ok();
  if (K == 0) return fail(SS_ERR_SHAPE, "K must be positive");
  if (M > 0x7FFFFFF0LL || N > 0x7FFFFFF0LL || K > 0x7FFFFF00LL || ldy > 0x7FFFFFFFLL || ldx > 0x7FFFFFFFLL)
    return fail(SS_ERR_SHAPE, "too large");
  ss_status s;
  if ((s = check_mat("X", X, M, K, ldx, 2)) != SS_OK) return s;
  // (output rows need no 16-byte alignment: the stores fall back to single elements)
  if ((s = check_mat("Y", Y, 1, N, ldy, esize(y_dt))) != SS_OK) return s;
  if (!tvals || !tmeta || !sw || !sx) return fail(SS_ERR_NULL, "tvals, tmeta, sw and sx are required");
  if (!aligned16(tvals) || !aligned16(tmeta)) return fail(SS_ERR_ALIGN, "tiled operand is not 16-byte aligned");
  return hip_status(ss::launch_quant_spgemm_prefill(q_dt == SS_I8 ? 0 : 1, y_dt == SS_BF16 ? 0 : 1,
                                                    static_cast<const uint16_t*>(X), ldx, M, K,
                                                    static_cast<const uint8_t*>(tvals), tmeta, sw, N, Y, ldy, sx,
                                                    (hipStream_t)stream),
                    "ss_quant_spgemm_prefill launch");
}

ss_status ss_spgemm_tiled_ws(ss_side side, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt, const void* tvals,
                             const uint8_t* tmeta, const void* dense, int64_t ldd, const float* sx, const float* sw,
                             ss_dtype y_dt, void* Y, int64_t ldy, void* workspace, int64_t ws_bytes, void* stream) {
  bool run = false;
  const ss_status s = check_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy, &run);
  if (s != SS_OK) return s;
  if (ws_bytes < 0) return fail(SS_ERR_SHAPE, "negative workspace size");
  if (!run) return ok();
  const int64_t need = ss_spgemm_tiled_workspace_bytes(side, M, N, Kc, ab_dt);
  if (need > 0) {
    if (!workspace) return fail(SS_ERR_NULL, "workspace is NULL (%lld bytes needed)", (long long)need);
    if (!aligned16(workspace)) return fail(SS_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (ws_bytes < need) return fail(SS_ERR_SHAPE, "workspace of %lld bytes, %lld needed", (long long)ws_bytes,
                                     (long long)need);
  }
  return run_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy,
                          need > 0 ? workspace : nullptr, stream);
}

ss_status ss_spgemm_tiled_epilogue(ss_side side, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt, const void* tvals,
                                   const uint8_t* tmeta, const void* dense, int64_t ldd, const float* sx,
                                   const float* sw, const float* bias, ss_act act, int gated, const void* residual,
                                   int64_t ldr, ss_dtype y_dt, void* Y, int64_t ldy, void* workspace,
                                   int64_t ws_bytes, void* stream) {
  if (y_dt != SS_BF16 && y_dt != SS_F32) return fail(SS_ERR_DTYPE, "output must be BF16 or F32");
  if (act < SS_ACT_NONE || act > SS_ACT_SILU) return fail(SS_ERR_UNSUPPORTED, "unknown activation %d", (int)act);
  if (gated && N % 2 != 0) return fail(SS_ERR_SHAPE, "a gate needs an even N, has %lld", (long long)N);
  bool run = false;
  ss_status s = check_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy, &run, gated != 0);
  if (s != SS_OK) return s;
  if (ws_bytes < 0) return fail(SS_ERR_SHAPE, "negative workspace size");
  if (!run) return ok();
  if (residual) {
    if ((s = check_mat("residual", residual, 1, gated ? N / 2 : N, ldr, esize(y_dt))) != SS_OK) return s;
    if (residual == Y && ldr != ldy) return fail(SS_ERR_SHAPE, "a residual in place needs ldr = ldy");
  }
  if ((uintptr_t)bias % 4 != 0) return fail(SS_ERR_ALIGN, "bias is not aligned to its elements");
  const int64_t need = ss_spgemm_tiled_workspace_bytes(side, M, N, Kc, ab_dt);
  if (need > 0) {
    if (!workspace) return fail(SS_ERR_NULL, "workspace is NULL (%lld bytes needed)", (long long)need);
    if (!aligned16(workspace)) return fail(SS_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (ws_bytes < need) return fail(SS_ERR_SHAPE, "workspace of %lld bytes, %lld needed", (long long)ws_bytes,
                                     (long long)need);
  }
  const ss::Epilogue ep{bias, residual, residual ? ldr : 0, (int)act, gated ? 1 : 0, y_dt == SS_F32 ? 1 : 0};
  return run_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy,
                          need > 0 ? workspace : nullptr, stream, &ep);
}

ss_status ss_prune24_block(const void* W, ss_dtype w_dt, int64_t rows, int64_t K, int64_t ldw, void* tvals,
                           uint8_t* tmeta, float* sw, void* stream) {
  if (w_dt != SS_F32 && w_dt != SS_BF16) return fail(SS_ERR_DTYPE, "input must be F32 or BF16");
  if (rows < 0 || K < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (K % 4 != 0) return fail(SS_ERR_SHAPE, "K=%lld is not a multiple of 4", (long long)K);
  if (rows > 0x7FFFFFF0LL || K > 0x3FFFFFF0LL) return fail(SS_ERR_SHAPE, "too large");
  if (rows == 0 || K == 0) return ok();
  ss_status s;
  if ((s = check_mat("input", W, rows, K, ldw, esize(w_dt))) != SS_OK) return s;
  if (!tvals || !tmeta) return fail(SS_ERR_NULL, "tiled outputs are NULL");
  if (!aligned16(tvals) || !aligned16(tmeta)) return fail(SS_ERR_ALIGN, "tiled outputs are not 16-byte aligned");
  if (!sw) return fail(SS_ERR_NULL, "sw is NULL");
  const int64_t Kc = ss_lifted_k(K, 2);
  return hip_status(ss::launch_prune24_block(w_dt == SS_BF16, W, ldw, rows, K, Kc, tvals, tmeta, sw,
                                             (hipStream_t)stream),
                    "ss_prune24_block launch");
}

ss_status ss_quant_group_act(const void* X, ss_dtype x_dt, int64_t M, int64_t K, int64_t ldx, void* Xq, int64_t ldq,
                             float* sx, void* stream) {
  if (x_dt != SS_F32 && x_dt != SS_BF16) return fail(SS_ERR_DTYPE, "input must be F32 or BF16");
  if (M < 0 || K < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (M > 0x7FFFFFF0LL || K > 0x3FFFFFF0LL) return fail(SS_ERR_SHAPE, "too large");
  if (M == 0 || K == 0) return ok();
  const int64_t Kc = ss_lifted_k(K, 2);
  if (M * ((Kc / 128 + 15) / 16) > 0x7FFFFFFFLL) return fail(SS_ERR_SHAPE, "too large");
  ss_status s;
  if ((s = check_mat("X", X, M, K, ldx, esize(x_dt))) != SS_OK) return s;
  if ((s = check_mat("Xq", Xq, M, Kc, ldq, 1)) != SS_OK) return s;
  if (!sx) return fail(SS_ERR_NULL, "sx is NULL");
  return hip_status(ss::launch_quant_group(x_dt == SS_BF16, X, ldx, M, K, Xq, ldq, Kc, sx, (hipStream_t)stream),
                    "ss_quant_group_act launch");
}

ss_status ss_spgemm_tiled_block(int64_t M, int64_t N, int64_t Kc, const void* tvals, const uint8_t* tmeta,
                                const void* dense, int64_t ldd, const float* sx, const float* sw, ss_dtype y_dt,
                                void* Y, int64_t ldy, void* stream) {
  if (y_dt != SS_BF16 && y_dt != SS_F32) return fail(SS_ERR_DTYPE, "output must be BF16 or F32");
  if (M < 0 || N < 0 || Kc < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (Kc % SS_KALIGN != 0) return fail(SS_ERR_SHAPE, "Kc=%lld is not a multiple of %d", (long long)Kc, SS_KALIGN);
  if (M == 0 || N == 0) return ok();
  if (Kc == 0) return fail(SS_ERR_SHAPE, "Kc must be positive");
  if (M > 0x7FFFFFF0LL || N > 0x7FFFFFF0LL || ldy > 0x7FFFFFFFLL || Kc / 64 > 0x7FFFFFF0LL)
    return fail(SS_ERR_SHAPE, "too large");
  ss_status s;
  if ((s = check_mat("dense", dense, M, Kc, ldd, 1)) != SS_OK) return s;
  if ((uint64_t)(M - 1) * (uint64_t)ldd + (uint64_t)Kc > 0xFFFFFFFFull)
    return fail(SS_ERR_UNSUPPORTED, "dense operand spans more than 4 GiB");
  if ((s = check_mat("Y", Y, 1, N, ldy, esize(y_dt))) != SS_OK) return s;
  if (!tvals || !tmeta) return fail(SS_ERR_NULL, "tiled operand is NULL");
  if (!aligned16(tvals) || !aligned16(tmeta)) return fail(SS_ERR_ALIGN, "tiled operand is not 16-byte aligned");
  if (!sx || !sw) return fail(SS_ERR_NULL, "block-scaled products need both scale arrays");
  return hip_status(ss::launch_spgemm_tiled_block(y_dt == SS_BF16 ? 0 : 1, N, M, Kc, static_cast<const uint8_t*>(tvals),
                                                  tmeta, dense, ldd, sx, sw, Y, ldy, (hipStream_t)stream),
                    "ss_spgemm_tiled_block launch");
}

ss_status ss_spgemm_tiled_batched(ss_side side, int64_t batch, int64_t M, int64_t N, int64_t Kc, ss_dtype ab_dt,
                                  const void* tvals, int64_t tvals_stride, const uint8_t* tmeta, int64_t tmeta_stride,
                                  const void* dense, int64_t ldd, int64_t dense_stride, const float* sx,
                                  int64_t sx_stride, const float* sw, int64_t sw_stride, ss_dtype y_dt, void* Y,
                                  int64_t ldy, int64_t y_stride, void* stream) {
  if (batch < 0) return fail(SS_ERR_SHAPE, "negative batch");
  bool run = false;
  const ss_status s = check_spgemm_tiled(side, M, N, Kc, ab_dt, tvals, tmeta, dense, ldd, sx, sw, y_dt, Y, ldy, &run);
  if (s != SS_OK) return s;
  if (!run || batch == 0) return ok();
  if (batch > 65535) return fail(SS_ERR_SHAPE, "batch=%lld exceeds 65535", (long long)batch);
  if (tvals_stride < 0 || tmeta_stride < 0 || dense_stride < 0 || sx_stride < 0 || sw_stride < 0 || y_stride < 0)
    return fail(SS_ERR_SHAPE, "negative stride");
  const int es = esize(ab_dt);
  if (tvals_stride % 16 || tmeta_stride % 16 || (dense_stride * es) % 16 || (y_stride * esize(y_dt)) % 16)
    return fail(SS_ERR_ALIGN, "operand strides must keep every problem 16-byte aligned");
  const bool sx_side = (side == SS_SPARSE_X);
  const int64_t R = sx_side ? M : N, C = sx_side ? N : M;
  const int ab = ab_dt == SS_I8 ? 0 : ab_dt == SS_FP8E4M3 ? 1 : 2;
  const int yt = y_dt == SS_BF16 ? 0 : y_dt == SS_F32 ? 1 : 2;
  return hip_status(ss::launch_spgemm_tiled_batched(sx_side, ab, yt, batch, R, C, Kc, static_cast<const uint8_t*>(tvals),
                                                    tvals_stride, tmeta, tmeta_stride, dense, ldd * es, dense_stride * es,
                                                    y_dt == SS_I32 ? nullptr : sx, sx_stride,
                                                    y_dt == SS_I32 ? nullptr : sw, sw_stride, Y, ldy, y_stride,
                                                    (hipStream_t)stream),
                    "ss_spgemm_tiled_batched launch");
}

ss_status ss_quant_lift_spgemm_decode(const void* X, ss_dtype x_dt, int64_t M, int64_t K, int64_t ldx, int n,
                                      ss_dtype q_dt, const void* tvals, const uint8_t* tmeta, const float* sw, int64_t N,
                                      ss_dtype y_dt, void* Y, int64_t ldy, float* sx_out, void* stream) {
  if (n < 2 || n > 8) return fail(SS_ERR_PATTERN, "n=%d outside 2..8", n);
  if (x_dt != SS_F32 && x_dt != SS_BF16) return fail(SS_ERR_DTYPE, "input must be F32 or BF16");
  if (q_dt != SS_I8 && q_dt != SS_FP8E4M3) return fail(SS_ERR_DTYPE, "codes must be I8 or FP8E4M3");
  if (y_dt != SS_BF16 && y_dt != SS_F32 && y_dt != SS_I32) return fail(SS_ERR_DTYPE, "output must be BF16, F32 or I32");
  if (y_dt == SS_I32 && q_dt != SS_I8) return fail(SS_ERR_DTYPE, "I32 output needs I8 codes");
  if (M < 0 || K < 0 || N < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (M == 0 || N == 0) return ok();
  if (K == 0) return fail(SS_ERR_SHAPE, "K must be positive");
  if (N > 0x7FFFFFF0LL || K > 0x3FFFFFF0LL || ldy > 0x7FFFFFFFLL) return fail(SS_ERR_SHAPE, "too large");
  const int64_t Kc = ss_lifted_k(K, n);
  if (!ss::quant_lift_spgemm_fits(x_dt == SS_BF16, M, K, Kc))
    return fail(SS_ERR_UNSUPPORTED, "M=%lld, K=%lld: the fused path takes 1..4 tokens with M*K' <= 131072 and K <= %d",
                (long long)M, (long long)K, x_dt == SS_BF16 ? 20480 : 16384);
  ss_status s;
  if ((s = check_mat("X", X, M, K, ldx, esize(x_dt))) != SS_OK) return s;
  if ((s = check_mat("Y", Y, 1, N, ldy, esize(y_dt))) != SS_OK) return s;
  if (!tvals || !tmeta) return fail(SS_ERR_NULL, "tiled operand is NULL");
  if (!aligned16(tvals) || !aligned16(tmeta)) return fail(SS_ERR_ALIGN, "tiled operand is not 16-byte aligned");
  if (!sw) return fail(SS_ERR_NULL, "sw is NULL");
  return hip_status(ss::launch_quant_lift_spgemm(x_dt == SS_BF16, q_dt == SS_I8 ? 0 : 1,
                                                 y_dt == SS_BF16 ? 0 : y_dt == SS_F32 ? 1 : 2, X, ldx, M, K, n, N, Kc,
                                                 static_cast<const uint8_t*>(tvals), tmeta, sw, Y, ldy, sx_out,
                                                 (hipStream_t)stream),
                    "ss_quant_lift_spgemm_decode launch");
}

ss_status ss_rotary_steps(int rot_dim, double base, ss_rope_scaling scaling, double factor, double original,
                          double low, double high, uint64_t* steps, float* mscale) {
  if (rot_dim < 2 || rot_dim % 2 != 0) return fail(SS_ERR_SHAPE, "rot_dim=%d must be even and at least 2", rot_dim);
  if (scaling < SS_ROPE_NONE || scaling > SS_ROPE_YARN) return fail(SS_ERR_UNSUPPORTED, "unknown scaling %d", (int)scaling);
  if (!(base > 0) || !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor))
    return fail(SS_ERR_SHAPE, "base and factor must be positive and finite");
  const bool ctx = scaling == SS_ROPE_SMOOTH || scaling == SS_ROPE_YARN;
  if (ctx && (!(original > 0) || !std::isfinite(original) || !(low > 0) || !(high > low) || !std::isfinite(high)))
    return fail(SS_ERR_SHAPE, "this scaling needs original > 0 and 0 < low < high");
  if (scaling == SS_ROPE_YARN && !(base > 1)) return fail(SS_ERR_SHAPE, "this scaling needs base > 1");
  if (!steps || !mscale) return fail(SS_ERR_NULL, "steps or mscale is NULL");
  const long double two_pi = 6.283185307179586476925286766559005768L;
  const int n = rot_dim / 2;
  long double bs = base;
  if (scaling == SS_ROPE_NTK && rot_dim > 2) bs *= powl((long double)factor, (long double)rot_dim / (rot_dim - 2));
  long double first = 0, last = 0;
  if (scaling == SS_ROPE_YARN) {
    auto pair_of = [&](double turns) {  // the (fractional) pair that turns so often over the original context
      return rot_dim * logl((long double)original / (two_pi * turns)) / (2 * logl((long double)base));
    };
    first = fmaxl(0, floorl(pair_of(high)));
    last = fminl(rot_dim - 1, ceill(pair_of(low)));
  }
  for (int i = 0; i < n; ++i) {
    long double f = powl(bs, -2.0L * i / rot_dim);
    if (scaling == SS_ROPE_LINEAR) f /= factor;
    if (ctx) {
      long double keep;
      if (scaling == SS_ROPE_SMOOTH) keep = ((long double)original * f / two_pi - low) / ((long double)high - low);
      else keep = 1 - (i - first) / fmaxl(last - first, 0.001L);
      keep = fminl(1, fmaxl(0, keep));
      f = f / factor * (1 - keep) + f * keep;
    }
    const long double turns = f / two_pi;
    const long double frac = turns - floorl(turns);
    const long double units = rintl(frac * 0x1p64L);
    steps[i] = units >= 0x1p64L ? 0 : (uint64_t)units;
  }
  *mscale = scaling == SS_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return ok();
}

ss_status ss_rotary(const void* x, ss_dtype x_dt, int64_t T, int64_t H, int64_t D, int64_t sxt, int64_t sxh,
                    const int32_t* pos, const uint64_t* steps, int64_t rot_dim, ss_rope_layout layout, float mscale,
                    int inverse, void* y, int64_t syt, int64_t syh, void* stream) {
  if (x_dt != SS_F32 && x_dt != SS_BF16) return fail(SS_ERR_DTYPE, "x must be F32 or BF16");
  if (T < 0 || H < 0 || D < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (layout != SS_ROPE_HALF && layout != SS_ROPE_INTERLEAVED) return fail(SS_ERR_UNSUPPORTED, "unknown layout %d", (int)layout);
  if (T == 0 || H == 0 || D == 0) return ok();
  if (rot_dim < 2 || rot_dim > D || rot_dim % 2 != 0)
    return fail(SS_ERR_SHAPE, "rot_dim=%lld must be even and within 2..%lld", (long long)rot_dim, (long long)D);
  if (T > 0x7FFFFFFF || H * D > 0x7FFFFFF || H > 0x7FFFFFF || D > 0x7FFFFFF) return fail(SS_ERR_SHAPE, "too large");
  // the stride of a single token or head is never taken
  if (T == 1) sxt = syt = D;
  if (H == 1) sxh = syh = D;
  if (sxt < 0 || sxh < 0 || syt < 0 || syh < 0) return fail(SS_ERR_SHAPE, "negative stride");
  if (syh < D || syt < D) return fail(SS_ERR_SHAPE, "y: strides below D=%lld", (long long)D);
  if (!x || !y || !pos || !steps) return fail(SS_ERR_NULL, "x, y, pos and steps are required");
  if (x == y && (sxt != syt || sxh != syh)) return fail(SS_ERR_SHAPE, "in place needs equal strides");
  if (!std::isfinite(mscale)) return fail(SS_ERR_SHAPE, "mscale must be finite");
  const int es = esize(x_dt);
  if ((uintptr_t)x % es || (uintptr_t)y % es || (uintptr_t)pos % 4 || (uintptr_t)steps % 8)
    return fail(SS_ERR_ALIGN, "a pointer is not aligned to its elements");
  ss::RotaryArgs a{x, y, pos, steps, T, sxt, sxh, syt, syh, (int)H, (int)D, (int)rot_dim, layout == SS_ROPE_HALF,
                   mscale, inverse ? -mscale : mscale};
  return hip_status(ss::launch_rotary(x_dt == SS_BF16, a, (hipStream_t)stream), "ss_rotary launch");
}

namespace {

constexpr int64_t kMostWindow = 1 << 30;  // wider windows, and more first tokens, than any sequence has keys

int64_t attn_workspace(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t window, int64_t sinks) {
  if (Tq < 0 || Tk < 0 || B < 0 || Hq < 0 || Hkv < 0 || D < 0 || (Hkv > 0 && Hq % Hkv != 0)) return -1;
  if (Tq == 0 || Tk == 0 || B == 0 || Hq == 0 || Hkv == 0 || D == 0) return 0;
  if (Tq > 0x7FFFFFFF || Tk > 0x7FFFFFFF || B > 0x7FFFFFFF || Hq > 0xFFFF || D > 128 || Tq * (Hq / Hkv) > 0x7FFFFF00LL)
    return -1;
  return ss::attn_workspace_bytes(Tq, Tk, B, Hq, Hkv, D, window, sinks);
}

// What every attention call asks of its heads, scale and window (window and sinks are clamped).
ss_status check_heads(int64_t Hq, int64_t Hkv, int64_t D, float scale, int causal, int64_t* window, int64_t* sinks) {
  if (Hkv == 0 || Hq % Hkv != 0)
    return fail(SS_ERR_SHAPE, "%lld query heads do not divide into %lld key heads", (long long)Hq, (long long)Hkv);
  if (D < 8 || D > 128 || D % 8 != 0) return fail(SS_ERR_UNSUPPORTED, "D=%lld must be a multiple of 8 within 8..128", (long long)D);
  if (!(scale > 0) || !std::isfinite(scale * 1.5f)) return fail(SS_ERR_SHAPE, "scale must be positive and finite");
  if (*window < 0 || *sinks < 0) return fail(SS_ERR_SHAPE, "window and sinks must not be negative");
  if (*window > 0 && !causal) return fail(SS_ERR_UNSUPPORTED, "a window needs the causal mask");
  *window = *window < kMostWindow ? *window : kMostWindow;
  *sinks = *window == 0 ? 0 : *sinks < kMostWindow ? *sinks : kMostWindow;
  return SS_OK;
}

struct Op { const char* name; const void* p; int64_t st, sh; bool used; };
ss_status check_rows(const Op& t) {
  if (!t.used) return SS_OK;
  if (!t.p) return fail(SS_ERR_NULL, "%s is NULL", t.name);
  if (t.st < 0 || t.sh < 0) return fail(SS_ERR_SHAPE, "%s: negative stride", t.name);
  if (!aligned16(t.p) || t.st % 8 || t.sh % 8)
    return fail(SS_ERR_ALIGN, "%s: pointer and strides must be 16-byte aligned", t.name);
  return SS_OK;
}

ss_status check_workspace(const void* workspace, int64_t ws_bytes, int64_t need) {
  if (need <= 0) return SS_OK;
  if (!workspace) return fail(SS_ERR_NULL, "workspace is NULL (%lld bytes needed)", (long long)need);
  if (!aligned16(workspace)) return fail(SS_ERR_ALIGN, "workspace is not 16-byte aligned");
  if (ws_bytes < need) return fail(SS_ERR_SHAPE, "workspace of %lld bytes, %lld needed", (long long)ws_bytes, (long long)need);
  return SS_OK;
}

ss_status attn_call(const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
                    int64_t svt, int64_t svh, void* o, int64_t sot, int64_t soh, float* lse, int64_t Tq, int64_t Tk,
                    int64_t B, int64_t Hq, int64_t Hkv, int64_t D, const int32_t* cu_q, const int32_t* cu_k,
                    const int32_t* k_len, float scale, int causal, int64_t window, int64_t sinks, void* workspace,
                    int64_t ws_bytes, void* stream) {
  if (Tq < 0 || Tk < 0 || B < 0 || Hq < 0 || Hkv < 0 || D < 0 || ws_bytes < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (Tq == 0 || B == 0 || Hq == 0) return ok();
  if (const ss_status s = check_heads(Hq, Hkv, D, scale, causal, &window, &sinks); s != SS_OK) return s;
  if (Tq > 0x7FFFFFFF || Tk > 0x7FFFFFFF || B > 0xFFFFFFF || Hq > 0xFFFF || Tq * (Hq / Hkv) > 0x7FFFFF00LL ||
      !ss::attn_fits(Tq, Tk, B, Hq, Hkv, window, sinks))
    return fail(SS_ERR_SHAPE, "too large");
  if ((!cu_q || !cu_k) && B != 1) return fail(SS_ERR_NULL, "cu_q and cu_k are required with %lld sequences", (long long)B);
  // the stride of a single token or head is never taken
  if (Tq <= 1) sqt = sot = D;
  if (Tk <= 1) skt = svt = D;
  if (Hq <= 1) sqh = soh = D;
  if (Hkv <= 1) skh = svh = D;
  for (const Op& t : {Op{"q", q, sqt, sqh, true}, Op{"k", k, skt, skh, Tk > 0}, Op{"v", v, svt, svh, Tk > 0},
                      Op{"o", o, sot, soh, true}})
    if (const ss_status s = check_rows(t); s != SS_OK) return s;
  if (sot < D || soh < D) return fail(SS_ERR_SHAPE, "o: strides below D=%lld", (long long)D);
  // a tile's lane offsets are 32-bit
  if (Tk > 0 && (skt >= (1 << 24) || svt >= (1 << 24))) return fail(SS_ERR_UNSUPPORTED, "token strides of k and v must be below 2^24");
  if ((uintptr_t)cu_q % 4 || (uintptr_t)cu_k % 4 || (uintptr_t)k_len % 4 || (uintptr_t)lse % 4)
    return fail(SS_ERR_ALIGN, "a pointer is not aligned to its elements");
  const int64_t need = ss::attn_workspace_bytes(Tq, Tk, B, Hq, Hkv, D, window, sinks);
  if (const ss_status s = check_workspace(workspace, ws_bytes, need); s != SS_OK) return s;
  ss::AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.k_len = k_len;
  a.sqt = sqt; a.sqh = sqh; a.skt = skt; a.skh = skh; a.svt = svt; a.svh = svh; a.sot = sot; a.soh = soh;
  a.Tq = Tq;
  a.Tk = Tk;
  a.B = (int)B;
  a.Hkv = (int)Hkv;
  a.G = (int)(Hq / Hkv);
  a.D = (int)D;
  a.c = scale * 1.44269504088896340736f;
  a.causal = causal != 0;
  a.window = (int)window;
  a.sinks = (int)sinks;
  return hip_status(ss::launch_attn(a, need > 0 ? workspace : nullptr, (hipStream_t)stream), "ss_attn launch");
}

// A paged cache and its table for B sequences; `s`: the strides as the kernels take them (of a single page, key or head,
// which are never taken, those of adjacent rows). `write`: its rows must not overlap.
ss_status check_paged(const ss_paged_kv* kv, int64_t Hkv, int64_t D, int64_t B, bool write, ss_paged_kv* s) {
  if (!kv) return fail(SS_ERR_NULL, "the cache is NULL");
  *s = *kv;
  if (s->pages < 0 || s->page < 1 || s->table_cols < 0) return fail(SS_ERR_SHAPE, "cache: pages, page or table_cols is out of range");
  if (s->pages > 0x7FFFFFFF || s->page > 0x7FFFFFFF || s->table_cols > 0x7FFFFFFF) return fail(SS_ERR_SHAPE, "cache: too large");
  if (Hkv <= 1) s->skh = s->svh = D;
  if (s->page <= 1) s->skt = s->svt = D;
  if (s->pages <= 1) s->skp = s->svp = D;
  for (const Op& t : {Op{"k pages", s->k, s->skt, s->skh, s->pages > 0}, Op{"v pages", s->v, s->svt, s->svh, s->pages > 0},
                      Op{"k pages", s->k, s->skp, s->skh, s->pages > 0}, Op{"v pages", s->v, s->svp, s->svh, s->pages > 0}})
    if (const ss_status e = check_rows(t); e != SS_OK) return e;
  for (int64_t x : {s->skp, s->svp}) if (x > 0xFFFFFFFFLL) return fail(SS_ERR_UNSUPPORTED, "cache: page strides must be below 2^32");
  for (int64_t x : {s->skt, s->svt}) if (x >= (1 << 24)) return fail(SS_ERR_UNSUPPORTED, "cache: key strides must be below 2^24");
  if (write && s->pages > 0)
    for (int64_t x : {s->skp, s->svp, s->skt, s->svt, s->skh, s->svh})
      if (x < D) return fail(SS_ERR_SHAPE, "cache: a stride below D=%lld", (long long)D);
  if (s->table_cols > 0) {
    if (!s->table) return fail(SS_ERR_NULL, "table is NULL");
    if ((uintptr_t)s->table % 4) return fail(SS_ERR_ALIGN, "table is not aligned to its elements");
    if (B > 1 && s->table_ld < s->table_cols)
      return fail(SS_ERR_SHAPE, "table: leading dimension %lld < %lld columns", (long long)s->table_ld, (long long)s->table_cols);
  }
  if (B <= 1) s->table_ld = s->table_cols;
  return SS_OK;
}

}  // namespace

int64_t ss_attn_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  return attn_workspace(Tq, Tk, B, Hq, Hkv, D, 0, 0);
}

ss_status ss_attn(const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
                  int64_t svt, int64_t svh, void* o, int64_t sot, int64_t soh, float* lse, int64_t Tq, int64_t Tk,
                  int64_t B, int64_t Hq, int64_t Hkv, int64_t D, const int32_t* cu_q, const int32_t* cu_k,
                  const int32_t* k_len, float scale, int causal, void* workspace, int64_t ws_bytes, void* stream) {
  return attn_call(q, sqt, sqh, k, skt, skh, v, svt, svh, o, sot, soh, lse, Tq, Tk, B, Hq, Hkv, D, cu_q, cu_k, k_len, scale,
                   causal, 0, 0, workspace, ws_bytes, stream);
}

int64_t ss_attn_window_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t window,
                                       int64_t sinks) {
  if (window < 0 || sinks < 0) return -1;
  window = window < kMostWindow ? window : kMostWindow;
  return attn_workspace(Tq, Tk, B, Hq, Hkv, D, window, window == 0 ? 0 : sinks < kMostWindow ? sinks : kMostWindow);
}

ss_status ss_attn_window(const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
                         int64_t svt, int64_t svh, void* o, int64_t sot, int64_t soh, float* lse, int64_t Tq, int64_t Tk,
                         int64_t B, int64_t Hq, int64_t Hkv, int64_t D, const int32_t* cu_q, const int32_t* cu_k,
                         const int32_t* k_len, float scale, int causal, int64_t window, int64_t sinks, void* workspace,
                         int64_t ws_bytes, void* stream) {
  return attn_call(q, sqt, sqh, k, skt, skh, v, svt, svh, o, sot, soh, lse, Tq, Tk, B, Hq, Hkv, D, cu_q, cu_k, k_len, scale,
                   causal, window, sinks, workspace, ws_bytes, stream);
}

ss_status ss_rmsnorm_act(const void* X, ss_dtype x_dt, int64_t M, int64_t K, int64_t ldx, const void* residual, int64_t ldr,
                         void* sum, int64_t lds, const void* w, ss_dtype w_dt, double eps, int n, ss_dtype y_dt, void* Y,
                         int64_t ldy, float* sx, void* stream) {
  if (n < 2 || n > 8) return fail(SS_ERR_PATTERN, "n=%d outside 2..8", n);
  if (x_dt != SS_F32 && x_dt != SS_BF16) return fail(SS_ERR_DTYPE, "input must be F32 or BF16");
  if (y_dt != SS_BF16 && y_dt != SS_I8 && y_dt != SS_FP8E4M3) return fail(SS_ERR_DTYPE, "output must be BF16, I8 or FP8E4M3");
  if (w && w_dt != SS_F32 && w_dt != x_dt) return fail(SS_ERR_DTYPE, "weights must be F32 or of the input's type");
  if (y_dt == SS_BF16 && n != 2) return fail(SS_ERR_PATTERN, "a BF16 output has no lift (n=%d)", n);
  if (y_dt == SS_BF16 && sx) return fail(SS_ERR_DTYPE, "a BF16 output has no scales");
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(SS_ERR_SHAPE, "eps must be finite and not negative");
  if (M < 0 || K < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (M > 0x7FFFFFFF || K > 0x7FFFFFF) return fail(SS_ERR_SHAPE, "too large");
  if (M == 0 || K == 0) return ok();
  const int64_t Kc = y_dt == SS_BF16 ? K : ss_lifted_k(K, n);
  const int es = esize(x_dt);
  ss_status s;
  if ((s = check_mat("X", X, M, K, ldx, es)) != SS_OK) return s;
  if (residual) {
    if ((s = check_mat("residual", residual, M, K, ldr, es)) != SS_OK) return s;
    if ((s = check_mat("sum", sum, M, K, lds, es)) != SS_OK) return s;
    if ((sum == X && lds != ldx) || (sum == residual && lds != ldr))
      return fail(SS_ERR_SHAPE, "sum: in place needs the input's leading dimension");
  } else if (sum) {
    return fail(SS_ERR_UNSUPPORTED, "sum without a residual");
  }
  if ((s = check_mat("Y", Y, M, Kc, ldy, esize(y_dt))) != SS_OK) return s;
  if (Y == X || (residual && (Y == residual || Y == sum))) return fail(SS_ERR_UNSUPPORTED, "Y must not overlap another operand");
  if (y_dt != SS_BF16 && !sx) return fail(SS_ERR_NULL, "sx is NULL");
  if (w && !aligned16(w)) return fail(SS_ERR_ALIGN, "w is not 16-byte aligned");
  ss::NormArgs a{};
  a.x = X; a.res = residual; a.w = w; a.sum = sum; a.y = Y; a.sx = sx;
  a.M = M; a.K = K; a.Kc = Kc; a.ldx = ldx; a.ldr = ldr; a.lds = lds; a.ldy = ldy;
  a.eps = eps;
  a.n = n;
  return hip_status(ss::launch_rmsnorm(x_dt == SS_BF16, w && w_dt == SS_BF16, out_code(y_dt), a, (hipStream_t)stream),
                    "ss_rmsnorm_act launch");
}

ss_status ss_paged_store(const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
                         int64_t svt, int64_t svh, int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, const int32_t* pos,
                         const int32_t* cu, const uint64_t* steps, int64_t rot_dim, ss_rope_layout layout, float mscale,
                         void* qo, int64_t sot, int64_t soh, const ss_paged_kv* cache, void* stream) {
  if (T < 0 || B < 0 || Hq < 0 || Hkv < 0 || D < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (layout != SS_ROPE_HALF && layout != SS_ROPE_INTERLEAVED) return fail(SS_ERR_UNSUPPORTED, "unknown layout %d", (int)layout);
  if (T == 0 || B == 0 || (Hkv == 0 && Hq == 0) || D == 0) return ok();
  if (Hkv == 0) return fail(SS_ERR_SHAPE, "query heads without key heads");
  if (D % 8 != 0) return fail(SS_ERR_UNSUPPORTED, "D=%lld must be a multiple of 8", (long long)D);
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0)
    return fail(SS_ERR_SHAPE, "rot_dim=%lld must be even and within 0..%lld", (long long)rot_dim, (long long)D);
  if (rot_dim == 0 && Hq > 0) return fail(SS_ERR_UNSUPPORTED, "query heads without a turn");
  if (!std::isfinite(mscale)) return fail(SS_ERR_SHAPE, "mscale must be finite");
  if (!cu && B != T) return fail(SS_ERR_NULL, "cu is required unless every sequence has one token");
  if (T > 0x7FFFFFFF || B > 0x7FFFFFF || D > 0xFFFF || Hq > 0xFFFF || Hkv > 0xFFFF || (Hq + 2 * Hkv) * D > 0x7FFFFFF)
    return fail(SS_ERR_SHAPE, "too large");
  // the stride of a single token or head is never taken
  if (T == 1) sqt = skt = svt = sot = D;
  if (Hq <= 1) sqh = soh = D;
  if (Hkv == 1) skh = svh = D;
  for (const Op& t : {Op{"q", q, sqt, sqh, Hq > 0}, Op{"k", k, skt, skh, true}, Op{"v", v, svt, svh, true},
                      Op{"the turned queries", qo, sot, soh, Hq > 0}}) {
    if (!t.used) continue;
    if (!t.p) return fail(SS_ERR_NULL, "%s: NULL", t.name);
    if (t.st < 0 || t.sh < 0) return fail(SS_ERR_SHAPE, "%s: negative stride", t.name);
    if ((uintptr_t)t.p % 2) return fail(SS_ERR_ALIGN, "%s: not aligned to its elements", t.name);
  }
  if (Hq > 0 && (sot < D || soh < D)) return fail(SS_ERR_SHAPE, "the turned queries: strides below D=%lld", (long long)D);
  if (Hq > 0 && q == qo && (sqt != sot || sqh != soh)) return fail(SS_ERR_SHAPE, "in place needs equal strides");
  if (!pos || (rot_dim > 0 && !steps)) return fail(SS_ERR_NULL, "pos and steps are required");
  if ((uintptr_t)pos % 4 || (uintptr_t)cu % 4 || (uintptr_t)steps % 8) return fail(SS_ERR_ALIGN, "a pointer is not aligned to its elements");
  ss_paged_kv c;
  if (const ss_status s = check_paged(cache, Hkv, D, B, true, &c); s != SS_OK) return s;
  ss::StoreArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.qo = static_cast<uint16_t*>(qo);
  a.kc = static_cast<uint16_t*>(c.k);
  a.vc = static_cast<uint16_t*>(c.v);
  a.pos = pos; a.cu = cu; a.table = c.table; a.steps = steps;
  a.T = T; a.B = B; a.ldt = c.table_ld;
  a.sqt = sqt; a.sqh = sqh; a.skt = skt; a.skh = skh; a.svt = svt; a.svh = svh; a.sot = sot; a.soh = soh;
  a.kp = c.skp; a.kt = c.skt; a.kh = c.skh; a.vp = c.svp; a.vt = c.svt; a.vh = c.svh;
  a.Hq = (int)Hq; a.Hkv = (int)Hkv; a.D = (int)D; a.rot = (int)rot_dim; a.half = layout == SS_ROPE_HALF;
  a.cols = (int)c.table_cols; a.pages = (int)c.pages; a.page = (int)c.page;
  a.mscale = mscale;
  return hip_status(ss::launch_paged_store(a, (hipStream_t)stream), "ss_paged_store launch");
}

int64_t ss_attn_paged_workspace_bytes(int64_t Tq, int64_t room, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t window,
                                      int64_t sinks) {
  if (Tq < 0 || room < 0 || B < 0 || Hq < 0 || Hkv < 0 || D < 0 || (Hkv > 0 && Hq % Hkv != 0) || window < 0 || sinks < 0) return -1;
  if (Tq == 0 || B == 0 || Hq == 0 || Hkv == 0 || D == 0) return 0;
  if (Tq > 0x7FFFFFFF || B > 0x7FFFFFFF || Hq > 0xFFFF || D > 128 || Tq * (Hq / Hkv) > 0x7FFFFF00LL) return -1;
  window = window < kMostWindow ? window : kMostWindow;
  return ss::flat_workspace_bytes(Tq, room, room, B, Hq, Hkv, D, window, window == 0 ? 0 : sinks < kMostWindow ? sinks : kMostWindow);
}

ss_status ss_attn_paged(const void* q, int64_t sqt, int64_t sqh, const ss_paged_kv* cache, void* o, int64_t sot, int64_t soh,
                        float* lse, int64_t Tq, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, const int32_t* cu_q,
                        const int32_t* k_len, float scale, int causal, int64_t window, int64_t sinks, void* workspace,
                        int64_t ws_bytes, void* stream) {
  if (Tq < 0 || B < 0 || Hq < 0 || Hkv < 0 || D < 0 || ws_bytes < 0) return fail(SS_ERR_SHAPE, "negative size");
  if (Tq == 0 || B == 0 || Hq == 0) return ok();
  ss_status s;
  if ((s = check_heads(Hq, Hkv, D, scale, causal, &window, &sinks)) != SS_OK) return s;
  if (Tq > 0x7FFFFFFF || B > 0xFFFFFFF || Hq > 0xFFFF || Tq * (Hq / Hkv) > 0x7FFFFF00LL || !ss::flat_fits(Tq, B, Hq, Hkv))
    return fail(SS_ERR_SHAPE, "too large");
  if (!cu_q && B != Tq && B != 1) return fail(SS_ERR_NULL, "cu_q is required unless every sequence has one token");
  if (Tq == 1) sqt = sot = D;
  if (Hq == 1) sqh = soh = D;
  for (const Op& t : {Op{"q", q, sqt, sqh, true}, Op{"o", o, sot, soh, true}})
    if ((s = check_rows(t)) != SS_OK) return s;
  if (sot < D || soh < D) return fail(SS_ERR_SHAPE, "o: strides below D=%lld", (long long)D);
  if (!k_len) return fail(SS_ERR_NULL, "k_len is NULL");
  if ((uintptr_t)cu_q % 4 || (uintptr_t)k_len % 4 || (uintptr_t)lse % 4) return fail(SS_ERR_ALIGN, "a pointer is not aligned to its elements");
  ss_paged_kv c;
  if ((s = check_paged(cache, Hkv, D, B, false, &c)) != SS_OK) return s;
  const int64_t room = c.table_cols * c.page;
  const int64_t need = ss::flat_workspace_bytes(Tq, room, room, B, Hq, Hkv, D, window, sinks);
  if ((s = check_workspace(workspace, ws_bytes, need)) != SS_OK) return s;
  ss::FlatArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(c.k);
  a.v = static_cast<const uint16_t*>(c.v);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.cu_q = cu_q; a.k_len = k_len; a.table = c.table;
  a.sqt = sqt; a.sqh = sqh; a.sot = sot; a.soh = soh;
  a.skp = (uint32_t)c.skp; a.skt = (uint32_t)c.skt; a.skh = c.skh; a.svp = (uint32_t)c.svp; a.svt = (uint32_t)c.svt; a.svh = c.svh;
  a.Tq = Tq; a.ldt = c.table_ld;
  a.B = (int)B; a.Hkv = (int)Hkv; a.G = (int)(Hq / Hkv); a.D = (int)D;
  a.pages = (int)c.pages; a.page = (int)c.page; a.cols = (int)c.table_cols;
  a.c = scale * 1.44269504088896340736f;
  a.causal = causal != 0;
  a.window = (int)window;
  a.sinks = (int)sinks;
  a.paged = 1;
  return hip_status(ss::launch_flat(a, room, room, need > 0 ? workspace : nullptr, (hipStream_t)stream), "ss_attn_paged launch");
}

}  // extern "C"
