// Python binding of the calls around a layer's products: spgemm_tiled_epilogue, rotary, attn.
//
// These run between products, often on one token, where a call's own time on the host is what counts: checking the
// tensors and marshalling some twenty arguments in Python took 7-12 us a call, the kernels 4-11 us. Here both take
// 0.4-0.6 us, an output from torch's allocator 0.7-1.1 more; the launch, 2.9 us, is the rest of a call's 4-5 us. Nothing is
// computed: sizes, strides, types and devices are checked (the C entry points cannot see how large a tensor behind a
// pointer is), outputs and workspaces come from torch, the call goes to the C ABI on the current stream of the tensors' GPU.
//
// No exception leaves a function: torch's become Python exceptions, a refused call raises the package's SSError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "ss.h"

namespace {

PyObject* g_error = nullptr;  // SSError(status, detail)

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(int status, const std::string& detail) {
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", status, detail.c_str()) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, detail.c_str());
  }
  throw Refused{};
}
void check(ss_status s) {
  if (s != SS_OK) refuse(s, ss_last_error());
}

// a required tensor, or with `optional` NULL for None
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None) {
    if (!optional) refuse(SS_ERR_NULL, std::string(name) + " is None");
    return nullptr;
  }
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: needs a tensor, has %s", name, Py_TYPE(o)->tp_name);
    throw Refused{};
  }
  return &THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}
void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
    throw Refused{};
  }
}

std::string shape(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}
void need_type(const at::Tensor* t, at::ScalarType want, const char* name) {
  if (t && t->scalar_type() != want)
    refuse(SS_ERR_DTYPE, std::string(name) + ": needs " + at::toString(want) + ", has " + at::toString(t->scalar_type()));
}
// [T, H, D], the values of a head adjacent
void need_heads(const at::Tensor* t, int64_t T, int64_t H, int64_t D, const char* name) {
  if (t->dim() != 3 || t->size(0) != T || t->size(1) != H || t->size(2) != D ||
      (t->stride(2) != 1 && D > 1 && t->numel() > 0))
    refuse(SS_ERR_SHAPE, std::string(name) + ": needs [" + std::to_string(T) + ", " + std::to_string(H) + ", " +
                             std::to_string(D) + "] with unit stride along the last dimension, has " + shape(*t));
}
void need_heads(const at::Tensor* t, const char* name) {
  if (t->dim() != 3) refuse(SS_ERR_SHAPE, std::string(name) + ": needs [tokens, heads, values], has " + shape(*t));
  need_heads(t, t->size(0), t->size(1), t->size(2), name);
}
// n values or more, adjacent
void need_vec(const at::Tensor* t, int64_t n, at::ScalarType type, const char* name, bool exact = false) {
  if (!t) return;
  need_type(t, type, name);
  if (!t->is_contiguous() || (exact ? t->dim() != 1 || t->numel() != n : t->numel() < n))
    refuse(SS_ERR_SHAPE, std::string(name) + ": needs " + std::to_string(n) + " contiguous values, has " + shape(*t));
}
void need_mat(const at::Tensor* t, int64_t rows, int64_t cols, const char* name) {
  if (t && (t->dim() != 2 || t->size(0) < rows || t->size(1) < cols || (t->size(0) > 0 && t->stride(1) != 1)))
    refuse(SS_ERR_SHAPE, std::string(name) + ": needs a row-major [" + std::to_string(rows) + ", >= " +
                             std::to_string(cols) + "] matrix, has " + shape(*t));
}
void need_bytes(const at::Tensor* t, int64_t n, const char* name) {
  if (t && (!t->is_contiguous() || (int64_t)t->nbytes() < n))
    refuse(SS_ERR_SHAPE, std::string(name) + ": needs " + std::to_string(n) + " contiguous bytes, has " +
                             std::to_string(t->nbytes()) + (t->is_contiguous() ? "" : " (not contiguous)"));
}
void same_gpu(const at::Device& dev, std::initializer_list<const at::Tensor*> ts) {
  if (dev.type() != at::kCUDA)
    refuse(SS_ERR_UNSUPPORTED, "tensor on " + dev.str() + ": the library runs on the GPU only");
  for (const at::Tensor* t : ts)
    if (t && t->device() != dev) refuse(SS_ERR_UNSUPPORTED, "tensor on " + t->device().str() + ", the call runs on " + dev.str());
}

// The tensors' GPU made the current one for a call (kernels launch on the current GPU), and its current stream.
struct Place {
  c10::DeviceGuard guard;
  void* stream;
  explicit Place(const at::Device& dev) : guard(dev), stream(c10::hip::getCurrentHIPStream(dev.index()).stream()) {}
};
template <typename T> T* ptr(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

// Body of a binding: what it returns, or the exception that ended it.
template <typename F> PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return THPVariable_Wrap(f());
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (x, pos, steps, layout, mscale, inverse, out)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> at::Tensor {
    count(n, 7);
    const at::Tensor *x = tensor(a[0], "x"), *pos = tensor(a[1], "pos"), *steps = tensor(a[2], "steps"),
                     *out = tensor(a[6], "out", true);
    need_heads(x, "x");
    const int64_t T = x->size(0), H = x->size(1), D = x->size(2);
    const bool bf16 = x->scalar_type() == at::kBFloat16;
    if (!bf16) need_type(x, at::kFloat, "x (or bf16)");
    need_vec(pos, T, at::kInt, "pos", true);
    need_vec(steps, steps->numel(), at::kLong, "steps", true);
    if (out) {
      need_heads(out, T, H, D, "out");
      need_type(out, x->scalar_type(), "out");
    }
    same_gpu(x->device(), {pos, steps, out});
    const Place at(x->device());
    at::Tensor y = out ? *out : at::empty({T, H, D}, x->options());
    check(ss_rotary(ptr<void>(x), bf16 ? SS_BF16 : SS_F32, T, H, D, x->stride(0), x->stride(1), ptr<int32_t>(pos),
                    ptr<uint64_t>(steps), 2 * steps->numel(), (ss_rope_layout)integer(a[3]), (float)number(a[4]),
                    truth(a[5]), y.data_ptr(), y.stride(0), y.stride(1), at.stream));
    return y;
  });
}

// (q, k, v, cu_q, cu_k, k_len, causal, scale or None, out, lse, workspace)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> at::Tensor {
    count(n, 11);
    const at::Tensor *q = tensor(a[0], "q"), *k = tensor(a[1], "k"), *v = tensor(a[2], "v"),
                     *cu_q = tensor(a[3], "cu_q", true), *cu_k = tensor(a[4], "cu_k", true),
                     *k_len = tensor(a[5], "k_len", true), *out = tensor(a[8], "out", true),
                     *lse = tensor(a[9], "lse", true), *ws = tensor(a[10], "workspace", true);
    need_heads(q, "q");
    need_heads(k, "k");
    const int64_t Tq = q->size(0), Hq = q->size(1), D = q->size(2), Tk = k->size(0), Hkv = k->size(1);
    need_heads(k, Tk, Hkv, D, "k");
    need_heads(v, Tk, Hkv, D, "v");
    if (out) need_heads(out, Tq, Hq, D, "out");
    need_type(q, at::kBFloat16, "q");
    need_type(k, at::kBFloat16, "k");
    need_type(v, at::kBFloat16, "v");
    need_type(out, at::kBFloat16, "out");
    if (lse) {
      need_type(lse, at::kFloat, "lse");
      if (lse->dim() != 2 || lse->size(0) != Hq || lse->size(1) != Tq || !lse->is_contiguous())
        refuse(SS_ERR_SHAPE, "lse: needs contiguous [" + std::to_string(Hq) + ", " + std::to_string(Tq) + "], has " + shape(*lse));
    }
    const int64_t B = cu_q ? cu_q->numel() - 1 : cu_k ? cu_k->numel() - 1 : 1;
    if (B < 0) refuse(SS_ERR_SHAPE, "cu_q and cu_k hold one value more than there are sequences");
    need_vec(cu_q, B + 1, at::kInt, "cu_q", true);
    need_vec(cu_k, B + 1, at::kInt, "cu_k", true);
    need_vec(k_len, B, at::kInt, "k_len", true);
    need_bytes(ws, 0, "workspace");
    same_gpu(q->device(), {k, v, cu_q, cu_k, k_len, out, lse, ws});
    const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)std::max<int64_t>(D, 1))) : (float)number(a[7]);
    const Place at(q->device());
    at::Tensor o = out ? *out : at::empty({Tq, Hq, D}, q->options());
    at::Tensor own;
    if (!ws) {
      const int64_t need = ss_attn_workspace_bytes(Tq, Tk, B, Hq, Hkv, D);
      if (need > 0) {
        own = at::empty({need}, q->options().dtype(at::kByte));
        ws = &own;
      }
    }
    check(ss_attn(ptr<void>(q), q->stride(0), q->stride(1), ptr<void>(k), k->stride(0), k->stride(1), ptr<void>(v),
                  v->stride(0), v->stride(1), o.data_ptr(), o.stride(0), o.stride(1), ptr<float>(lse), Tq, Tk, B, Hq, Hkv,
                  D, ptr<int32_t>(cu_q), ptr<int32_t>(cu_k), ptr<int32_t>(k_len), scale, truth(a[6]), ptr<void>(ws),
                  ws ? (int64_t)ws->nbytes() : 0, at.stream));
    return o;
  });
}

// (side, M, N, Kc, tvals, tmeta, dense, sx, sw, bias, act, gated, residual, y_dt, out, workspace)
PyObject* spgemm_tiled_epilogue(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> at::Tensor {
    count(n, 16);
    const ss_side side = (ss_side)integer(a[0]);
    const int64_t M = integer(a[1]), N = integer(a[2]), Kc = integer(a[3]);
    const at::Tensor *tv = tensor(a[4], "tvals"), *tm = tensor(a[5], "tmeta"), *dense = tensor(a[6], "dense"),
                     *sx = tensor(a[7], "sx", true), *sw = tensor(a[8], "sw", true), *bias = tensor(a[9], "bias", true),
                     *res = tensor(a[12], "residual", true), *out = tensor(a[14], "out", true),
                     *ws = tensor(a[15], "workspace", true);
    const bool gated = truth(a[11]);
    const int64_t y_code = integer(a[13]);
    if (y_code != SS_BF16 && y_code != SS_F32) refuse(SS_ERR_DTYPE, "the output must be bf16 or f32");
    const ss_dtype y_dt = (ss_dtype)y_code;
    const at::ScalarType y_type = y_dt == SS_BF16 ? at::kBFloat16 : at::kFloat;
    ss_dtype ab;
    switch (dense->scalar_type()) {
      case at::kChar: ab = SS_I8; break;
      case at::kFloat8_e4m3fn: ab = SS_FP8E4M3; break;
      case at::kBFloat16: ab = SS_BF16; break;
      default: refuse(SS_ERR_DTYPE, std::string("dense: needs int8, float8_e4m3fn or bf16, has ") + at::toString(dense->scalar_type()));
    }
    if (M < 0 || N < 0) refuse(SS_ERR_SHAPE, "negative size");
    const int64_t cols = gated ? N / 2 : N, rows = side == SS_SPARSE_X ? M : N, dn = side == SS_SPARSE_X ? N : M;
    need_bytes(tv, ss_tiled_vals_bytes(rows, Kc, ab), "tvals");
    need_bytes(tm, ss_tiled_meta_bytes(rows, Kc, ab), "tmeta");
    need_mat(dense, dn, Kc, "dense");
    need_vec(sx, M, at::kFloat, "sx");
    need_vec(sw, N, at::kFloat, "sw");
    need_vec(bias, N, at::kFloat, "bias");
    need_type(res, y_type, "residual");
    need_mat(res, M, cols, "residual");
    need_type(out, y_type, "out");
    need_mat(out, M, cols, "out");
    need_bytes(ws, 0, "workspace");
    same_gpu(dense->device(), {tv, tm, sx, sw, bias, res, out, ws});
    const Place at(dense->device());
    at::Tensor y = out ? *out : at::empty({M, cols}, dense->options().dtype(y_type));
    at::Tensor own;
    if (!ws) {
      const int64_t need = ss_spgemm_tiled_workspace_bytes(side, M, N, Kc, ab);
      if (need > 0) {
        own = at::empty({need}, dense->options().dtype(at::kByte));
        ws = &own;
      }
    }
    check(ss_spgemm_tiled_epilogue(side, M, N, Kc, ab, ptr<void>(tv), ptr<uint8_t>(tm), ptr<void>(dense), dense->stride(0),
                                   ptr<float>(sx), ptr<float>(sw), ptr<float>(bias), (ss_act)integer(a[10]), gated,
                                   ptr<void>(res), res ? res->stride(0) : 0, y_dt, y.data_ptr(), y.stride(0), ptr<void>(ws),
                                   ws ? (int64_t)ws->nbytes() : 0, at.stream));
    return y;
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"rotary", fast(rotary), METH_FASTCALL, nullptr},
                         {"attn", fast(attn), METH_FASTCALL, nullptr},
                         {"spgemm_tiled_epilogue", fast(spgemm_tiled_epilogue), METH_FASTCALL, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_ssbind", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__ssbind(void) { return PyModule_Create(&module_def); }
