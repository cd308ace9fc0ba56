// native_call.cpp — the short way from torch tensors to the MXFP4, 8-bit, layer
// norm and gradient entry points of libbiasact.so.  The library's small calls take the GPU 2 to 5 us; their
// checks and marshalling in Python take 1.6 us (quantise) to 3 us (product) of
// host time beside a launch's 2 to 3, in C++ 0.1 to 0.2.
//
// Each function makes the call and returns True, or the library's status where
// that is not BA_OK; it returns False without having called anything when an
// argument is not what the call takes, and the binding then goes through its own
// checks, which say what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "biasact.h"

namespace {

decltype(&mxfp4_quantize) p_quantize = nullptr;
decltype(&mxfp4_dequantize) p_dequantize = nullptr;
decltype(&gemm_mxfp4_bias_act) p_gemm = nullptr;
decltype(&gemm_mxfp4_bias_add_act) p_gemm_add = nullptr;

decltype(&fp8_quantize) p_f8_quantize = nullptr;
decltype(&fp8_dequantize) p_f8_dequantize = nullptr;
decltype(&gemm_fp8_bias_act) p_f8_gemm = nullptr;
decltype(&gemm_fp8_bias_add_act) p_f8_gemm_add = nullptr;
decltype(&bias_act_grad) p_act_grad = nullptr;
decltype(&layer_norm) p_norm = nullptr;
decltype(&layer_norm_grad) p_norm_grad = nullptr;

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool on_device(const at::Tensor& t) { return t.is_cuda() && t.is_contiguous(); }

// BA_* code of a floating-point tensor, or -1
int float_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return BA_F32;
    case at::kHalf: return BA_F16;
    case at::kBFloat16: return BA_BF16;
    default: return -1;
  }
}

// codes [rows, 64 g] and scales [rows, 4 g], uint8 on the device
bool packed(const at::Tensor* c, const at::Tensor* s, int64_t* rows, int64_t* g) {
  if (!c || !s || c->scalar_type() != at::kByte || s->scalar_type() != at::kByte || c->dim() != 2 || s->dim() != 2)
    return false;
  *rows = s->size(0);
  *g = s->size(1) / 4;
  return s->size(1) % 4 == 0 && c->size(0) == *rows && c->size(1) == 64 * *g && on_device(*c) && on_device(*s);
}

constexpr int kNotTaken = -1;      // no call made; else the call's status

hipStream_t current_stream() { return c10::hip::getCurrentHIPStream().stream(); }

// (X, codes, scales, axis)
template <bool BACK>
int quantize(PyObject* const* a) {
  const at::Tensor *X = tensor(a[0]), *c = tensor(a[1]), *s = tensor(a[2]);
  if (!X || !PyLong_CheckExact(a[3])) return kNotTaken;
  const long axis = PyLong_AsLong(a[3]);
  int64_t rows, g;
  if ((axis != 0 && axis != 1) || X->dim() != 2 || !on_device(*X) || !packed(c, s, &rows, &g)) return kNotTaken;
  const int64_t xr = X->size(axis == 1 ? 0 : 1), K = X->size(axis == 1 ? 1 : 0);
  const int dt = float_code(*X);
  if (xr != rows || (K + 127) / 128 != g || dt < 0) return kNotTaken;
  return BACK ? p_dequantize(c->data_ptr(), s->data_ptr(), X->data_ptr(), rows, K, (int)axis, dt, current_stream())
              : p_quantize(X->data_ptr(), c->data_ptr(), s->data_ptr(), rows, K, (int)axis, dt, current_stream());
}

int act_code(PyObject* o) {
  static const char* const names[] = {"none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"};
  if (!PyUnicode_CheckExact(o)) return -1;
  const char* s = PyUnicode_AsUTF8(o);
  for (int i = 0; s && i < 6; ++i)
    if (strcmp(s, names[i]) == 0) return i;
  return -1;
}

// (A, a_scales or None, B, b_scales, bias or None, R or None, C, act, alpha)
int gemm(PyObject* const* a) {
  const at::Tensor *A = tensor(a[0]), *B = tensor(a[2]), *Bs = tensor(a[3]), *C = tensor(a[6]);
  const at::Tensor *As = nullptr, *bias = nullptr, *R = nullptr;
  int64_t M, N, K, g;
  if (!A || !C || C->dim() != 2 || !packed(B, Bs, &N, &g)) return kNotTaken;
  int ta = BA_MXFP4, tb = BA_F32;
  if (a[1] != Py_None) {
    int64_t ga;
    As = tensor(a[1]);
    if (!packed(A, As, &M, &ga) || ga != g) return kNotTaken;
    K = 128 * g;
  } else {
    ta = float_code(*A);
    if (A->dim() != 2 || !on_device(*A) || (ta != BA_F16 && ta != BA_BF16)) return kNotTaken;
    M = A->size(0);
    K = A->size(1);
    if ((K + 127) / 128 != g) return kNotTaken;
  }
  const int tc = float_code(*C);
  if (tc < 0 || C->size(0) != M || C->size(1) != N || !on_device(*C)) return kNotTaken;
  if (a[4] != Py_None) {
    bias = tensor(a[4]);
    if (!bias || bias->numel() != N || !on_device(*bias) || (tb = float_code(*bias)) < 0) return kNotTaken;
  }
  if (a[5] != Py_None) {
    R = tensor(a[5]);
    if (!R || R->sizes() != C->sizes() || R->scalar_type() != C->scalar_type() || !on_device(*R)) return kNotTaken;
  }
  const int act = act_code(a[7]);
  const double alpha = PyFloat_CheckExact(a[8]) ? PyFloat_AS_DOUBLE(a[8]) : 0.0;
  if (act < 0 || !PyFloat_CheckExact(a[8])) return kNotTaken;
  const uint32_t dt = BA_DTYPES(ta, BA_MXFP4, tb, tc);
  void* const as = As ? As->data_ptr() : nullptr;
  void* const bp = bias ? bias->data_ptr() : nullptr;
  return R ? p_gemm_add(A->data_ptr(), as, B->data_ptr(), Bs->data_ptr(), bp, R->data_ptr(), C->data_ptr(), M, N, K,
                        dt, act, (float)alpha, current_stream())
           : p_gemm(A->data_ptr(), as, B->data_ptr(), Bs->data_ptr(), bp, C->data_ptr(), M, N, K, dt, act, (float)alpha,
                    current_stream());
}

// ---- 8-bit operands, layer norm, gradients ------------------------------------------
// These calls also want their tensors on the current device, whose current stream
// they are queued on.

bool here(const at::Tensor& t) { return on_device(t) && t.get_device() == c10::hip::current_device(); }

int f8_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat8_e4m3fn: return BA_F8E4M3;
    case at::kFloat8_e5m2: return BA_F8E5M2;
    default: return -1;
  }
}

// codes [rows, 128 kb] in 8-bit floating point and scales [rows or ceil(rows / 128), 4 ceil(kb / 4)] in uint8
bool f8_packed(const at::Tensor* c, const at::Tensor* s, int64_t* rows, int64_t* kb, int* block_rows) {
  if (!c || !s || f8_code(*c) < 0 || s->scalar_type() != at::kByte || c->dim() != 2 || s->dim() != 2) return false;
  *rows = c->size(0);
  *kb = c->size(1) / 128;
  if (c->size(1) % 128 != 0 || s->size(1) != (*kb + 3) / 4 * 4 || !here(*c) || !here(*s)) return false;
  if (s->size(0) == *rows) *block_rows = 1;
  else if (s->size(0) == (*rows + 127) / 128) *block_rows = 128;
  else return false;
  return true;
}

// An optional tensor (None: null) of the type that dt gives, or that it gives dt where dt is -1; of n values
bool optional(PyObject* o, int64_t n, int* dt, void** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || t->numel() != n || !here(*t)) return false;
  const int code = float_code(*t);
  if (code < 0 || (*dt >= 0 && code != *dt)) return false;
  *dt = code;
  *p = t->data_ptr();
  return true;
}

// (X, codes, scales, axis)
template <bool BACK>
int f8_quantize(PyObject* const* a) {
  const at::Tensor *X = tensor(a[0]), *c = tensor(a[1]), *s = tensor(a[2]);
  if (!X || !PyLong_CheckExact(a[3])) return kNotTaken;
  const long axis = PyLong_AsLong(a[3]);
  int64_t rows, kb;
  int block;
  if ((axis != 0 && axis != 1) || X->dim() != 2 || !here(*X) || !f8_packed(c, s, &rows, &kb, &block)) return kNotTaken;
  const int64_t xr = X->size(axis == 1 ? 0 : 1), K = X->size(axis == 1 ? 1 : 0);
  const int dt = float_code(*X);
  if (xr != rows || (K + 127) / 128 != kb || dt < 0) return kNotTaken;
  const uint32_t dts = BA_DTYPES(dt, f8_code(*c), 0, 0);
  return BACK ? p_f8_dequantize(c->data_ptr(), s->data_ptr(), X->data_ptr(), rows, K, (int)axis, block, dts, current_stream())
              : p_f8_quantize(X->data_ptr(), c->data_ptr(), s->data_ptr(), rows, K, (int)axis, block, dts, current_stream());
}

// (A, a_scales, B, b_scales, bias or None, R or None, Z or None, C, act, alpha)
template <uint32_t SUMS>
int f8_gemm(PyObject* const* a) {
  const at::Tensor *A = tensor(a[0]), *B = tensor(a[2]), *C = tensor(a[7]);
  int64_t M, N, ka, kb;
  int block_a, block_b;
  const at::Tensor *As = tensor(a[1]), *Bs = tensor(a[3]);
  if (!f8_packed(A, As, &M, &ka, &block_a) || !f8_packed(B, Bs, &N, &kb, &block_b) || ka != kb) return kNotTaken;
  if (!C || C->dim() != 2 || C->size(0) != M || C->size(1) != N || !here(*C)) return kNotTaken;
  int tc = float_code(*C), tb = -1;
  void *bias, *rp, *zp;
  if (tc < 0 || !optional(a[4], N, &tb, &bias)) return kNotTaken;
  for (int i = 5; i < 7; ++i)                          // R and Z: C's shape and type
    if (a[i] != Py_None && (!tensor(a[i]) || tensor(a[i])->sizes() != C->sizes())) return kNotTaken;
  if (!optional(a[5], M * N, &tc, &rp) || !optional(a[6], M * N, &tc, &zp)) return kNotTaken;
  const int act = act_code(a[8]);
  if (act < 0 || !PyFloat_CheckExact(a[9])) return kNotTaken;
  const float alpha = (float)PyFloat_AS_DOUBLE(a[9]);
  const uint32_t dt = BA_DTYPES(f8_code(*A), f8_code(*B), tb < 0 ? BA_F32 : tb, (uint32_t)tc | SUMS);
  return a[5] != Py_None
             ? p_f8_gemm_add(A->data_ptr(), As->data_ptr(), block_a, B->data_ptr(), Bs->data_ptr(), block_b, bias, rp, zp,
                             C->data_ptr(), M, N, 128 * ka, dt, act, alpha, current_stream())
             : p_f8_gemm(A->data_ptr(), As->data_ptr(), block_a, B->data_ptr(), Bs->data_ptr(), block_b, bias, zp,
                         C->data_ptr(), M, N, 128 * ka, dt, act, alpha, current_stream());
}

// [rows, n] on this device in floating point; or its code is -1
int matrix(const at::Tensor* t, int64_t* rows, int64_t* n) {
  if (!t || t->dim() != 2 || !here(*t)) return -1;
  *rows = t->size(0);
  *n = t->size(1);
  return float_code(*t);
}

bool workspace(PyObject* o, void** p, size_t* bytes) {
  *p = nullptr;
  *bytes = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || !here(*t)) return false;
  *p = t->data_ptr();
  *bytes = t->nbytes();
  return true;
}

// (dY, Z or None, dZ or None, dbias or None, act, alpha, workspace or None)
int act_grad(PyObject* const* a) {
  int64_t M, N, m, n;
  const int dt = matrix(tensor(a[0]), &M, &N);
  if (dt < 0) return kNotTaken;
  for (int i = 1; i < 3; ++i)
    if (a[i] != Py_None && (matrix(tensor(a[i]), &m, &n) != dt || m != M || n != N)) return kNotTaken;
  int tb = -1;
  void *dbias, *ws;
  size_t bytes;
  if (!optional(a[3], N, &tb, &dbias) || !workspace(a[6], &ws, &bytes)) return kNotTaken;
  const int act = act_code(a[4]);
  if (act < 0 || !PyFloat_CheckExact(a[5])) return kNotTaken;
  auto ptr = [&](int i) { return a[i] == Py_None ? nullptr : tensor(a[i])->data_ptr(); };
  return p_act_grad(ptr(0), ptr(1), ptr(2), dbias, M, N, BA_DTYPES(dt, 0, tb < 0 ? BA_F32 : tb, 0), act,
                    (float)PyFloat_AS_DOUBLE(a[5]), ws, bytes, current_stream());
}

// (X, gamma or None, beta or None, Y, mean or None, rstd or None, eps)
int norm(PyObject* const* a) {
  int64_t rows, N, m, n;
  const int dx = matrix(tensor(a[0]), &rows, &N), dy = matrix(tensor(a[3]), &m, &n);
  if (dx < 0 || dy < 0 || m != rows || n != N || !PyFloat_CheckExact(a[6])) return kNotTaken;
  int dw = -1, f32 = BA_F32;
  void *gamma, *beta, *mean, *rstd;
  if (!optional(a[1], N, &dw, &gamma) || !optional(a[2], N, &dw, &beta) || !optional(a[4], rows, &f32, &mean) ||
      !optional(a[5], rows, &f32, &rstd))
    return kNotTaken;
  return p_norm(tensor(a[0])->data_ptr(), gamma, beta, tensor(a[3])->data_ptr(), (float*)mean, (float*)rstd, rows, N,
                (float)PyFloat_AS_DOUBLE(a[6]), BA_DTYPES(dx, dw < 0 ? BA_F32 : dw, 0, dy), current_stream());
}

// (dY, X, gamma or None, mean, rstd, dX, dgamma or None, dbeta or None, workspace or None)
int norm_grad(PyObject* const* a) {
  int64_t rows, N, m, n;
  const int dy = matrix(tensor(a[0]), &rows, &N), dx = matrix(tensor(a[1]), &m, &n);
  if (dx < 0 || dy < 0 || m != rows || n != N || matrix(tensor(a[5]), &m, &n) != dx || m != rows || n != N) return kNotTaken;
  int dw = -1, f32 = BA_F32;
  void *gamma, *mean, *rstd, *dgamma, *dbeta, *ws;
  size_t bytes;
  if (a[3] == Py_None || a[4] == Py_None || !optional(a[2], N, &dw, &gamma) || !optional(a[3], rows, &f32, &mean) ||
      !optional(a[4], rows, &f32, &rstd) || !optional(a[6], N, &dw, &dgamma) || !optional(a[7], N, &dw, &dbeta) ||
      !workspace(a[8], &ws, &bytes))
    return kNotTaken;
  return p_norm_grad(tensor(a[0])->data_ptr(), tensor(a[1])->data_ptr(), gamma, (float*)mean, (float*)rstd,
                     tensor(a[5])->data_ptr(), dgamma, dbeta, rows, N, BA_DTYPES(dx, dw < 0 ? BA_F32 : dw, 0, dy), ws, bytes,
                     current_stream());
}

// No C++ exception reaches the interpreter: a call that throws is one that the
// binding's own checks get to see.
template <int (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int rc = kNotTaken;
  if (p_quantize && p_f8_quantize && n == N) {
    try {
      rc = F(args);
    } catch (...) {
      rc = kNotTaken;
    }
    if (PyErr_Occurred()) PyErr_Clear();
  }
  return rc == kNotTaken || rc == BA_OK ? PyBool_FromLong(rc == BA_OK) : PyLong_FromLong(rc);
}

// Addresses of the four entry points, in the order above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_dequantize = reinterpret_cast<decltype(p_dequantize)>(p[1]);
  p_gemm = reinterpret_cast<decltype(p_gemm)>(p[2]);
  p_gemm_add = reinterpret_cast<decltype(p_gemm_add)>(p[3]);
  p_quantize = reinterpret_cast<decltype(p_quantize)>(p[0]);
  Py_RETURN_NONE;
}

// Addresses of the seven others, in the order above.
PyObject* bind_layer(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind_layer takes seven addresses");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_f8_dequantize = reinterpret_cast<decltype(p_f8_dequantize)>(p[1]);
  p_f8_gemm = reinterpret_cast<decltype(p_f8_gemm)>(p[2]);
  p_f8_gemm_add = reinterpret_cast<decltype(p_f8_gemm_add)>(p[3]);
  p_act_grad = reinterpret_cast<decltype(p_act_grad)>(p[4]);
  p_norm = reinterpret_cast<decltype(p_norm)>(p[5]);
  p_norm_grad = reinterpret_cast<decltype(p_norm_grad)>(p[6]);
  p_f8_quantize = reinterpret_cast<decltype(p_f8_quantize)>(p[0]);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction as_method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {
    {"bind", as_method(&bind), METH_FASTCALL, nullptr},
    {"quantize", as_method(&call<quantize<false>, 4>), METH_FASTCALL, nullptr},
    {"dequantize", as_method(&call<quantize<true>, 4>), METH_FASTCALL, nullptr},
    {"gemm", as_method(&call<gemm, 9>), METH_FASTCALL, nullptr},
    {"bind_layer", as_method(&bind_layer), METH_FASTCALL, nullptr},
    {"f8_quantize", as_method(&call<f8_quantize<false>, 4>), METH_FASTCALL, nullptr},
    {"f8_dequantize", as_method(&call<f8_quantize<true>, 4>), METH_FASTCALL, nullptr},
    {"f8_gemm", as_method(&call<f8_gemm<0u>, 10>), METH_FASTCALL, nullptr},
    {"f8_gemm_f32_sums", as_method(&call<f8_gemm<BA_SUMS_F32>, 10>), METH_FASTCALL, nullptr},
    {"act_grad", as_method(&call<act_grad, 7>), METH_FASTCALL, nullptr},
    {"norm", as_method(&call<norm, 7>), METH_FASTCALL, nullptr},
    {"norm_grad", as_method(&call<norm_grad, 9>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
