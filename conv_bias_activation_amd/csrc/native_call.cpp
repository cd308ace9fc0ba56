// native_call.cpp — the short way from torch tensors to the MXFP4 entry points
// of libbiasact.so.  The library's small calls take the GPU 2 to 5 us; their
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
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "biasact.h"

namespace {

decltype(&mxfp4_quantize) p_quantize = nullptr;
decltype(&mxfp4_dequantize) p_dequantize = nullptr;
decltype(&gemm_mxfp4_bias_act) p_gemm = nullptr;
decltype(&gemm_mxfp4_bias_add_act) p_gemm_add = nullptr;

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

// No C++ exception reaches the interpreter: a call that throws is one that the
// binding's own checks get to see.
template <int (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int rc = kNotTaken;
  if (p_quantize && n == N) {
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

template <class F>
PyCFunction as_method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {
    {"bind", as_method(&bind), METH_FASTCALL, nullptr},
    {"quantize", as_method(&call<quantize<false>, 4>), METH_FASTCALL, nullptr},
    {"dequantize", as_method(&call<quantize<true>, 4>), METH_FASTCALL, nullptr},
    {"gemm", as_method(&call<gemm, 9>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
