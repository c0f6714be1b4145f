// Native part of the Python binding for the MLP-block operators: reads what a call needs from
// its torch tensors, checks what the C-ABI cannot see of them, and calls the C-ABI.  These
// calls stand beside kernels of a few microseconds, and reading half a dozen tensors in Python
// takes about ten: layernorm of one row measured 7.8 us of host time that way (1.5 of them in
// ctypes).
//
// bind(path) takes the entry points from the library that the package has loaded.  Every
// function takes (handle, device, ...) and returns the C-ABI's status; bad tensors raise
// ValueError.  C++ exceptions end here.
#include <Python.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <stdexcept>
#include <string>

#include "gemm.h"

namespace {

decltype(&gemm_run_act) p_run_act;
decltype(&gemm_run_dact) p_run_dact;
decltype(&gemm_act_mx) p_act_mx;
decltype(&gemm_act_grad_mx) p_act_grad_mx;
decltype(&gemm_layernorm) p_layernorm;
decltype(&gemm_layernorm_grad) p_layernorm_grad;

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct BadType : std::runtime_error {
  using std::runtime_error::runtime_error;
};

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// The tensor behind an argument, or null for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw BadType(std::string(name) + " has to be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) throw Bad(std::string(name) + " is missing");
  return *t;
}

struct Mat {
  void* p = nullptr;
  int64_t ld = 0;
};
// A row-major M x N matrix (of a single row or without elements any stride does).
Mat mat(const at::Tensor& t, int64_t M, int64_t N, int device, const char* name) {
  if (t.dim() != 2 || t.size(0) != M || t.size(1) != N)
    throw Bad(std::string(name) + " has to be (" + std::to_string(M) + ", " + std::to_string(N) + "): got " +
              text(t.sizes()));
  if (t.get_device() != device)
    throw Bad(std::string(name) + " has to be on cuda:" + std::to_string(device) + ": got " + t.device().str());
  if (N > 1 && M > 0 && t.stride(1) != 1)
    throw Bad(std::string(name) + " has to be a row-major matrix: got strides " + text(t.strides()));
  return {t.data_ptr(), M > 1 ? t.stride(0) : std::max({t.stride(0), N, (int64_t)1})};
}
Mat mat_or(const at::Tensor* t, int64_t M, int64_t N, int device, const char* name, at::ScalarType type) {
  if (!t) return {};
  if (t->scalar_type() != type)
    throw Bad(std::string(name) + " has to be " + at::toString(type) + ": got " + at::toString(t->scalar_type()));
  return mat(*t, M, N, device, name);
}

int type_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return GEMM_TYPE_BF16;
  if (t.scalar_type() == at::kFloat) return GEMM_TYPE_F32;
  throw Bad(std::string(name) + " has to be bfloat16 or float32: got " + at::toString(t.scalar_type()));
}

// A contiguous vector of n values; float32, or with `type` of either activation type.
void* vec(const at::Tensor* t, int64_t n, int device, const char* name, int* type = nullptr) {
  if (!t) return nullptr;
  if (t->dim() != 1 || t->size(0) != n || !t->is_contiguous() || t->get_device() != device)
    throw Bad(std::string(name) + " has to be a contiguous vector of " + std::to_string(n) + " values on cuda:" +
              std::to_string(device) + ": got " + text(t->sizes()) + " on " + t->device().str());
  if (type)
    *type = type_of(*t, name);
  else if (t->scalar_type() != at::kFloat)
    throw Bad(std::string(name) + " has to be float32: got " + at::toString(t->scalar_type()));
  return t->data_ptr();
}

// A kept activation argument: bf16, or block-scaled E4M3 codes with their scales.
struct Kept {
  int kind = GEMM_Z_NONE;
  Mat z, s;
};
Kept kept(const at::Tensor& z, const at::Tensor* scales, int64_t M, int64_t N, int device) {
  if (!scales) return {GEMM_Z_BF16, mat_or(&z, M, N, device, "z (without scales)", at::kBFloat16), {}};
  if (z.scalar_type() != at::kFloat8_e4m3fn && z.scalar_type() != at::kByte)
    throw Bad(std::string("z with scales has to be float8_e4m3fn or uint8 codes: got ") +
              at::toString(z.scalar_type()));
  return {GEMM_Z_MX, mat(z, M, N, device, "z"), mat_or(scales, M, (N + 31) / 32, device, "z_scales", at::kByte)};
}

int act_of(PyObject* o) {
  static const char* const names[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  for (int i = 0; s && i < 5; ++i)
    if (std::strcmp(s, names[i]) == 0) return i;
  PyErr_Clear();
  throw Bad(std::string("act is one of none, relu, gelu, gelu_tanh, silu: got ") + (s ? s : "no text"));
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw BadType("a number is wanted");
  }
  return (float)v;
}
int flag(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw BadType(std::string(name) + " has to be a flag");
  }
  return v;
}
// (a handle's address and a device index, integers from the package itself)
gemm_handle_t handle(PyObject* o) {
  if (!PyLong_Check(o)) throw BadType("a handle's address is wanted");
  return (gemm_handle_t)PyLong_AsVoidPtr(o);
}
int device_of(PyObject* o) {
  if (!PyLong_Check(o)) throw BadType("a device index is wanted");
  return (int)PyLong_AsLong(o);
}

// C = op(A) op(B)
struct Product {
  int64_t M, N, K;
  Mat A, B, C;
  int tA, tB, dtype;
};
Product product(PyObject* oa, PyObject* ob, PyObject* oc, PyObject* ta, PyObject* tb, int device) {
  const at::Tensor &A = needed(oa, "A"), &B = needed(ob, "B"), &C = needed(oc, "C");
  if (A.dim() != 2 || B.dim() != 2 || C.dim() != 2) throw Bad("A, B and C have to be matrices");
  Product p;
  p.tA = flag(ta, "transA");
  p.tB = flag(tb, "transB");
  p.M = C.size(0);
  p.N = C.size(1);
  p.K = A.size(p.tA ? 0 : 1);
  if (A.size(p.tA ? 1 : 0) != p.M || B.size(p.tB ? 1 : 0) != p.K || B.size(p.tB ? 0 : 1) != p.N)
    throw Bad("op(A) times op(B) is not C's: A " + text(A.sizes()) + ", B " + text(B.sizes()) + ", C " +
              text(C.sizes()));
  const bool bf16 = A.scalar_type() == at::kBFloat16;
  if (A.scalar_type() != B.scalar_type() || (!bf16 && A.scalar_type() != at::kFloat8_e4m3fn))
    throw Bad(std::string("A and B have to be bfloat16 or float8_e4m3fn: got ") + at::toString(A.scalar_type()) + ", " +
              at::toString(B.scalar_type()));
  const bool f32 = type_of(C, "C") == GEMM_TYPE_F32;
  p.dtype = bf16 ? (f32 ? GEMM_BF16_F32 : GEMM_BF16_BF16) : (f32 ? GEMM_E4M3_F32 : GEMM_E4M3_BF16);
  p.A = mat(A, A.size(0), A.size(1), device, "A");
  p.B = mat(B, B.size(0), B.size(1), device, "B");
  p.C = mat(C, p.M, p.N, device, "C");
  return p;
}

// f(args) with the number of arguments checked and exceptions turned into Python's; the
// launch itself runs without the interpreter lock.
template <class F>
PyObject* call(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted: got %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong((long)f());
  } catch (const BadType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  }
  return nullptr;
}
template <class F>
gemm_status_t unlocked(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  const gemm_status_t st = f();
  PyEval_RestoreThread(s);
  return st;
}

// (handle, device, A, B, C, transA, transB, alpha, act, bias, residual, beta, z, z_scales)
PyObject* run_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 14, [&] {
    const int dev = device_of(a[1]);
    const Product p = product(a[2], a[3], a[4], a[5], a[6], dev);
    gemm_epilogue_t e{};
    e.act = act_of(a[8]);
    e.bias = vec(tensor(a[9], "bias"), p.N, dev, "bias", &e.bias_type);
    if (const at::Tensor* r = tensor(a[10], "residual")) {
      const Mat m = mat_or(r, p.M, p.N, dev, "residual", THPVariable_Unpack(a[4]).scalar_type());
      e.residual = m.p;
      e.ld_residual = m.ld;
      e.beta = number(a[11]);
    }
    if (const at::Tensor* z = tensor(a[12], "z")) {
      const Kept k = kept(*z, tensor(a[13], "z_scales"), p.M, p.N, dev);
      e.z_kind = k.kind;
      e.z = k.z.p;
      e.ld_z = k.z.ld;
      e.z_scales = (uint8_t*)k.s.p;
      e.ld_z_scales = k.s.ld;
    } else if (a[13] != Py_None) {
      throw Bad("z_scales without z");
    }
    const gemm_handle_t h = handle(a[0]);
    const float alpha = number(a[7]);
    return unlocked([&] {
      return p_run_act(h, p.tA, p.tB, p.M, p.N, p.K, alpha, p.A.p, p.A.ld, p.B.p, p.B.ld, &e, p.C.p, p.C.ld, p.dtype);
    });
  });
}

// (handle, device, A, B, C, z, z_scales, transA, transB, alpha, act, dbias)
PyObject* run_dact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&] {
    const int dev = device_of(a[1]);
    const Product p = product(a[2], a[3], a[4], a[7], a[8], dev);
    const Kept k = kept(needed(a[5], "z"), tensor(a[6], "z_scales"), p.M, p.N, dev);
    const int act = act_of(a[10]);
    float* db = (float*)vec(tensor(a[11], "dbias"), p.N, dev, "dbias");
    const gemm_handle_t h = handle(a[0]);
    const float alpha = number(a[9]);
    return unlocked([&] {
      return p_run_dact(h, p.tA, p.tB, p.M, p.N, p.K, alpha, p.A.p, p.A.ld, p.B.p, p.B.ld, act, k.kind, k.z.p, k.z.ld,
                        (const uint8_t*)k.s.p, k.s.ld, db, p.C.p, p.C.ld, p.dtype);
    });
  });
}

const at::Tensor* scales_of(PyObject* o) {
  const at::Tensor* s = tensor(o, "scales");
  if (!s) throw Bad("codes need their scales");
  return s;
}

// (handle, device, z, out, codes, scales, act)
PyObject* act_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 7, [&] {
    const int dev = device_of(a[1]);
    const at::Tensor& z = needed(a[2], "z");
    if (z.dim() != 2) throw Bad("z has to be a matrix");
    const int64_t M = z.size(0), N = z.size(1);
    const Mat zm = mat_or(&z, M, N, dev, "z", at::kBFloat16);
    const Mat om = mat_or(&needed(a[3], "out"), M, N, dev, "out", at::kBFloat16);
    const Kept k = kept(needed(a[4], "codes"), scales_of(a[5]), M, N, dev);
    const int act = act_of(a[6]);
    const gemm_handle_t h = handle(a[0]);
    return unlocked([&] {
      return p_act_mx(h, M, N, act, zm.p, zm.ld, om.p, om.ld, k.z.p, k.z.ld, (uint8_t*)k.s.p, k.s.ld);
    });
  });
}

// (handle, device, codes, scales, act, dh, dz, dbias, h)
PyObject* act_grad_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const int dev = device_of(a[1]);
    const at::Tensor& q = needed(a[2], "codes");
    if (q.dim() != 2) throw Bad("codes has to be a matrix");
    const int64_t M = q.size(0), N = q.size(1);
    const Kept k = kept(q, scales_of(a[3]), M, N, dev);
    const int act = act_of(a[4]);
    const Mat dh = mat_or(tensor(a[5], "dh"), M, N, dev, "dh", at::kBFloat16);
    const Mat dz = mat_or(tensor(a[6], "dz"), M, N, dev, "dz", at::kBFloat16);
    float* db = (float*)vec(tensor(a[7], "dbias"), N, dev, "dbias");
    const Mat hm = mat_or(tensor(a[8], "h"), M, N, dev, "h", at::kBFloat16);
    const gemm_handle_t h = handle(a[0]);
    return unlocked([&] {
      return p_act_grad_mx(h, M, N, act, k.z.p, k.z.ld, (const uint8_t*)k.s.p, k.s.ld, dh.p, dh.ld, dz.p, dz.ld, db,
                           hm.p, hm.ld);
    });
  });
}

// (handle, device, x, y, gamma, beta, eps, mean, rstd)
PyObject* layernorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const int dev = device_of(a[1]);
    const at::Tensor &x = needed(a[2], "x"), &y = needed(a[3], "y");
    if (x.dim() != 2) throw Bad("x has to be a matrix");
    const int64_t M = x.size(0), N = x.size(1);
    const Mat xm = mat(x, M, N, dev, "x"), ym = mat(y, M, N, dev, "y");
    int wt = GEMM_TYPE_F32, bt = GEMM_TYPE_F32;
    const void* g = vec(tensor(a[4], "gamma"), N, dev, "gamma", &wt);
    const void* b = vec(tensor(a[5], "beta"), N, dev, "beta", &bt);
    if (g && b && wt != bt) throw Bad("gamma and beta have to be of one type");
    if (!g) wt = bt;
    float* mean = (float*)vec(tensor(a[7], "mean"), M, dev, "mean");
    float* rstd = (float*)vec(tensor(a[8], "rstd"), M, dev, "rstd");
    const int xt = type_of(x, "x"), yt = type_of(y, "y");
    const gemm_handle_t h = handle(a[0]);
    const float eps = number(a[6]);
    return unlocked(
        [&] { return p_layernorm(h, M, N, xm.p, xm.ld, xt, g, b, wt, eps, ym.p, ym.ld, yt, mean, rstd); });
  });
}

// (handle, device, dy, x, mean, rstd, dx, gamma, dgamma, dbeta, residual)
PyObject* layernorm_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&] {
    const int dev = device_of(a[1]);
    const at::Tensor &dy = needed(a[2], "dy"), &x = needed(a[3], "x");
    if (x.dim() != 2) throw Bad("x has to be a matrix");
    const int64_t M = x.size(0), N = x.size(1);
    const Mat dym = mat(dy, M, N, dev, "dy"), xm = mat(x, M, N, dev, "x");
    const Mat dx = mat_or(&needed(a[6], "dx"), M, N, dev, "dx", x.scalar_type());
    const Mat res = mat_or(tensor(a[10], "residual"), M, N, dev, "residual", x.scalar_type());
    const float* mean = (const float*)vec(&needed(a[4], "mean"), M, dev, "mean");
    const float* rstd = (const float*)vec(&needed(a[5], "rstd"), M, dev, "rstd");
    int wt = GEMM_TYPE_F32;
    const void* g = vec(tensor(a[7], "gamma"), N, dev, "gamma", &wt);
    float* dg = (float*)vec(tensor(a[8], "dgamma"), N, dev, "dgamma");
    float* db = (float*)vec(tensor(a[9], "dbeta"), N, dev, "dbeta");
    const int xt = type_of(x, "x"), yt = type_of(dy, "dy");
    const gemm_handle_t h = handle(a[0]);
    return unlocked([&] {
      return p_layernorm_grad(h, M, N, dym.p, dym.ld, yt, xm.p, xm.ld, xt, mean, rstd, g, wt, res.p, res.ld, dx.p,
                              dx.ld, dg, db);
    });
  });
}

// bind(path): the entry points of the loaded library
PyObject* bind(PyObject*, PyObject* arg) {
  const char* path = PyUnicode_AsUTF8(arg);
  if (!path) return nullptr;
  void* lib = dlopen(path, RTLD_NOW | RTLD_NOLOAD);
  auto take = [&](auto& f, const char* name) {
    f = lib ? (std::remove_reference_t<decltype(f)>)dlsym(lib, name) : nullptr;
    return f != nullptr;
  };
  if (!take(p_run_act, "gemm_run_act") || !take(p_run_dact, "gemm_run_dact") || !take(p_act_mx, "gemm_act_mx") ||
      !take(p_act_grad_mx, "gemm_act_grad_mx") || !take(p_layernorm, "gemm_layernorm") ||
      !take(p_layernorm_grad, "gemm_layernorm_grad")) {
    PyErr_Format(PyExc_RuntimeError, "%s is not loaded, or lacks an entry point", path);
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void*)f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr}, FAST(run_act),   FAST(run_dact),       FAST(act_mx),
                         FAST(act_grad_mx),               FAST(layernorm), FAST(layernorm_grad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Native part of the binding.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
