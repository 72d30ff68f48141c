// binding.cpp -- argument marshalling of the per-layer, per-token calls (the 8-bit dense operators)
// as a CPython extension: tensor checks and the C ABI call without ctypes.  A decode step makes these
// calls once per layer, and their kernels take 2 to 8 us: checked from Python, a call of nine tensors
// costs the host as much as that again.
//
// The functions of the C ABI are called through the addresses that init() receives (taken from the
// loaded libscion.so), so that there is one copy of the library in the process.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/scion.h"

namespace {

using at::ScalarType;

struct Abi {
  decltype(&scion_rmsnorm_forward) rmsnorm;
  decltype(&scion_fp8_quantize_device) quantize;
  decltype(&scion_fp8_forward) forward;
  decltype(&scion_fp8_gated_forward) gated;
} abi;

enum Kind { kFloat, kBf16, kF32, kCodes, kScales };  // element types an argument may have

bool has_kind(ScalarType t, Kind k) {
  switch (k) {
    case kFloat: return t == at::kFloat || t == at::kBFloat16;
    case kBf16: return t == at::kBFloat16;
    case kF32: return t == at::kFloat;
    case kCodes: return t == at::kFloat8_e4m3fn || t == at::kByte;
    case kScales: return t == at::kFloat8_e8m0fnu || t == at::kByte;
  }
  return false;
}

const char* kind_name(Kind k) {
  static const char* names[] = {"float32 or bfloat16", "bfloat16", "float32", "float8_e4m3fn or uint8",
                                "float8_e8m0fnu or uint8"};
  return names[k];
}

// Reads the tensor arguments of one call; the first one that does not fit raises ValueError.
struct Args {
  int dev;
  bool ok = true;
  explicit Args(int d) : dev(d) {}

  void* tensor(PyObject* o, const char* name, Kind kind, int64_t numel, ScalarType* type = nullptr) {
    if (!ok) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_ValueError, "%s must be a tensor", name);
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous CUDA tensor on the current device", name);
      ok = false;
    } else if (!has_kind(t.scalar_type(), kind)) {
      PyErr_Format(PyExc_ValueError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()), kind_name(kind));
      ok = false;
    } else if (t.numel() != numel) {
      PyErr_Format(PyExc_ValueError, "%s has %lld elements, expected %lld", name, (long long)t.numel(), (long long)numel);
      ok = false;
    }
    if (!ok) return nullptr;
    if (type) *type = t.scalar_type();
    return t.data_ptr();
  }
  void* optional(PyObject* o, const char* name, Kind kind, int64_t numel, ScalarType* type = nullptr) {
    return o == Py_None ? nullptr : tensor(o, name, kind, numel, type);
  }
};

int abi_type(ScalarType t) { return t == at::kFloat ? SCION_F32 : SCION_BF16; }

// An int argument; values outside C int raise OverflowError like ctypes' callers expect of Python.
bool get_int(PyObject* o, int* v) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) return false;
  if (n < INT_MIN || n > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument out of the range of a C int");
    return false;
  }
  *v = int(n);
  return true;
}

// stream: None (torch's current one), an address, or an object with .cuda_stream
bool get_stream(PyObject* o, int dev, void** s) {
  if (o == Py_None) {
    *s = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream();
    return true;
  }
  PyObject* v = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!v) return false;
  *s = reinterpret_cast<void*>(PyLong_AsUnsignedLongLong(v));
  Py_DECREF(v);
  return !PyErr_Occurred();
}

bool get_handle(PyObject* o, const scion_fp8** h) {
  *h = reinterpret_cast<const scion_fp8*>(PyLong_AsUnsignedLongLong(o));
  return !PyErr_Occurred();
}

bool want(Py_ssize_t n, Py_ssize_t expected) {
  if (n == expected) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, n);
  return false;
}

int64_t groups(int64_t n) { return (n + 127) / 128; }

// rmsnorm(x, T, weight, eps, resid, resid_out, y, y_codes, y_scales, stream) -> status
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int T;
  void* s;
  if (!want(n, 10) || !get_int(a[1], &T)) return nullptr;
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const int dev = c10::cuda::current_device();
  if (!THPVariable_Check(a[2])) {
    PyErr_SetString(PyExc_ValueError, "weight must be a tensor");
    return nullptr;
  }
  const int64_t d = THPVariable_Unpack(a[2]).numel();
  Args g(dev);
  ScalarType xt = at::kFloat, rt, ot;
  const void* x = g.tensor(a[0], "x", kFloat, T * d, &xt);
  const void* w = g.tensor(a[2], "weight", kBf16, d);
  rt = ot = xt;
  const void* resid = g.optional(a[4], "resid", kFloat, T * d, &rt);
  ot = rt;
  void* resid_out = g.optional(a[5], "resid_out", kFloat, T * d, &ot);
  if (g.ok && resid && ot != rt) {
    PyErr_SetString(PyExc_ValueError, "resid and resid_out must have one dtype");
    return nullptr;
  }
  void* y = g.optional(a[6], "y", kBf16, T * d);
  void* yc = g.optional(a[7], "y_codes", kCodes, T * d);
  void* ys = g.optional(a[8], "y_scales", kScales, T * groups(d));
  if (!g.ok || !get_stream(a[9], dev, &s)) return nullptr;
  if (d > INT_MAX) return PyLong_FromLong(SCION_EINVAL);
  return PyLong_FromLong(abi.rmsnorm(x, abi_type(xt), resid, abi_type(ot), w, float(eps), T, int(d), resid_out, y,
                                     static_cast<uint8_t*>(yc), static_cast<uint8_t*>(ys), s));
  END_HANDLE_TH_ERRORS
}

// quantize(src, codes, scales, block_rows, stream) -> status
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int br;
  void* s;
  if (!want(n, 5) || !get_int(a[3], &br)) return nullptr;
  if (!THPVariable_Check(a[0]) || THPVariable_Unpack(a[0]).dim() != 2) {
    PyErr_SetString(PyExc_ValueError, "src must be a [rows, cols] tensor");
    return nullptr;
  }
  const int64_t rows = THPVariable_Unpack(a[0]).size(0), cols = THPVariable_Unpack(a[0]).size(1);
  const int dev = c10::cuda::current_device();
  Args g(dev);
  ScalarType st = at::kFloat;
  const void* src = g.tensor(a[0], "src", kFloat, rows * cols, &st);
  void* codes = g.tensor(a[1], "codes", kCodes, rows * cols);
  void* scales = g.tensor(a[2], "scales", kScales, (br > 1 ? (rows + br - 1) / br : rows) * groups(cols));
  if (!g.ok || !get_stream(a[4], dev, &s)) return nullptr;
  if (cols > INT_MAX) return PyLong_FromLong(SCION_EINVAL);
  return PyLong_FromLong(abi.quantize(abi_type(st), src, rows, int(cols), br, static_cast<uint8_t*>(codes),
                                      static_cast<uint8_t*>(scales), s));
  END_HANDLE_TH_ERRORS
}

// The common part of the two products: (x_codes, x_scales, T, handle, n, k, device, ...).
struct Product {
  int T = 0, n = 0, k = 0, dev = 0;
  const scion_fp8* h = nullptr;
  const uint8_t* x = nullptr;
  const uint8_t* sx = nullptr;
  bool read(PyObject* const* a, Args& g) {
    int layer_dev;
    if (!get_int(a[2], &T) || !get_handle(a[3], &h) || !get_int(a[4], &n) || !get_int(a[5], &k) || !get_int(a[6], &layer_dev))
      return false;
    dev = g.dev = c10::cuda::current_device();
    if (dev != layer_dev) {
      PyErr_Format(PyExc_ValueError, "the layer is on device %d, the current device is %d", layer_dev, dev);
      return false;
    }
    x = static_cast<const uint8_t*>(g.tensor(a[0], "x_codes", kCodes, int64_t(T) * k));
    sx = static_cast<const uint8_t*>(g.tensor(a[1], "x_scales", kScales, T * groups(k)));
    return g.ok;
  }
};

// forward(x_codes, x_scales, T, handle, n, k, device, out, base, stream) -> status
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Product p;
  Args g(0);
  void* s;
  if (!want(n, 10) || !p.read(a, g)) return nullptr;
  ScalarType ot = at::kFloat;
  void* out = g.tensor(a[7], "out", kFloat, int64_t(p.T) * p.n, &ot);
  const void* base = g.optional(a[8], "base", kF32, int64_t(p.T) * p.n);
  if (!g.ok || !get_stream(a[9], p.dev, &s)) return nullptr;
  return PyLong_FromLong(abi.forward(p.x, p.sx, p.T, p.h, static_cast<const float*>(base), out, abi_type(ot), s));
  END_HANDLE_TH_ERRORS
}

// gated(x_codes, x_scales, T, handle, n, k, device, h, h_codes, h_scales, stream) -> status
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Product p;
  Args g(0);
  void* s;
  if (!want(n, 11) || !p.read(a, g)) return nullptr;
  void* h = g.optional(a[7], "h", kBf16, int64_t(p.T) * p.n);
  void* hc = g.optional(a[8], "h_codes", kCodes, int64_t(p.T) * p.n);
  void* hs = g.optional(a[9], "h_scales", kScales, p.T * groups(p.n));
  if (!g.ok || !get_stream(a[10], p.dev, &s)) return nullptr;
  return PyLong_FromLong(abi.gated(p.x, p.sx, p.T, p.h, h, static_cast<uint8_t*>(hc), static_cast<uint8_t*>(hs), s));
  END_HANDLE_TH_ERRORS
}

// init(rmsnorm, quantize, forward, gated): addresses of the ABI's functions
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "KKKK", &f[0], &f[1], &f[2], &f[3])) return nullptr;
  abi.rmsnorm = reinterpret_cast<decltype(abi.rmsnorm)>(f[0]);
  abi.quantize = reinterpret_cast<decltype(abi.quantize)>(f[1]);
  abi.forward = reinterpret_cast<decltype(abi.forward)>(f[2]);
  abi.gated = reinterpret_cast<decltype(abi.gated)>(f[3]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rmsnorm)), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(quantize)), METH_FASTCALL, nullptr},
    {"forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(forward)), METH_FASTCALL, nullptr},
    {"gated", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gated)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers this was compiled with
PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", SCION_TORCH) < 0) Py_CLEAR(m);
  return m;
}
