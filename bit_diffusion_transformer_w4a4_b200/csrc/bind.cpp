// Argument marshalling of the operators around the 4-bit layers: torch tensors
// to the structs of include/svdq.h, and the current stream of their device.
// In C++ because a call on a few tokens takes the GPU 2 to 5 us, which the
// same checks written in Python (3 to 4 us) would exceed.  The library's entry
// points are handed over by address (init), so this module does not link it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "svdq.h"

namespace {

decltype(&svdq_dense_forward) g_dense = nullptr;
decltype(&svdq_rms_quantize8) g_rms8 = nullptr;
decltype(&svdq_rope_apply) g_rope = nullptr;

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a tensor, got %.80s", what, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    raise(PyExc_TypeError, "%s: expected an integer", what);
  }
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

int device_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return SVDQ_BF16;
    case at::kHalf: return SVDQ_FP16;
    case at::kFloat: return SVDQ_FP32;
    case at::kFloat8_e4m3fn: return SVDQ_E4M3;
    case at::kChar: return SVDQ_INT8;
    default: return -1;
  }
}

svdq_dtype dtype_in(const at::Tensor& t, unsigned allowed, const char* what) {
  const int d = dtype_of(t);
  if (d < 0 || !(allowed >> d & 1)) raise(PyExc_TypeError, "%s: dtype %s is not supported here", what, at::toString(t.scalar_type()));
  return static_cast<svdq_dtype>(d);
}

void like(const at::Tensor& t, at::ScalarType type, int dev, const char* what) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s: dtype %s, expected %s", what, at::toString(t.scalar_type()), at::toString(type));
  if (device_of(t) != dev) raise(PyExc_ValueError, "%s is not on the other tensors' device", what);
}

// Row distance of a [rows x cols] matrix with contiguous rows.
int64_t matrix(const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, int dev, const char* what) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    raise(PyExc_ValueError, "%s: expected a matrix of %lld x %lld", what, static_cast<long long>(rows), static_cast<long long>(cols));
  like(t, type, dev, what);
  if (cols > 1 && t.stride(1) != 1) raise(PyExc_ValueError, "%s: the elements of a row must be contiguous", what);
  return t.stride(0);
}

void* vector(PyObject* o, int64_t n, at::ScalarType type, int dev, const char* what) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 1 || t.size(0) != n) raise(PyExc_ValueError, "%s: expected %lld elements", what, static_cast<long long>(n));
  like(t, type, dev, what);
  if (n > 1 && t.stride(0) != 1) raise(PyExc_ValueError, "%s must be contiguous", what);
  return t.data_ptr();
}

// A [G x cols] tensor (or [cols]: one row) whose row g serves rows
// g * each .. of M.
const void* rows_of(PyObject* o, int64_t M, int64_t cols, at::ScalarType type, int dev, const char* what, int64_t* ld,
                    int64_t* each) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() == 1) {
    *ld = cols;
    *each = M > 0 ? M : 1;
    return vector(o, cols, type, dev, what);
  }
  if (*each == 0) *each = M > 0 ? M : 1;
  if (*each < 1) raise(PyExc_ValueError, "%s: rows each must be positive", what);
  // rows of no tokens: as many as there are
  *ld = matrix(t, M > 0 ? (M - 1) / *each + 1 : t.dim() == 2 ? t.size(0) : 0, cols, type, dev, what);
  return t.data_ptr();
}

// call(stream) with the tensors' device current, on `stream` or the device's
// current one.
template <class F>
PyObject* run(int dev, PyObject* stream, F call) {
  void* given = stream == Py_None ? nullptr : reinterpret_cast<void*>(static_cast<intptr_t>(integer(stream, "stream")));
  svdq_status code;
  if (dev < 0) {
    if (c10::cuda::device_count() > 0) raise(PyExc_ValueError, "the tensors are not on a CUDA device");
    code = call(given);  // the library reports the missing device
  } else {
    c10::cuda::OptionalCUDAGuard guard;
    if (dev != c10::cuda::current_device()) guard.set_index(static_cast<c10::DeviceIndex>(dev));
    if (stream == Py_None) given = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    code = call(given);
  }
  return PyLong_FromLong(code);
}

template <class F>
PyObject* guarded(F body) {
  try {
    return body();
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    return nullptr;
  }
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
}

constexpr unsigned k16 = 1u << SVDQ_BF16 | 1u << SVDQ_FP16, k8 = 1u << SVDQ_E4M3 | 1u << SVDQ_INT8;

// dense(a, w, y, a_scale, w_scale, bias, act, gate, gate_rows, residual, device_error, stream) -> status
PyObject* dense(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    count(n, 12);
    const at::Tensor &a = tensor(v[0], "a"), &w = tensor(v[1], "w"), &y = tensor(v[2], "y");
    svdq_dense_desc d = {};
    d.in = dtype_in(a, k16 | k8, "a");
    d.out = dtype_in(y, k16, "y");
    if (a.dim() != 2 || w.dim() != 2) raise(PyExc_ValueError, "a and w must be matrices");
    const int dev = device_of(a);
    const at::ScalarType it = a.scalar_type(), ot = y.scalar_type();
    d.M = a.size(0);
    d.K = a.size(1);
    d.N = w.size(0);
    d.lda = matrix(a, d.M, d.K, it, dev, "a");
    d.ldw = matrix(w, d.N, d.K, it, dev, "w");
    d.ldy = matrix(y, d.M, d.N, ot, dev, "y");
    d.a = a.data_ptr();
    d.w = w.data_ptr();
    d.y = y.data_ptr();
    d.a_scale = static_cast<const float*>(vector(v[3], d.M, at::kFloat, dev, "a_scale"));
    d.w_scale = static_cast<const float*>(vector(v[4], d.N, at::kFloat, dev, "w_scale"));
    d.bias = vector(v[5], d.N, ot, dev, "bias");
    d.act = static_cast<svdq_act>(integer(v[6], "act"));
    if (v[7] != Py_None) {
      d.gate_rows = integer(v[8], "gate_rows");
      d.gate = rows_of(v[7], d.M, d.N, ot, dev, "gate", &d.ldg, &d.gate_rows);
    }
    if (v[9] != Py_None) {
      const at::Tensor& r = tensor(v[9], "residual");
      d.ldr = matrix(r, d.M, d.N, ot, dev, "residual");
      d.residual = r.data_ptr();
    }
    d.device_error = static_cast<int*>(vector(v[10], 1, at::kInt, dev, "device_error"));
    return run(dev, v[11], [&](void* s) { return g_dense(&d, s); });
  });
}

// rms8(x, codes, scales, residual, h, weight, weight_rows, eps, norm, stream) -> status
PyObject* rms8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    count(n, 10);
    const at::Tensor &x = tensor(v[0], "x"), &codes = tensor(v[1], "codes");
    svdq_rms8_desc d = {};
    d.in = dtype_in(x, k16 | 1u << SVDQ_FP32, "x");
    d.out = dtype_in(codes, k8, "codes");
    if (x.dim() != 2) raise(PyExc_ValueError, "x must be a matrix");
    const int dev = device_of(x);
    const at::ScalarType it = x.scalar_type();
    d.M = x.size(0);
    d.K = x.size(1);
    d.ldx = matrix(x, d.M, d.K, it, dev, "x");
    d.ldc = matrix(codes, d.M, d.K, codes.scalar_type(), dev, "codes");
    d.x = x.data_ptr();
    d.codes = codes.data_ptr();
    if (v[2] == Py_None) raise(PyExc_TypeError, "scales: expected a tensor");
    d.scales = static_cast<float*>(vector(v[2], d.M, at::kFloat, dev, "scales"));
    if (v[3] != Py_None) {
      const at::Tensor& r = tensor(v[3], "residual");
      d.ldr = matrix(r, d.M, d.K, it, dev, "residual");
      d.residual = r.data_ptr();
    }
    if (v[4] != Py_None) {
      const at::Tensor& h = tensor(v[4], "h");
      d.ldh = matrix(h, d.M, d.K, it, dev, "h");
      d.h = h.data_ptr();
    }
    if (v[5] != Py_None) {
      d.weight_rows = integer(v[6], "weight_rows");
      d.weight = rows_of(v[5], d.M, d.K, it, dev, "weight", &d.ldw, &d.weight_rows);
    }
    const double eps = PyFloat_AsDouble(v[7]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    d.eps = static_cast<float>(eps);
    d.norm = truth(v[8]);
    return run(dev, v[9], [&](void* s) { return g_rms8(&d, s); });
  });
}

// Heads [S, H, D] or [B, S, H, D] and their output (None: in place).
svdq_rope_tensor heads(PyObject* o, PyObject* out, int64_t B, int64_t S, int64_t D, at::ScalarType type, int dev,
                       const char* what) {
  const at::Tensor& x = tensor(o, what);
  const at::Tensor& y = out == Py_None ? x : tensor(out, "the output");
  const int64_t n = x.dim();
  if (!((n == 4 && x.size(0) == B) || (n == 3 && B == 1)) || x.size(n - 3) != S || x.size(n - 1) != D)
    raise(PyExc_ValueError, "%s: the shape does not fit %lld sequences of %lld tokens with heads of %lld", what,
          static_cast<long long>(B), static_cast<long long>(S), static_cast<long long>(D));
  like(x, type, dev, what);
  if (y.sizes() != x.sizes()) raise(PyExc_ValueError, "%s: the output has another shape", what);
  like(y, type, dev, what);
  if (x.stride(n - 1) != 1 || y.stride(n - 1) != 1) raise(PyExc_ValueError, "%s: the elements of a head must be contiguous", what);
  return {x.data_ptr(), y.data_ptr(), x.size(n - 2),
          {n == 4 ? x.stride(0) : 0, x.stride(n - 3), x.stride(n - 2)},
          {n == 4 ? y.stride(0) : 0, y.stride(n - 3), y.stride(n - 2)}};
}

// rope(handle, head_dim, axes, q, pos, k, q_out, k_out, inverse, stream) -> status
PyObject* rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    count(n, 10);
    const auto h = reinterpret_cast<svdq_rope_t>(static_cast<intptr_t>(integer(v[0], "handle")));
    const int64_t D = integer(v[1], "head_dim"), axes = integer(v[2], "axes");
    const at::Tensor &q = tensor(v[3], "q"), &pos = tensor(v[4], "pos");
    const svdq_dtype type = dtype_in(q, k16 | 1u << SVDQ_FP32, "q");
    if (q.dim() != 3 && q.dim() != 4) raise(PyExc_ValueError, "q: expected [(B,) S, H, %lld]", static_cast<long long>(D));
    const int64_t B = q.dim() == 4 ? q.size(0) : 1, S = q.size(q.dim() - 3);
    const int dev = device_of(q);
    const svdq_rope_tensor tq = heads(v[3], v[6], B, S, D, q.scalar_type(), dev, "q");
    svdq_rope_tensor tk = {};
    if (v[5] != Py_None) tk = heads(v[5], v[7], B, S, D, q.scalar_type(), dev, "k");
    svdq_rope_positions p = {};
    switch (pos.scalar_type()) {
      case at::kInt: p.type = SVDQ_POS_INT32; break;
      case at::kLong: p.type = SVDQ_POS_INT64; break;
      case at::kFloat: p.type = SVDQ_POS_FP32; break;
      default: raise(PyExc_TypeError, "pos: dtype %s is not supported here", at::toString(pos.scalar_type()));
    }
    if (device_of(pos) != dev) raise(PyExc_ValueError, "pos is not on the other tensors' device");
    const bool flat = pos.dim() == 2 && pos.size(1) == axes;
    p.p = pos.data_ptr();
    if (flat && pos.size(0) == B * S) {
      p.batch_stride = S * pos.stride(0);
      p.token_stride = pos.stride(0);
      p.axis_stride = pos.stride(1);
    } else if (flat && pos.size(0) == S) {
      p.token_stride = pos.stride(0);
      p.axis_stride = pos.stride(1);
    } else if (pos.dim() == 3 && pos.size(0) == B && pos.size(1) == S && pos.size(2) == axes) {
      p.batch_stride = pos.stride(0);
      p.token_stride = pos.stride(1);
      p.axis_stride = pos.stride(2);
    } else {
      raise(PyExc_ValueError, "pos: expected [S, axes], [B * S, axes] or [B, S, axes]");
    }
    const int inverse = truth(v[8]);
    return run(dev, v[9], [&](void* s) {
      return g_rope(h, type, B, S, &p, &tq, v[5] == Py_None ? nullptr : &tk, inverse, s);
    });
  });
}

// init(address of svdq_dense_forward, svdq_rms_quantize8, svdq_rope_apply)
PyObject* init(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 3);
    g_dense = reinterpret_cast<decltype(g_dense)>(static_cast<intptr_t>(integer(v[0], "address")));
    g_rms8 = reinterpret_cast<decltype(g_rms8)>(static_cast<intptr_t>(integer(v[1], "address")));
    g_rope = reinterpret_cast<decltype(g_rope)>(static_cast<intptr_t>(integer(v[2], "address")));
    Py_RETURN_NONE;
  });
}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(init)), METH_FASTCALL, nullptr},
    {"dense", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dense)), METH_FASTCALL, nullptr},
    {"rms8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rms8)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
