// The Python binding's checks and output tensors of the MX operators, in C++.
//
// A decode step calls these operators on a few rows, where a call's time is
// the host's: with the checks and the allocations in Python a call took 8 to
// 11 us, more than its kernel.  Every function takes positional arguments from
// the wrapper of the same name in __init__.py, checks the tensors, allocates
// outputs given as None, and calls the C ABI (w4.h).  It returns the outputs,
// or the status as an int where the C ABI refused.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/impl/VirtualGuardImpl.h>

#include <stdexcept>
#include <string>

#include "w4.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

struct PythonError {};  // the Python exception is set

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const Tensor& on_device(PyObject* o, const char* name) {
  if (o == Py_None) throw Refused(std::string(name) + " is required");
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA (HIP) tensor");
  return t;
}

// The current device, asked for once the first argument is on some device (a
// host tensor is refused where there is none, too).
int current_device(PyObject* first, const char* name) {
  on_device(first, name);
  static const c10::impl::VirtualGuardImpl guard(c10::DeviceType::CUDA);
  return guard.getDevice().index();
}

// A device tensor of the binding's kind: dense, on the current device.
const Tensor& tensor(PyObject* o, const char* name, int dev) {
  const Tensor& t = on_device(o, name);
  if (t.get_device() != dev)
    throw Refused(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                  "; the library works on the current device (cuda:" + std::to_string(dev) + ")");
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  return t;
}

void need_dtype(const Tensor& t, const char* name, at::ScalarType want) {
  if (t.scalar_type() != want)
    throw Refused(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " +
                  c10::toString(want));
}

void need_shape(const Tensor& t, const char* name, at::IntArrayRef want) {
  if (t.sizes() != want)
    throw Refused(std::string(name) + " has shape " + shape_of(t.sizes()) + ", expected " + shape_of(want));
}

const Tensor& bytes(PyObject* o, const char* name, int dev) {
  const Tensor& t = tensor(o, name, dev);
  need_dtype(t, name, at::kByte);
  return t;
}

// w4_dtype of a dense input; -1 where there is none
int dtype_code(at::ScalarType s) {
  return s == at::kFloat ? W4_F32 : s == at::kBFloat16 ? W4_BF16 : s == at::kHalf ? W4_F16 : -1;
}

// [rows, k] of fp32, bf16 or fp16
const Tensor& dense(PyObject* o, const char* name, int dev) {
  const Tensor& t = tensor(o, name, dev);
  if (dtype_code(t.scalar_type()) < 0)
    throw Refused(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) +
                  ", expected float32, bfloat16 or float16");
  if (t.dim() != 2) throw Refused(std::string(name) + " must be [rows, k]");
  if (t.size(1) % 32)
    throw Refused(std::string(name) + " has rows of " + std::to_string(t.size(1)) +
                  " values, expected a multiple of 32");
  return t;
}

int64_t width(long fmt, int64_t k) {
  if (fmt == W4_MXFP4) return k / 2;
  if (fmt == W4_MXFP8) return k;
  throw Refused("unknown MX format " + std::to_string(fmt));
}

Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
}

Tensor byte_output(PyObject* o, const char* name, at::IntArrayRef shape, const Tensor& like, int dev) {
  if (o == Py_None) return empty(shape, at::kByte, like);
  const Tensor& t = bytes(o, name, dev);
  need_shape(t, name, shape);
  return t;
}

// y of a product: given, or allocated as y_dtype (a w4_dtype)
Tensor product_output(PyObject* o, long y_dtype, int64_t m, int64_t n, const Tensor& like, int dev) {
  if (o == Py_None) {
    if (y_dtype != W4_F32 && y_dtype != W4_BF16) throw Refused("y_dtype must be float32 or bfloat16");
    return empty({m, n}, y_dtype == W4_F32 ? at::kFloat : at::kBFloat16, like);
  }
  const Tensor& t = tensor(o, "y", dev);
  if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
    throw Refused(std::string("y has dtype ") + c10::toString(t.scalar_type()) + ", expected float32 or bfloat16");
  need_shape(t, "y", {m, n});
  return t;
}

const uint8_t* u8(const Tensor& t) { return static_cast<const uint8_t*>(t.const_data_ptr()); }
uint8_t* u8(Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

// The current HIP stream of the device, which `query` (set by __init__.py)
// names.  The outputs' memory is this stream's too.
PyObject* query = nullptr;

void* stream(int dev) {
  if (PyErr_Occurred()) throw PythonError();  // (from reading an argument)
  PyObject* d = PyLong_FromLong(dev);
  PyObject* v = query && d ? PyObject_CallFunctionObjArgs(query, d, nullptr) : nullptr;
  Py_XDECREF(d);
  void* handle = v ? PyLong_AsVoidPtr(v) : nullptr;
  Py_XDECREF(v);
  if (PyErr_Occurred()) throw PythonError();
  return handle;
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
  return r;
}

PyObject* status(w4_status s) { return PyLong_FromLong(s); }

// Runs f on exactly n arguments; what it throws becomes a Python exception.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t n, F&& f) {
  if (got != n) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, got);
    return nullptr;
  }
  try {
    PyObject* r = f();
    if (PyErr_Occurred()) {
      Py_XDECREF(r);
      return nullptr;
    }
    return r;
  } catch (const PythonError&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (x, fmt, q, scales) -> (q, scales)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const int dev = current_device(a[0], "x");
    const Tensor& x = dense(a[0], "x", dev);
    const long fmt = PyLong_AsLong(a[1]);
    const int64_t rows = x.size(0), k = x.size(1);
    Tensor q = byte_output(a[2], "q", {rows, width(fmt, k)}, x, dev);
    Tensor s = byte_output(a[3], "scales", {rows, k / 32}, x, dev);
    const w4_status st = w4_mx_quantize(fmt, rows, k, x.const_data_ptr(), dtype_code(x.scalar_type()), u8(q), u8(s),
                                        stream(dev));
    return st ? status(st) : pair(q, s);
  });
}

// (q, scales, fmt, out, out_dtype) -> out
PyObject* dequant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const int dev = current_device(a[0], "q");
    const Tensor& q = bytes(a[0], "q", dev);
    const long fmt = PyLong_AsLong(a[2]), code = PyLong_AsLong(a[4]);
    if (q.dim() != 2) throw Refused("q must be [rows, k/2] or [rows, k]");
    width(fmt, 0);
    const int64_t rows = q.size(0), k = fmt == W4_MXFP4 ? 2 * q.size(1) : q.size(1);
    const Tensor& s = bytes(a[1], "scales", dev);
    need_shape(s, "scales", {rows, k / 32});
    Tensor out;
    if (a[3] == Py_None) {
      if (code != W4_F32 && code != W4_BF16) throw Refused("out_dtype must be float32 or bfloat16");
      out = empty({rows, k}, code == W4_F32 ? at::kFloat : at::kBFloat16, q);
    } else {
      out = tensor(a[3], "out", dev);
      if (out.scalar_type() != at::kFloat && out.scalar_type() != at::kBFloat16)
        throw Refused(std::string("out has dtype ") + c10::toString(out.scalar_type()) +
                      ", expected float32 or bfloat16");
      need_shape(out, "out", {rows, k});
    }
    const w4_status st =
        w4_mx_dequant(fmt, rows, k, u8(q), u8(s), out.data_ptr(), dtype_code(out.scalar_type()), stream(dev));
    return st ? status(st) : THPVariable_Wrap(out);
  });
}

// (x, gamma, eps, fmt or None, residual, residual_out, y, q, scales)
// -> (q, scales, residual_out)
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const int dev = current_device(a[0], "x");
    const Tensor& x = dense(a[0], "x", dev);
    const int64_t rows = x.size(0), k = x.size(1);
    const at::ScalarType dt = x.scalar_type();
    auto like_x = [&](PyObject* o, const char* name) -> const Tensor& {
      const Tensor& t = tensor(o, name, dev);
      need_dtype(t, name, dt);
      need_shape(t, name, {rows, k});
      return t;
    };
    const Tensor& gamma = tensor(a[1], "gamma", dev);
    need_dtype(gamma, "gamma", dt);
    need_shape(gamma, "gamma", {k});
    const double eps = PyFloat_AsDouble(a[2]);
    const bool mx = a[3] != Py_None;
    const long fmt = mx ? PyLong_AsLong(a[3]) : W4_MXFP8;
    const void* residual = nullptr;
    Tensor ro, q, s;
    if (a[4] != Py_None) {
      residual = like_x(a[4], "residual").const_data_ptr();
      ro = a[5] == Py_None ? empty({rows, k}, dt, x) : like_x(a[5], "residual_out");
    } else if (a[5] != Py_None) {
      throw Refused("residual_out without a residual");
    }
    void* y = a[6] == Py_None ? nullptr : like_x(a[6], "y").data_ptr();
    if (mx) {
      q = byte_output(a[7], "q", {rows, width(fmt, k)}, x, dev);
      s = byte_output(a[8], "scales", {rows, k / 32}, x, dev);
    } else {
      if (a[6] == Py_None) throw Refused("y is required without an MX format");
      if (a[7] != Py_None || a[8] != Py_None) throw Refused("q or scales without an MX format");
    }
    const w4_status st = w4_mx_rmsnorm(fmt, rows, k, x.const_data_ptr(), residual, gamma.const_data_ptr(),
                                       dtype_code(dt), (float)eps, residual ? ro.data_ptr() : nullptr, y,
                                       mx ? u8(q) : nullptr, mx ? u8(s) : nullptr, stream(dev));
    if (st) return status(st);
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    auto put = [&](int i, const Tensor& t) {
      if (t.defined()) {
        PyTuple_SET_ITEM(r, i, THPVariable_Wrap(t));
      } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(r, i, Py_None);
      }
    };
    put(0, q);
    put(1, s);
    put(2, ro);
    return r;
  });
}

// the activations of a product against the weight's k; their rows
int64_t activations(const Tensor& xq, const Tensor& xs, long fmt, int64_t k) {
  const int64_t w = width(fmt, k);
  if (xq.dim() != 2 || xq.size(1) != w)
    throw Refused("xq has shape " + shape_of(xq.sizes()) + ", expected [m, " + std::to_string(w) + "]");
  need_shape(xs, "xs", {xq.size(0), k / 32});
  return xq.size(0);
}

// (xq, xs, wq, ws, fmt, y, y_dtype) -> y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const int dev = current_device(a[2], "wq");
    const Tensor& wq = bytes(a[2], "wq", dev);
    if (wq.dim() != 2) throw Refused("wq must be [n, k/2]");
    const int64_t rows = wq.size(0), k = 2 * wq.size(1);
    const Tensor& ws = bytes(a[3], "ws", dev);
    need_shape(ws, "ws", {rows, k / 32});
    const Tensor& xq = bytes(a[0], "xq", dev);
    const Tensor& xs = bytes(a[1], "xs", dev);
    const long fmt = PyLong_AsLong(a[4]);
    const int64_t m = activations(xq, xs, fmt, k);
    Tensor y = product_output(a[5], PyLong_AsLong(a[6]), m, rows, wq, dev);
    const w4_status st = w4_mx_linear(fmt, rows, k, u8(wq), u8(ws), u8(xq), u8(xs), m, y.data_ptr(),
                                      dtype_code(y.scalar_type()), stream(dev));
    return st ? status(st) : THPVariable_Wrap(y);
  });
}

// (xq, xs, wq, ws, offsets, fmt, rows or None, y, y_dtype) -> y
PyObject* grouped_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const int dev = current_device(a[2], "wq");
    const Tensor& wq = bytes(a[2], "wq", dev);
    if (wq.dim() != 3) throw Refused("wq must be [experts, n, k/2]");
    const int64_t experts = wq.size(0), cols = wq.size(1), k = 2 * wq.size(2);
    const Tensor& ws = bytes(a[3], "ws", dev);
    need_shape(ws, "ws", {experts, cols, k / 32});
    const Tensor& off = tensor(a[4], "offsets", dev);
    need_dtype(off, "offsets", at::kInt);
    need_shape(off, "offsets", {experts + 1});
    const Tensor& xq = bytes(a[0], "xq", dev);
    const Tensor& xs = bytes(a[1], "xs", dev);
    const long fmt = PyLong_AsLong(a[5]);
    const int64_t tokens = activations(xq, xs, fmt, k);
    int64_t m = tokens;
    const int32_t* index = nullptr;
    if (a[6] != Py_None) {
      const Tensor& rows = tensor(a[6], "rows", dev);
      need_dtype(rows, "rows", at::kInt);
      if (rows.dim() != 1) throw Refused("rows must be [number of rows of y]");
      m = rows.size(0);
      index = static_cast<const int32_t*>(rows.const_data_ptr());
    }
    if (experts > INT32_MAX) return status(W4_ESHAPE);
    Tensor y = product_output(a[7], PyLong_AsLong(a[8]), m, cols, wq, dev);
    const w4_status st = w4_mx_grouped_linear(fmt, (int32_t)experts, cols, k, u8(wq), u8(ws), tokens, u8(xq), u8(xs),
                                              m, static_cast<const int32_t*>(off.const_data_ptr()), index,
                                              y.data_ptr(), dtype_code(y.scalar_type()), stream(dev));
    return st ? status(st) : THPVariable_Wrap(y);
  });
}

// (function of a device index that names its current stream)
PyObject* set_stream_query(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    Py_INCREF(a[0]);
    Py_XDECREF(query);
    query = a[0];
    Py_RETURN_NONE;
  });
}

#define W4_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {W4_METHOD(quantize), W4_METHOD(dequant),        W4_METHOD(rmsnorm),
                         W4_METHOD(linear),   W4_METHOD(grouped_linear), W4_METHOD(set_stream_query), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w4mx", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w4mx() { return PyModule_Create(&module); }
