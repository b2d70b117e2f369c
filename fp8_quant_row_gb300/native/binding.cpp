// binding.cpp -- native argument marshalling of the 8-bit row operators and their product.
//
// A call for one token takes the device two or three microseconds; checks and allocations from
// Python took ten and more. These functions check the tensors, allocate the outputs that are not
// given, call the C ABI (whose addresses init() receives) on the current torch stream and wrap the
// results. Refusals are TypeErrors, statuses of the library go to the Python check().
#include <Python.h>

#include <cstdarg>
#include <cstdint>
#include <optional>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

using RmsFn = int (*)(void*, void*, float*, const void*, const void*, const void*, int, int64_t,
                      int64_t, float, cudaStream_t);
using SiluFn = int (*)(void*, float*, const void*, const void*, int64_t, int, int64_t, int64_t,
                       cudaStream_t);
using MatmulFn = int (*)(void*, const int8_t*, int64_t, const float*, const int8_t*, const float*,
                         const void*, int, int64_t, int64_t, int64_t, cudaStream_t);
RmsFn g_rms = nullptr;
SiluFn g_silu = nullptr;
MatmulFn g_matmul = nullptr;
PyObject* g_check = nullptr;  // raises the library's error of a status

// Thrown once a Python error is set.
struct Refused {};

[[noreturn]] void refuse(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_TypeError, format, args);
  va_end(args);
  throw Refused{};
}

// The argument's tensor; null for None where that is allowed.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse("%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return &THPVariable_Unpack(o);
}

// The library launches on the current device: x and the other tensors have to be there.
at::Device device_of(const at::Tensor& x, const char* name,
                     std::initializer_list<const at::Tensor*> others) {
  const at::Device dev = x.device();
  for (const at::Tensor* t : others)
    if (t && t->device() != dev)
      refuse("tensors on %s and on %s: expected one device", dev.str().c_str(),
             t->device().str().c_str());
  if (!dev.is_cuda()) refuse("%s: expected a CUDA tensor, got %s", name, dev.str().c_str());
  const int current = c10::cuda::current_device();
  if (dev.index() != current)
    refuse("%s is on %s, but the current device is cuda:%d", name, dev.str().c_str(), current);
  return dev;
}

void contiguous(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type || !t.is_contiguous())
    refuse("%s: expected a contiguous CUDA %s tensor, got %s (contiguous=%d)", name,
           c10::toString(type), c10::toString(t.scalar_type()), int(t.is_contiguous()));
}

// A float32 vector of n contiguous values.
float* scales(const at::Tensor& t, int64_t n, const char* name) {
  if (t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous())
    refuse("%s: expected %lld contiguous float32 values, got %lld of %s", name, (long long)n,
           (long long)t.numel(), c10::toString(t.scalar_type()));
  return static_cast<float*>(t.data_ptr());
}

struct Rows {
  int64_t rows, cols, ld;
};

// Rows that lie at one stride, columns adjacent.
Rows strided_rows(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type || t.dim() < 1)
    refuse("%s: expected a %s tensor [..., cols], got %s of %lld dimensions", name,
           c10::toString(type), c10::toString(t.scalar_type()), (long long)t.dim());
  const at::IntArrayRef size = t.sizes(), stride = t.strides();
  const int64_t cols = size.back();
  Rows r{cols ? t.numel() / cols : 0, cols, cols};
  if (t.is_contiguous()) return r;
  bool fine = stride.back() == 1 || cols == 1;
  int64_t expected = -1;  // stride of the next dimension outwards
  for (int64_t d = t.dim() - 2; d >= 0 && fine; --d) {
    if (size[d] == 1) continue;
    if (expected < 0) r.ld = stride[d];
    else fine = stride[d] == expected;
    expected = stride[d] * size[d];
  }
  if (!fine)
    refuse("%s: its rows do not lie at one row stride with adjacent columns", name);
  return r;
}

// An output: the given tensor, checked, or a new one, made by data().
class Out {
 public:
  Out(const at::Tensor* given, PyObject* given_object, at::IntArrayRef shape, at::ScalarType type,
      const char* name)
      : given_(given), given_object_(given_object), shape_(shape.begin(), shape.end()), type_(type) {
    if (given && (given->scalar_type() != type || given->sizes() != shape || !given->is_contiguous()))
      refuse("%s: expected a contiguous %s tensor of the result's shape", name,
             c10::toString(type));
  }
  void* data(at::Device dev) {
    if (given_) return given_->data_ptr();
    made_ = at::detail::empty_cuda(shape_, type_, dev, std::nullopt);
    return made_.data_ptr();
  }
  // The Python object, a new reference.
  PyObject* object() {
    if (!given_) {
      PyObject* o = THPVariable_Wrap(std::move(made_));
      if (!o) throw Refused{};
      return o;
    }
    Py_INCREF(given_object_);
    return given_object_;
  }

 private:
  const at::Tensor* given_;
  PyObject* given_object_;
  at::Tensor made_;
  c10::SmallVector<int64_t, 5> shape_;
  at::ScalarType type_;
};

// Other Python threads run during an allocation, which may wait for the device, and a launch, which
// waits while the stream's queue is full. (No Python object is touched meanwhile.)
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// A tuple of the outputs.
PyObject* results(std::initializer_list<Out*> outs) {
  PyObject* tuple = PyTuple_New(Py_ssize_t(outs.size()));
  if (!tuple) throw Refused{};
  Py_ssize_t i = 0;
  try {
    for (Out* o : outs) PyTuple_SET_ITEM(tuple, i++, o->object());
  } catch (...) {
    Py_DECREF(tuple);
    throw;
  }
  return tuple;
}

at::ScalarType row_type(long code) { return code == 0 ? at::kChar : at::kFloat8_e4m3fn; }

// Raises for a status that is not 0.
void check(int status, const char* where) {
  if (status == 0) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", status, where);
  if (r) {
    Py_DECREF(r);
    PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, status);
  }
  throw Refused{};
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("expected %zd arguments, got %zd", want, n);
}

// rms_norm_quant(x, weight, residual, q_type, eps, residual_out, q, scale)
PyObject* rms_norm_quant(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 8);
  const at::Tensor& x = *tensor(arg[0], "x");
  const at::Tensor& weight = *tensor(arg[1], "weight");
  const at::Tensor* residual = tensor(arg[2], "residual", true);
  const long type = PyLong_AsLong(arg[3]);
  const double eps = PyFloat_AsDouble(arg[4]);
  if (PyErr_Occurred()) throw Refused{};
  const at::Tensor* residual_out = tensor(arg[5], "residual_out", true);
  const at::Tensor* q = tensor(arg[6], "q", true);
  const at::Tensor* scale = tensor(arg[7], "scale", true);
  const at::Device dev = device_of(x, "x", {&weight, residual, residual_out, q, scale});
  contiguous(x, at::kBFloat16, "x");
  contiguous(weight, at::kBFloat16, "weight");
  if (x.dim() < 1) refuse("x: expected [..., cols]");
  const at::IntArrayRef shape = x.sizes();
  const int64_t cols = shape.back(), rows = cols ? x.numel() / cols : 0;
  if (weight.numel() != cols)
    refuse("weight: expected %lld values, got %lld", (long long)cols, (long long)weight.numel());
  std::optional<Out> h;
  if (residual) {
    contiguous(*residual, at::kBFloat16, "residual");
    if (residual->sizes() != shape) refuse("residual: expected x's shape");
    h.emplace(residual_out, arg[5], shape, at::kBFloat16, "residual_out");
  } else if (residual_out) {
    refuse("residual_out: given without a residual");
  }
  Out qo(q, arg[6], shape, row_type(type), "q");
  Out so(scale, arg[7], shape.slice(0, shape.size() - 1), at::kFloat, "scale");
  int status = 0;
  {
    Unlocked unlocked;
    void* hp = h ? h->data(dev) : nullptr;
    void* qp = qo.data(dev);
    status = g_rms(hp, qp, static_cast<float*>(so.data(dev)), x.data_ptr(),
                   residual ? residual->data_ptr() : nullptr, weight.data_ptr(), int(type), rows,
                   cols, float(eps), c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  }
  check(status, "fp8q_rms_norm_quant");
  return h ? results({&*h, &qo, &so}) : results({&qo, &so});
}

// silu_mul_quant(gate, up, q_type, q, scale)
PyObject* silu_mul_quant(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 5);
  const at::Tensor& gate = *tensor(arg[0], "gate");
  const at::Tensor& up = *tensor(arg[1], "up");
  const long type = PyLong_AsLong(arg[2]);
  if (PyErr_Occurred()) throw Refused{};
  const at::Tensor* q = tensor(arg[3], "q", true);
  const at::Tensor* scale = tensor(arg[4], "scale", true);
  const at::Device dev = device_of(gate, "gate", {&up, q, scale});
  const Rows g = strided_rows(gate, at::kBFloat16, "gate");
  const Rows u = strided_rows(up, at::kBFloat16, "up");
  const at::IntArrayRef shape = gate.sizes();
  if (up.sizes() != shape || (g.rows > 1 && u.ld != g.ld))
    refuse("gate and up: expected one shape and one row stride");
  Out qo(q, arg[3], shape, row_type(type), "q");
  Out so(scale, arg[4], shape.slice(0, shape.size() - 1), at::kFloat, "scale");
  int status = 0;
  {
    Unlocked unlocked;
    void* qp = qo.data(dev);
    status = g_silu(qp, static_cast<float*>(so.data(dev)), gate.data_ptr(), up.data_ptr(),
                    g.rows > 1 ? g.ld : g.cols, int(type), g.rows, g.cols,
                    c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  }
  check(status, "fp8q_silu_mul_quant");
  return results({&qo, &so});
}

// int8_matmul(a, a_scale, w, w_scale, bias, out_type, out)
PyObject* int8_matmul(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 7);
  const at::Tensor& a = *tensor(arg[0], "a");
  const at::Tensor& a_scale = *tensor(arg[1], "a_scale");
  const at::Tensor& w = *tensor(arg[2], "w");
  const at::Tensor& w_scale = *tensor(arg[3], "w_scale");
  const at::Tensor* bias = tensor(arg[4], "bias", true);
  const long type = PyLong_AsLong(arg[5]);
  if (PyErr_Occurred()) throw Refused{};
  const at::Tensor* out = tensor(arg[6], "out", true);
  const at::Device dev = device_of(a, "a", {&a_scale, &w, &w_scale, bias, out});
  const Rows r = strided_rows(a, at::kChar, "a");
  if (w.scalar_type() != at::kChar || w.dim() != 2 || w.size(1) != r.cols || !w.is_contiguous())
    refuse("w: expected a contiguous int8 [n, %lld]", (long long)r.cols);
  const int64_t channels = w.size(0);
  const float* as = scales(a_scale, r.rows, "a_scale");
  const float* ws = scales(w_scale, channels, "w_scale");
  if (bias) {
    contiguous(*bias, at::kBFloat16, "bias");
    if (bias->numel() != channels)
      refuse("bias: expected %lld values, got %lld", (long long)channels, (long long)bias->numel());
  }
  c10::SmallVector<int64_t, 8> shape(a.sizes().begin(), a.sizes().end());
  shape.back() = channels;
  Out o(out, arg[6], shape, type == 0 ? at::kBFloat16 : at::kFloat, "out");
  int status = 0;
  {
    Unlocked unlocked;
    status = g_matmul(o.data(dev), static_cast<const int8_t*>(a.data_ptr()),
                      r.rows > 1 ? r.ld : r.cols, as, static_cast<const int8_t*>(w.data_ptr()), ws,
                      bias ? bias->data_ptr() : nullptr, int(type), r.rows, channels, r.cols,
                      c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  }
  check(status, "fp8q_int8_matmul");
  return o.object();
}

// init(rms, silu, matmul, check): the C entry points' addresses and the error raiser
PyObject* init(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 4);
  void* f[3];
  for (int i = 0; i < 3; ++i) f[i] = PyLong_AsVoidPtr(arg[i]);
  if (PyErr_Occurred()) throw Refused{};
  g_rms = reinterpret_cast<RmsFn>(f[0]);
  g_silu = reinterpret_cast<SiluFn>(f[1]);
  g_matmul = reinterpret_cast<MatmulFn>(f[2]);
  Py_XDECREF(g_check);
  Py_INCREF(arg[3]);
  g_check = arg[3];
  Py_RETURN_NONE;
}

// No C++ exception passes into the interpreter.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(arg, n);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<init>("init"), method<rms_norm_quant>("rms_norm_quant"),
                           method<silu_mul_quant>("silu_mul_quant"),
                           method<int8_matmul>("int8_matmul"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&g_module); }
