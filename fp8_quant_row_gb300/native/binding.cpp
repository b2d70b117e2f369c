// binding.cpp -- native argument marshalling of the 8-bit row operators, their product and the paged
// cache.
//
// A call for one token takes the device two or three microseconds; checks and allocations from
// Python took ten and more. These functions check the tensors, allocate the outputs that are not
// given, call the C ABI (whose addresses init() receives) on the current torch stream and wrap the
// results. Refusals are TypeErrors, statuses of the library go to the Python check().
#include <Python.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <optional>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8q.h"

namespace {

using RmsFn = int (*)(void*, void*, float*, const void*, const void*, const void*, int, int64_t,
                      int64_t, float, cudaStream_t);
using SiluFn = int (*)(void*, float*, const void*, const void*, int64_t, int, int64_t, int64_t,
                       cudaStream_t);
using MatmulFn = int (*)(void*, const int8_t*, int64_t, const float*, const int8_t*, const float*,
                         const void*, int, int64_t, int64_t, int64_t, cudaStream_t);
using RopeFn = decltype(&fp8q_qk_norm_rope);
using WriteFn = decltype(&fp8q_cache_write);
using ReadFn = decltype(&fp8q_cache_read);
using AttnFn = decltype(&fp8q_paged_attention);
using AttnSizeFn = decltype(&fp8q_paged_attention_workspace);
RmsFn g_rms = nullptr;
SiluFn g_silu = nullptr;
MatmulFn g_matmul = nullptr;
RopeFn g_rope = nullptr;
WriteFn g_write = nullptr;
ReadFn g_read = nullptr;
AttnFn g_attn = nullptr;
AttnSizeFn g_attn_size = nullptr;
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

// ------------------------------------------------------------------------------------------
// the paged cache
// ------------------------------------------------------------------------------------------

// Heads of tokens: [tokens, heads, dim] bf16, a token's heads adjacent; ld: values between tokens.
struct Heads {
  int64_t tokens, heads, dim, ld;
};

Heads head_rows(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3)
    refuse("%s: expected a bfloat16 tensor [tokens, heads, head_dim], got %s of %lld dimensions", name,
           c10::toString(t.scalar_type()), (long long)t.dim());
  Heads h{t.size(0), t.size(1), t.size(2), 0};
  const bool fine = (t.stride(2) == 1 || h.dim <= 1) && (t.stride(1) == h.dim || h.heads <= 1);
  if (!fine && t.numel() > 0)
    refuse("%s: a token's heads have to be adjacent (strides %lld, %lld)", name,
           (long long)t.stride(1), (long long)t.stride(2));
  h.ld = h.tokens > 1 ? t.stride(0) : h.heads * h.dim;
  return h;
}

// An output of heads: the given tensor, strided as inputs may be, or a new contiguous one.
class HeadsOut {
 public:
  HeadsOut(const at::Tensor* given, PyObject* object, const Heads& like, const char* name)
      : given_(given), object_(object), shape_{like.tokens, like.heads, like.dim},
        ld_(like.heads * like.dim) {
    if (!given) return;
    const Heads h = head_rows(*given, name);
    if (h.tokens != like.tokens || h.heads != like.heads || h.dim != like.dim)
      refuse("%s: expected the shape [%lld, %lld, %lld]", name, (long long)like.tokens,
             (long long)like.heads, (long long)like.dim);
    ld_ = h.ld;
  }
  int64_t ld() const { return ld_; }
  void* data(at::Device dev) {
    if (given_) return given_->data_ptr();
    made_ = at::detail::empty_cuda(shape_, at::kBFloat16, dev, std::nullopt);
    return made_.data_ptr();
  }
  PyObject* object() {
    if (given_) {
      Py_INCREF(object_);
      return object_;
    }
    PyObject* o = THPVariable_Wrap(std::move(made_));
    if (!o) throw Refused{};
    return o;
  }

 private:
  const at::Tensor* given_;
  PyObject* object_;
  at::Tensor made_;
  std::array<int64_t, 3> shape_;
  int64_t ld_;
};

// A head's norm weight.
const void* head_weight(const at::Tensor* w, int64_t dim, const char* name) {
  if (!w) return nullptr;
  contiguous(*w, at::kBFloat16, name);
  if (w->numel() != dim)
    refuse("%s: expected %lld values, got %lld", name, (long long)dim, (long long)w->numel());
  return w->data_ptr();
}

// inv_freq, positions, axis, interleaved: arg[0 .. 3]; false without a rotation.
bool rotary_of(fp8q_rotary* r, PyObject* const* arg, int64_t tokens, const at::Tensor* const t[3]) {
  const at::Tensor *freq = t[0], *pos = t[1], *axis = t[2];
  const int interleaved = PyObject_IsTrue(arg[3]);
  if (interleaved < 0) throw Refused{};
  if (!freq) {
    if (pos || axis) refuse("positions and axis: given without inv_freq");
    return false;
  }
  if (!pos) refuse("positions: needed with inv_freq");
  if (freq->scalar_type() != at::kDouble || freq->dim() != 1 || !freq->is_contiguous())
    refuse("inv_freq: expected contiguous float64 values, got %s of %lld dimensions",
           c10::toString(freq->scalar_type()), (long long)freq->dim());
  if (freq->size(0) > INT32_MAX) refuse("inv_freq: too many values");
  const bool wide = pos->scalar_type() == at::kLong;
  if ((!wide && pos->scalar_type() != at::kInt) || pos->dim() < 1 || pos->dim() > 2 ||
      pos->size(-1) != tokens || (pos->stride(-1) != 1 && tokens > 1))
    refuse("positions: expected int32 or int64 [tokens] or [axes, tokens] with %lld adjacent tokens",
           (long long)tokens);
  r->axes = pos->dim() == 2 ? int(std::min<int64_t>(pos->size(0), INT32_MAX)) : 1;
  if (axis) {
    if (axis->scalar_type() != at::kInt || axis->numel() != freq->size(0) || !axis->is_contiguous())
      refuse("axis: expected %lld contiguous int32 values", (long long)freq->size(0));
  } else if (r->axes != 1) {
    refuse("axis: needed for positions on %d axes", r->axes);
  }
  r->inv_freq = static_cast<const double*>(freq->data_ptr());
  r->axis = axis ? static_cast<const int32_t*>(axis->data_ptr()) : nullptr;
  r->positions = pos->data_ptr();
  r->position_stride = pos->dim() == 2 ? pos->stride(0) : tokens;
  r->position_bytes = wide ? 8 : 4;
  r->pairs = int(freq->size(0));
  r->interleaved = interleaved;
  return true;
}

// k, v, k_scale, v_scale: arg[0 .. 3].
fp8q_paged_cache cache_of(const at::Tensor* const t[4]) {
  const at::Tensor &k = *t[0], &v = *t[1];
  fp8q_paged_cache c{};
  const at::ScalarType type = k.scalar_type();
  if (type == at::kChar) c.type = FP8Q_INT8;
  else if (type == at::kFloat8_e4m3fn) c.type = FP8Q_E4M3;
  else if (type == at::kBFloat16) c.type = FP8Q_BF16;
  else refuse("cache.k: expected int8, float8_e4m3fn or bfloat16, got %s", c10::toString(type));
  if (v.scalar_type() != type || k.dim() != 4 || v.sizes() != k.sizes())
    refuse("cache.k and cache.v: expected one type and shape [pages, heads, page_size, head_dim]");
  c.pages = k.size(0);
  c.heads = k.size(1);
  c.page_size = k.size(2);
  c.head_dim = k.size(3);
  const int64_t page = c.heads * c.page_size * c.head_dim, rows = c.heads * c.page_size;
  auto stride = [&](const at::Tensor& x, int64_t size, const char* name) {
    int64_t expected = 1;
    bool fine = true;
    for (int64_t d = x.dim() - 1; d > 0; --d) {
      fine = fine && (x.size(d) == 1 || x.stride(d) == expected);
      expected *= x.size(d);
    }
    if (!fine && x.numel() > 0) refuse("%s: a page has to be contiguous", name);
    return c.pages > 1 ? x.stride(0) : size;
  };
  c.k_stride = stride(k, page, "cache.k");
  c.v_stride = stride(v, page, "cache.v");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  if (c.type == FP8Q_BF16) {
    if (t[2] || t[3]) refuse("cache: scales beside bfloat16 values");
    return c;
  }
  const at::IntArrayRef shape = k.sizes().slice(0, 3);
  for (int i = 2; i < 4; ++i) {
    const char* name = i == 2 ? "cache.k_scale" : "cache.v_scale";
    if (!t[i] || t[i]->scalar_type() != at::kFloat || t[i]->sizes() != shape)
      refuse("%s: expected float32 [pages, heads, page_size]", name);
    (i == 2 ? c.k_scale_stride : c.v_scale_stride) = stride(*t[i], rows, name);
    (i == 2 ? c.k_scale : c.v_scale) = static_cast<float*>(t[i]->data_ptr());
  }
  return c;
}

// A page table: int32 [batch, width], rows at one stride.
struct Table {
  const int32_t* p;
  int64_t ld, width;
};
Table table_of(const at::Tensor& t, int64_t batch) {
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != batch ||
      (t.size(1) > 1 && t.stride(1) != 1))
    refuse("page_table: expected int32 [%lld, width] with adjacent pages", (long long)batch);
  return Table{static_cast<const int32_t*>(t.data_ptr()), batch > 1 ? t.stride(0) : t.size(1),
               t.size(1)};
}

// qk_norm_rope(q, k, inv_freq, positions, axis, interleaved, q_weight, k_weight, eps, q_out, k_out)
PyObject* qk_norm_rope(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 11);
  const at::Tensor &q = *tensor(arg[0], "q"), &k = *tensor(arg[1], "k");
  const at::Tensor* rot[3] = {tensor(arg[2], "inv_freq", true), tensor(arg[3], "positions", true),
                              tensor(arg[4], "axis", true)};
  const at::Tensor* qw = tensor(arg[6], "q_weight", true);
  const at::Tensor* kw = tensor(arg[7], "k_weight", true);
  const double eps = PyFloat_AsDouble(arg[8]);
  if (PyErr_Occurred()) throw Refused{};
  const at::Tensor* q_out = tensor(arg[9], "q_out", true);
  const at::Tensor* k_out = tensor(arg[10], "k_out", true);
  const at::Device dev =
      device_of(q, "q", {&k, rot[0], rot[1], rot[2], qw, kw, q_out, k_out});
  const Heads qh = head_rows(q, "q"), kh = head_rows(k, "k");
  if (kh.tokens != qh.tokens || kh.dim != qh.dim) refuse("q and k: expected one number of tokens and head_dim");
  const void* qwp = head_weight(qw, qh.dim, "q_weight");
  const void* kwp = head_weight(kw, qh.dim, "k_weight");
  fp8q_rotary r{};
  const bool turned = rotary_of(&r, arg + 2, qh.tokens, rot);
  HeadsOut qo(q_out, arg[9], qh, "q_out"), ko(k_out, arg[10], kh, "k_out");
  int status = 0;
  {
    Unlocked unlocked;
    void *qp = qo.data(dev), *kp = ko.data(dev);
    status = g_rope(qp, qo.ld(), kp, ko.ld(), q.data_ptr(), qh.ld, k.data_ptr(), kh.ld, qwp, kwp,
                    float(eps), turned ? &r : nullptr, qh.tokens, qh.heads, kh.heads, qh.dim,
                    c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  }
  check(status, "fp8q_qk_norm_rope");
  PyObject* tuple = PyTuple_New(2);
  if (!tuple) throw Refused{};
  try {
    PyTuple_SET_ITEM(tuple, 0, qo.object());
    PyTuple_SET_ITEM(tuple, 1, ko.object());
  } catch (...) {
    Py_DECREF(tuple);
    throw;
  }
  return tuple;
}

// cache_write(k, v, ck, cv, sk, sv, slots, q, inv_freq, positions, axis, interleaved, q_weight,
//             k_weight, eps, q_out)
PyObject* cache_write(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 16);
  const at::Tensor &k = *tensor(arg[0], "k"), &v = *tensor(arg[1], "v");
  const at::Tensor* parts[4] = {tensor(arg[2], "cache.k"), tensor(arg[3], "cache.v"),
                                tensor(arg[4], "cache.k_scale", true),
                                tensor(arg[5], "cache.v_scale", true)};
  const at::Tensor& slots = *tensor(arg[6], "slots");
  const at::Tensor* q = tensor(arg[7], "q", true);
  const at::Tensor* rot[3] = {tensor(arg[8], "inv_freq", true), tensor(arg[9], "positions", true),
                              tensor(arg[10], "axis", true)};
  const at::Tensor* qw = tensor(arg[12], "q_weight", true);
  const at::Tensor* kw = tensor(arg[13], "k_weight", true);
  const double eps = PyFloat_AsDouble(arg[14]);
  if (PyErr_Occurred()) throw Refused{};
  const at::Tensor* q_out = tensor(arg[15], "q_out", true);
  const at::Device dev = device_of(k, "k", {&v, parts[0], parts[1], parts[2], parts[3], &slots, q,
                                            rot[0], rot[1], rot[2], qw, kw, q_out});
  const fp8q_paged_cache cache = cache_of(parts);
  const Heads kh = head_rows(k, "k"), vh = head_rows(v, "v");
  if (vh.tokens != kh.tokens || vh.heads != kh.heads || vh.dim != kh.dim)
    refuse("k and v: expected one shape");
  if (kh.heads != cache.heads || kh.dim != cache.head_dim)
    refuse("k: expected the cache's [tokens, %lld, %lld]", (long long)cache.heads,
           (long long)cache.head_dim);
  if (slots.scalar_type() != at::kLong || slots.numel() != kh.tokens || !slots.is_contiguous())
    refuse("slots: expected %lld contiguous int64 values", (long long)kh.tokens);
  std::optional<HeadsOut> qo;
  Heads qh{kh.tokens, 0, kh.dim, 0};
  if (q) {
    qh = head_rows(*q, "q");
    if (qh.tokens != kh.tokens || qh.dim != kh.dim || qh.heads < 1)
      refuse("q: expected [%lld, heads, %lld]", (long long)kh.tokens, (long long)kh.dim);
    qo.emplace(q_out, arg[15], qh, "q_out");
  } else if (q_out || qw) {
    refuse("q_out and q_weight: given without q");
  }
  const void* qwp = head_weight(qw, kh.dim, "q_weight");
  const void* kwp = head_weight(kw, kh.dim, "k_weight");
  fp8q_rotary r{};
  const bool turned = rotary_of(&r, arg + 8, kh.tokens, rot);
  int status = 0;
  {
    Unlocked unlocked;
    void* qp = qo ? qo->data(dev) : nullptr;
    status = g_write(&cache, static_cast<const int64_t*>(slots.data_ptr()), qp, qo ? qo->ld() : 0,
                     q ? q->data_ptr() : nullptr, qh.ld, k.data_ptr(), kh.ld, v.data_ptr(), vh.ld,
                     qwp, kwp, float(eps), turned ? &r : nullptr, kh.tokens, qh.heads,
                     c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  }
  check(status, "fp8q_cache_write");
  if (qo) return qo->object();
  Py_RETURN_NONE;
}

// cache_read(ck, cv, sk, sv, page_table, offsets, rows, k, v)
PyObject* cache_read(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 9);
  const at::Tensor* parts[4] = {tensor(arg[0], "cache.k"), tensor(arg[1], "cache.v"),
                                tensor(arg[2], "cache.k_scale", true),
                                tensor(arg[3], "cache.v_scale", true)};
  const at::Tensor &table = *tensor(arg[4], "page_table"), &offsets = *tensor(arg[5], "offsets");
  const int64_t rows = PyLong_AsLongLong(arg[6]);
  if (PyErr_Occurred()) throw Refused{};
  const at::Tensor *k = tensor(arg[7], "k", true), *v = tensor(arg[8], "v", true);
  const at::Device dev = device_of(*parts[0], "cache.k", {parts[1], parts[2], parts[3], &table,
                                                          &offsets, k, v});
  const fp8q_paged_cache cache = cache_of(parts);
  if (rows < 0) refuse("rows: expected 0 or more");
  if (offsets.scalar_type() != at::kLong || offsets.dim() != 1 || offsets.size(0) < 1 ||
      !offsets.is_contiguous())
    refuse("offsets: expected contiguous int64 [batch + 1]");
  const int64_t batch = offsets.size(0) - 1;
  const Table t = table_of(table, batch);
  const std::array<int64_t, 3> shape{rows, cache.heads, cache.head_dim};
  Out ko(k, arg[7], shape, at::kBFloat16, "k"), vo(v, arg[8], shape, at::kBFloat16, "v");
  int status = 0;
  {
    Unlocked unlocked;
    void *kp = ko.data(dev), *vp = vo.data(dev);
    status = g_read(kp, vp, &cache, t.p, t.ld, t.width, static_cast<const int64_t*>(offsets.data_ptr()),
                    batch, rows, c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  }
  check(status, "fp8q_cache_read");
  return results({&ko, &vo});
}

// paged_attention(q, ck, cv, sk, sv, page_table, lengths, scale, window, return_lse, out, lse)
PyObject* paged_attention(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 12);
  const at::Tensor& q = *tensor(arg[0], "q");
  const at::Tensor* parts[4] = {tensor(arg[1], "cache.k"), tensor(arg[2], "cache.v"),
                                tensor(arg[3], "cache.k_scale", true),
                                tensor(arg[4], "cache.v_scale", true)};
  const at::Tensor &table = *tensor(arg[5], "page_table"), &lengths = *tensor(arg[6], "lengths");
  const bool own_scale = arg[7] != Py_None;
  const double scale = own_scale ? PyFloat_AsDouble(arg[7]) : 0.0;
  const int64_t window = PyLong_AsLongLong(arg[8]);
  const int want_lse = PyObject_IsTrue(arg[9]);
  if (PyErr_Occurred()) throw Refused{};
  const at::Tensor *out = tensor(arg[10], "out", true), *lse = tensor(arg[11], "lse", true);
  const at::Device dev = device_of(q, "q", {parts[0], parts[1], parts[2], parts[3], &table, &lengths,
                                            out, lse});
  const fp8q_paged_cache cache = cache_of(parts);
  const Heads qh = head_rows(q, "q");
  if (qh.dim != cache.head_dim || cache.heads < 1 || qh.heads < 1 || qh.heads % cache.heads != 0)
    refuse("q: expected [batch, a multiple of %lld heads, %lld]", (long long)cache.heads,
           (long long)cache.head_dim);
  if (lengths.scalar_type() != at::kInt || lengths.numel() != qh.tokens || !lengths.is_contiguous())
    refuse("lengths: expected %lld contiguous int32 values", (long long)qh.tokens);
  const Table t = table_of(table, qh.tokens);
  if (lse && !want_lse) refuse("lse: given without return_lse");
  const std::array<int64_t, 3> shape{qh.tokens, qh.heads, qh.dim};
  Out o(out, arg[10], shape, at::kBFloat16, "out");
  std::optional<Out> l;
  if (want_lse) l.emplace(lse, arg[11], at::IntArrayRef(shape).slice(0, 2), at::kFloat, "lse");
  int status = 0;
  at::Tensor workspace;  // (stays this stream's when it goes: later work of the stream may take it)
  {
    Unlocked unlocked;
    const int64_t bytes = g_attn_size(&cache, qh.tokens, qh.heads, t.width);
    void* wp = nullptr;
    if (bytes > 0) {
      workspace = at::detail::empty_cuda({bytes}, at::kByte, dev, std::nullopt);
      wp = workspace.data_ptr();
    }
    void* op = o.data(dev);
    float* lp = l ? static_cast<float*>(l->data(dev)) : nullptr;
    status = g_attn(op, lp, q.data_ptr(), qh.ld, &cache, t.p, t.ld, t.width,
                    static_cast<const int32_t*>(lengths.data_ptr()), qh.tokens, qh.heads,
                    own_scale ? float(scale) : 1.0f / std::sqrt(float(qh.dim)), window, wp,
                    bytes > 0 ? bytes : 0, c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  }
  check(status, "fp8q_paged_attention");
  return l ? results({&o, &*l}) : o.object();
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

// init_cache(rope, write, read, attention, workspace): the paged cache's entry points
PyObject* init_cache(PyObject* const* arg, Py_ssize_t n) {
  arguments(n, 5);
  void* f[5];
  for (int i = 0; i < 5; ++i) f[i] = PyLong_AsVoidPtr(arg[i]);
  if (PyErr_Occurred()) throw Refused{};
  g_rope = reinterpret_cast<RopeFn>(f[0]);
  g_write = reinterpret_cast<WriteFn>(f[1]);
  g_read = reinterpret_cast<ReadFn>(f[2]);
  g_attn = reinterpret_cast<AttnFn>(f[3]);
  g_attn_size = reinterpret_cast<AttnSizeFn>(f[4]);
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

PyMethodDef g_methods[] = {method<init>("init"), method<init_cache>("init_cache"),
                           method<rms_norm_quant>("rms_norm_quant"),
                           method<silu_mul_quant>("silu_mul_quant"),
                           method<int8_matmul>("int8_matmul"), method<qk_norm_rope>("qk_norm_rope"),
                           method<cache_write>("cache_write"), method<cache_read>("cache_read"),
                           method<paged_attention>("paged_attention"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&g_module); }
