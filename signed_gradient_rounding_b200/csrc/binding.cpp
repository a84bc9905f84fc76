// Compiled half of the Python binding, for the 8-bit chain: checks the tensors, allocates
// the outputs and calls the C ABI on the tensors' device and stream.
//
// These calls are also made for single tokens, whose kernels take a few microseconds;
// the same marshalling in Python (ctypes and torch.empty) took 12 to 20 microseconds a
// call, this takes about a third of that.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/ar.h"

namespace {

PyObject* g_ar_error = nullptr;  // the package's ArError, set by set_error_type

struct Refused : std::runtime_error {  // -> ValueError
  using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python exception is already set

constexpr auto kE4m3 = at::kFloat8_e4m3fn;

std::string str(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

bool none(PyObject* o) { return o == Py_None; }

// The device index of the call's first tensor.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
  return t.get_device();
}

void on(const at::Tensor& t, const char* name, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    throw Refused(std::string(name) + " must be a CUDA tensor on cuda:" + std::to_string(dev));
}

void typed(const at::Tensor& t, const char* name, at::ScalarType dtype) {
  if (t.scalar_type() != dtype)
    throw Refused(std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
}

ar_dtype dtype_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return AR_F32;
  if (t.scalar_type() == at::kBFloat16) return AR_BF16;
  throw Refused(std::string(name) + " must be float32 or bfloat16, got " + c10::toString(t.scalar_type()));
}

// Row pitch (elements) of a matrix whose columns are contiguous.
int64_t pitch(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) throw Refused(std::string(name) + " must be a matrix, got " + str(t.sizes()));
  if (t.size(1) > 1 && t.stride(1) != 1) throw Refused(std::string(name) + " must have contiguous columns");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

int64_t pitch(const at::Tensor& t, const char* name, int dev, int64_t rows, int64_t cols) {
  on(t, name, dev);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    throw Refused(std::string(name) + " must be " + str({rows, cols}) + ", got " + str(t.sizes()));
  return pitch(t, name);
}

// A contiguous tensor of this type and shape.
void* flat(const at::Tensor& t, const char* name, int dev, at::ScalarType dtype, at::IntArrayRef shape) {
  on(t, name, dev);
  typed(t, name, dtype);
  if (t.sizes() != shape || !t.is_contiguous())
    throw Refused(std::string(name) + " must be a contiguous tensor " + str(shape) + ", got " + str(t.sizes()));
  return t.data_ptr();
}

// Row pitch of a stack of matrices [count, rows, cols] that follow one another.
int64_t stack_pitch(const at::Tensor& t, const char* name) {
  if (t.dim() != 3) throw Refused(std::string(name) + " must be a stack of matrices, got " + str(t.sizes()));
  const int64_t p = t.size(1) > 1 ? t.stride(1) : t.size(2);
  if ((t.size(2) > 1 && t.stride(2) != 1) || (t.size(0) > 1 && t.stride(0) != p * t.size(1)))
    throw Refused(std::string(name) + " must have contiguous columns, and matrices that follow one another");
  return p;
}

// The bytes of a matrix.
struct Bytes {
  uintptr_t at;
  int64_t rows, width, pitch;
  bool same(const Bytes& o) const { return at == o.at && (pitch == o.pitch || rows <= 1); }
};

Bytes bytes_of(const at::Tensor& t, int64_t ld) {  // (the last axis is a row, all others are rows)
  const int64_t el = static_cast<int64_t>(t.element_size()), cols = t.size(-1);
  return {reinterpret_cast<uintptr_t>(t.data_ptr()), cols > 0 ? t.numel() / cols : 0, cols * el, ld * el};
}

Bytes bytes_of(const at::Tensor& t) {  // contiguous
  return {reinterpret_cast<uintptr_t>(t.data_ptr()), 1, t.numel() * static_cast<int64_t>(t.element_size()), 0};
}

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }

// Whether the two have a byte in common.  Rows of either may lie between rows of the other.
bool meet(const Bytes& a, const Bytes& b) {
  if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  if ((a.rows > 1 && a.pitch < a.width) || (b.rows > 1 && b.pitch < b.width)) return false;  // (the library refuses these)
  const int64_t gap = static_cast<int64_t>(a.at - b.at);  // of a's first row behind b's
  if (gap >= (b.rows - 1) * b.pitch + b.width || -gap >= (a.rows - 1) * a.pitch + a.width) return false;
  if (a.rows > 1 && b.rows > 1 && a.pitch == b.pitch) {
    // row i of a and row j of b meet where -a.width < gap + (i - j) pitch < b.width
    const int64_t lo = floor_div(-a.width - gap, a.pitch) + 1, hi = -floor_div(gap - b.width, a.pitch) - 1;
    return std::max(lo, 1 - b.rows) <= std::min(hi, a.rows - 1);
  }
  if (a.rows > b.rows) return meet(b, a);
  for (int64_t i = 0; i < a.rows; ++i) {  // rows j of b: -a.width < gap + i a.pitch - j b.pitch < b.width
    const int64_t from = gap + i * a.pitch;
    if (b.rows == 1) {
      if (from > -a.width && from < b.width) return true;
      continue;
    }
    const int64_t lo = floor_div(from - b.width, b.pitch) + 1, hi = -floor_div(-from - a.width, b.pitch) - 1;
    if (std::max<int64_t>(lo, 0) <= std::min(hi, b.rows - 1)) return true;
  }
  return false;
}

void apart(const Bytes& out, const char* out_name, const Bytes& in, const char* name) {
  if (meet(out, in)) throw Refused(std::string(out_name) + " must not overlap " + name);
}

// An output that may be this input itself, and must not overlap it otherwise.
void same_or_apart(const Bytes& out, const char* out_name, const Bytes& in, const char* name) {
  if (!out.same(in) && meet(out, in))
    throw Refused(std::string(out_name) + " must be " + name + " itself, with its pitch, or not overlap it");
}

int32_t* status_of(PyObject* o, int dev) {
  if (none(o)) return nullptr;
  const at::Tensor& t = tensor(o, "status");
  on(t, "status", dev);
  typed(t, "status", at::kInt);
  if (t.numel() < 1) throw Refused("status must have an element");
  return t.data_ptr<int32_t>();
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, int dev) {
  return at::detail::empty_cuda(shape, dtype, c10::Device(c10::kCUDA, dev), std::nullopt);
}

// The call's stream: a torch.cuda.Stream, or the device's current one (None).  A given stream is the
// current one while this lives, so that the call's new tensors come from its pool: memory that was
// freed on another stream may still be in use there.
class CallStream {
 public:
  CallStream(PyObject* o, int dev) : before_(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev))) {
    if (none(o)) {
      ptr_ = before_.stream();
      return;
    }
    PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) throw Raised();
    ptr_ = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw Raised();
    guard_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(ptr_), static_cast<c10::DeviceIndex>(dev)));
  }
  void* get() const { return ptr_; }

  // After the launch on a given stream: the memory of the tensors that it was given is not handed out
  // again before that stream is done with them, nor that of the new ones, which the caller goes on to
  // use on the stream that was current, before that one is.
  void used(std::initializer_list<const at::Tensor*> given, std::initializer_list<const at::Tensor*> made) const {
    if (!guard_) return;
    record(given, guard_->current_stream());
    record(made, before_);
  }

 private:
  static void record(std::initializer_list<const at::Tensor*> tensors, c10::cuda::CUDAStream stream) {
    for (const at::Tensor* t : tensors)
      if (t && t->defined() && t->numel() > 0)
        c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), stream);
  }

  c10::cuda::CUDAStream before_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
  void* ptr_ = nullptr;
};

const at::Tensor* maybe(PyObject* o) { return none(o) ? nullptr : &THPVariable_Unpack(o); }

// Run the call with the tensors' device current; raise ArError unless it is AR_OK.
template <class F>
void launch(int dev, const char* what, F&& call) {
  ar_status s;
  if (c10::cuda::current_device() == dev) {
    s = call();
  } else {
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    s = call();
  }
  if (s == AR_OK) return;
  PyObject* e = PyObject_CallFunction(g_ar_error, "is", static_cast<int>(s), what);
  if (e) {
    PyErr_SetObject(g_ar_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

template <class... T>
PyObject* wrap_all(const T&... t) {
  PyObject* tuple = PyTuple_New(sizeof...(t));
  if (!tuple) return nullptr;
  Py_ssize_t i = 0;
  bool ok = true;
  auto put = [&](const at::Tensor& x) {
    PyObject* o = wrap(x);
    if (!o) ok = false;
    PyTuple_SET_ITEM(tuple, i++, o);
  };
  (put(t), ...);
  if (!ok) {
    Py_DECREF(tuple);
    return nullptr;
  }
  return tuple;
}

// No C++ exception leaves an entry point.
template <class F>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, F&& body) {
  if (nargs != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, nargs);
    return nullptr;
  }
  try {
    return body();
  } catch (const Raised&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* type = nullptr;
    if (PyObject* torch = PyImport_ImportModule("torch")) {
      type = PyObject_GetAttrString(torch, "OutOfMemoryError");
      Py_DECREF(torch);
    }
    PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    return nullptr;
  }
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

// (x, weight, eps, residual, want_bf16, want_scaled, sum_out, stream) -> (y, q, scale, h)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const int dev = device_of(x, "x");
    const CallStream st(a[7], dev);
    const ar_dtype xd = dtype_of(x, "x");
    const int64_t ldx = pitch(x, "x"), rows = x.size(0), cols = x.size(1);
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    const bool want_y = truth(a[4]), want_q = truth(a[5]);
    const void* rp = nullptr;
    ar_dtype rd = xd, wd = AR_BF16;
    int64_t ldr = cols, lds = cols;
    at::Tensor h;
    if (!none(a[3])) {
      const at::Tensor& r = tensor(a[3], "residual");
      ldr = pitch(r, "residual", dev, rows, cols);
      rd = dtype_of(r, "residual");
      rp = r.data_ptr();
      if (none(a[6])) {
        h = empty({rows, cols}, r.scalar_type(), dev);
      } else {
        h = tensor(a[6], "sum_out");
        lds = pitch(h, "sum_out", dev, rows, cols);
        typed(h, "sum_out", r.scalar_type());
        apart(bytes_of(h, lds), "sum_out", bytes_of(x, ldx), "x");
        same_or_apart(bytes_of(h, lds), "sum_out", bytes_of(r, ldr), "residual");
      }
    } else if (!none(a[6])) {
      throw Refused("sum_out needs a residual");
    }
    const void* wp = nullptr;
    if (!none(a[1])) {
      const at::Tensor& w = tensor(a[1], "weight");
      wd = dtype_of(w, "weight");
      wp = flat(w, "weight", dev, w.scalar_type(), {cols});
      if (!none(a[6])) apart(bytes_of(h, lds), "sum_out", bytes_of(w), "weight");
    }
    at::Tensor y, q, s;
    if (want_y) y = empty({rows, cols}, at::kBFloat16, dev);
    if (want_q) {
      q = empty({rows, cols}, kE4m3, dev);
      s = empty({rows, blocks_of(cols)}, at::kFloat, dev);
    }
    launch(dev, "ar_rms_norm", [&] {
      return ar_rms_norm(x.data_ptr(), xd, ldx, rows, cols, rp, rd, ldr, wp, wd, static_cast<float>(eps),
                         h.defined() ? h.data_ptr() : nullptr, lds,
                         want_y ? static_cast<uint16_t*>(y.data_ptr()) : nullptr, cols,
                         want_q ? static_cast<uint8_t*>(q.data_ptr()) : nullptr, cols,
                         want_q ? s.data_ptr<float>() : nullptr, st.get());
    });
    st.used({&x, maybe(a[1]), maybe(a[3]), maybe(a[6])}, {&y, &q, &s, none(a[6]) ? &h : nullptr});
    return wrap_all(y, q, s, h);
  });
}

// (x, block_rows, stream) -> (q, scale)
PyObject* quant_scaled(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 3, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const int dev = device_of(x, "x");
    const ar_dtype xd = dtype_of(x, "x");
    const CallStream st(a[2], dev);
    // (anything else than the two becomes 0, which the library refuses: a number past 32 bits must not become one of them)
    const int64_t asked = integer(a[1]), block_rows = asked == 1 || asked == 128 ? asked : 0;
    const bool stack = x.dim() == 3;
    const int64_t ldx = stack ? stack_pitch(x, "x") : pitch(x, "x");
    const int64_t count = stack ? x.size(0) : 1, rows = x.size(-2), cols = x.size(-1);
    const int64_t rb = block_rows == 1 ? rows : blocks_of(rows), cb = blocks_of(cols);
    at::Tensor q = empty(x.sizes(), kE4m3, dev);
    at::Tensor s = stack ? empty({count, rb, cb}, at::kFloat, dev) : empty({rb, cb}, at::kFloat, dev);
    launch(dev, "ar_quant_scaled", [&] {
      return ar_quant_scaled(x.data_ptr(), xd, ldx, count, rows, cols, static_cast<int32_t>(block_rows),
                             static_cast<uint8_t*>(q.data_ptr()), cols, s.data_ptr<float>(), st.get());
    });
    st.used({&x}, {&q, &s});
    return wrap_all(q, s);
  });
}

// (a, b, stream) -> (q, scale)
PyObject* silu_mul_scaled(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded(nargs, 3, [&]() -> PyObject* {
    const at::Tensor &a = tensor(args[0], "a"), &b = tensor(args[1], "b");
    const int dev = device_of(a, "a");
    const CallStream st(args[2], dev);
    typed(a, "a", at::kBFloat16);
    const int64_t lda = pitch(a, "a"), rows = a.size(0), cols = a.size(1);
    const int64_t ldb = pitch(b, "b", dev, rows, cols);
    typed(b, "b", at::kBFloat16);
    at::Tensor q = empty({rows, cols}, kE4m3, dev), s = empty({rows, blocks_of(cols)}, at::kFloat, dev);
    launch(dev, "ar_silu_mul_scaled", [&] {
      return ar_silu_mul_scaled(static_cast<const uint16_t*>(a.data_ptr()), lda,
                                static_cast<const uint16_t*>(b.data_ptr()), ldb, rows, cols,
                                static_cast<uint8_t*>(q.data_ptr()), cols, s.data_ptr<float>(), st.get());
    });
    st.used({&a, &b}, {&q, &s});
    return wrap_all(q, s);
  });
}

// The output: `o`, or a new matrix; its row pitch in *ldy.
at::Tensor output(PyObject* o, int dev, int64_t rows, int64_t cols, int64_t* ldy) {
  if (none(o)) {
    *ldy = cols;
    return empty({rows, cols}, at::kBFloat16, dev);
  }
  const at::Tensor& t = tensor(o, "out");
  *ldy = pitch(t, "out", dev, rows, cols);
  typed(t, "out", at::kBFloat16);
  return t;
}

// The same object for an output that was passed in.
PyObject* result(PyObject* o, const at::Tensor& t) {
  if (none(o)) return wrap(t);
  Py_INCREF(o);
  return o;
}

// (Xq, x_scale, Wq, w_scale, add, out, status, stream) -> Y
PyObject* linear_scaled(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const at::Tensor &X = tensor(a[0], "Xq"), &W = tensor(a[2], "Wq");
    const int dev = device_of(X, "Xq");
    const CallStream st(a[7], dev);
    typed(X, "Xq", kE4m3);
    typed(W, "Wq", kE4m3);
    on(W, "Wq", dev);
    const int64_t ldx = pitch(X, "Xq"), ldw = pitch(W, "Wq");
    const int64_t n = X.size(0), in = X.size(1), out = W.size(0), nb = blocks_of(in);
    if (W.size(1) != in) throw Refused("Wq must be [out, " + std::to_string(in) + "], got " + str(W.sizes()));
    const void* xs = flat(tensor(a[1], "x_scale"), "x_scale", dev, at::kFloat, {n, nb});
    const void* ws = flat(tensor(a[3], "w_scale"), "w_scale", dev, at::kFloat, {blocks_of(out), nb});
    const void* add = nullptr;
    int64_t ldadd = out, ldy = out;
    if (!none(a[4])) {
      const at::Tensor& t = tensor(a[4], "add");
      ldadd = pitch(t, "add", dev, n, out);
      typed(t, "add", at::kBFloat16);
      add = t.data_ptr();
    }
    int32_t* status = status_of(a[6], dev);
    at::Tensor Y = output(a[5], dev, n, out, &ldy);
    if (!none(a[5])) {
      const Bytes y = bytes_of(Y, ldy);
      apart(y, "out", bytes_of(X, ldx), "Xq");
      apart(y, "out", bytes_of(W, ldw), "Wq");
      apart(y, "out", bytes_of(THPVariable_Unpack(a[1])), "x_scale");
      apart(y, "out", bytes_of(THPVariable_Unpack(a[3])), "w_scale");
      if (add) same_or_apart(y, "out", bytes_of(THPVariable_Unpack(a[4]), ldadd), "add");
    }
    launch(dev, "ar_linear_scaled", [&] {
      return ar_linear_scaled(static_cast<const uint8_t*>(X.data_ptr()), ldx, static_cast<const float*>(xs), n, in,
                              static_cast<const uint8_t*>(W.data_ptr()), ldw, static_cast<const float*>(ws), out,
                              static_cast<const uint16_t*>(add), ldadd, static_cast<uint16_t*>(Y.data_ptr()), ldy, status,
                              st.get());
    });
    st.used({&X, maybe(a[1]), &W, maybe(a[3]), maybe(a[4]), maybe(a[5]), maybe(a[6])}, {none(a[5]) ? &Y : nullptr});
    return result(a[5], Y);
  });
}

// (X, offsets, W_hi, W_lo, out, status, stream) -> Y
PyObject* grouped_linear(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 7, [&]() -> PyObject* {
    const at::Tensor &X = tensor(a[0], "X"), &W = tensor(a[2], "W_hi");
    const int dev = device_of(X, "X");
    const CallStream st(a[6], dev);
    typed(X, "X", at::kBFloat16);
    typed(W, "W_hi", at::kBFloat16);
    on(W, "W_hi", dev);
    const int64_t ldx = pitch(X, "X"), ldw = stack_pitch(W, "W_hi");
    const int64_t n = X.size(0), in = X.size(1), experts = W.size(0), out = W.size(1);
    if (W.size(2) != in) throw Refused("W_hi must be [experts, out, " + std::to_string(in) + "], got " + str(W.sizes()));
    const void* lo = nullptr;
    if (!none(a[3])) {
      const at::Tensor& L = tensor(a[3], "W_lo");
      on(L, "W_lo", dev);
      typed(L, "W_lo", at::kBFloat16);
      if (L.sizes() != W.sizes() || stack_pitch(L, "W_lo") != ldw)
        throw Refused("W_lo must have the shape and strides of W_hi");
      lo = L.data_ptr();
    }
    const void* offsets = flat(tensor(a[1], "offsets"), "offsets", dev, at::kInt, {experts + 1});
    int32_t* status = status_of(a[5], dev);
    int64_t ldy = out;
    at::Tensor Y = output(a[4], dev, n, out, &ldy);
    if (!none(a[4])) {
      const Bytes y = bytes_of(Y, ldy);
      apart(y, "out", bytes_of(X, ldx), "X");
      apart(y, "out", bytes_of(W, ldw), "W_hi");
      if (lo) apart(y, "out", bytes_of(THPVariable_Unpack(a[3]), ldw), "W_lo");
      apart(y, "out", bytes_of(THPVariable_Unpack(a[1])), "offsets");
    }
    launch(dev, "ar_grouped_linear", [&] {
      return ar_grouped_linear(static_cast<const uint16_t*>(X.data_ptr()), ldx, n, in,
                               static_cast<const int32_t*>(offsets), experts,
                               static_cast<const uint16_t*>(W.data_ptr()), static_cast<const uint16_t*>(lo), ldw, out,
                               static_cast<uint16_t*>(Y.data_ptr()), ldy, status, st.get());
    });
    st.used({&X, maybe(a[1]), &W, maybe(a[3]), maybe(a[4]), maybe(a[5])}, {none(a[4]) ? &Y : nullptr});
    return result(a[4], Y);
  });
}

// (Xq, x_scale, offsets, Wq, w_scale, out, status, stream) -> Y
PyObject* grouped_linear_scaled(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const at::Tensor &X = tensor(a[0], "Xq"), &W = tensor(a[3], "Wq");
    const int dev = device_of(X, "Xq");
    const CallStream st(a[7], dev);
    typed(X, "Xq", kE4m3);
    typed(W, "Wq", kE4m3);
    on(W, "Wq", dev);
    const int64_t ldx = pitch(X, "Xq"), ldw = stack_pitch(W, "Wq");
    const int64_t n = X.size(0), in = X.size(1), experts = W.size(0), out = W.size(1), nb = blocks_of(in);
    if (W.size(2) != in) throw Refused("Wq must be [experts, out, " + std::to_string(in) + "], got " + str(W.sizes()));
    const void* xs = flat(tensor(a[1], "x_scale"), "x_scale", dev, at::kFloat, {n, nb});
    const void* ws = flat(tensor(a[4], "w_scale"), "w_scale", dev, at::kFloat, {experts, blocks_of(out), nb});
    const void* offsets = flat(tensor(a[2], "offsets"), "offsets", dev, at::kInt, {experts + 1});
    int32_t* status = status_of(a[6], dev);
    int64_t ldy = out;
    at::Tensor Y = output(a[5], dev, n, out, &ldy);
    if (!none(a[5])) {
      const Bytes y = bytes_of(Y, ldy);
      apart(y, "out", bytes_of(X, ldx), "Xq");
      apart(y, "out", bytes_of(W, ldw), "Wq");
      apart(y, "out", bytes_of(THPVariable_Unpack(a[1])), "x_scale");
      apart(y, "out", bytes_of(THPVariable_Unpack(a[4])), "w_scale");
      apart(y, "out", bytes_of(THPVariable_Unpack(a[2])), "offsets");
    }
    launch(dev, "ar_grouped_linear_scaled", [&] {
      return ar_grouped_linear_scaled(static_cast<const uint8_t*>(X.data_ptr()), ldx, static_cast<const float*>(xs), n, in,
                                      static_cast<const int32_t*>(offsets), experts,
                                      static_cast<const uint8_t*>(W.data_ptr()), ldw, static_cast<const float*>(ws), out,
                                      static_cast<uint16_t*>(Y.data_ptr()), ldy, status, st.get());
    });
    st.used({&X, maybe(a[1]), maybe(a[2]), &W, maybe(a[4]), maybe(a[5]), maybe(a[6])}, {none(a[5]) ? &Y : nullptr});
    return result(a[5], Y);
  });
}

PyObject* set_error_type(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_ar_error);
  g_ar_error = type;
  Py_RETURN_NONE;
}

#define AR_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {AR_FAST(rms_norm),
                           AR_FAST(quant_scaled),
                           AR_FAST(silu_mul_scaled),
                           AR_FAST(linear_scaled),
                           AR_FAST(grouped_linear),
                           AR_FAST(grouped_linear_scaled),
                           {"set_error_type", set_error_type, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
