// CPython module fp8_rowwise_scaled_amd._layer_binding: torch tensors in, the C ABI of
// fp8gg_layer.h, torch tensors out.
//
// A decode step's calls run 3 to 5 us on the GPU.  Checked and allocated from Python
// they took 9 to 13 us of host time each (one allocation 1.3 to 1.6 us, a tensor's check
// 0.3 us); here a norm with four outputs takes 6, the launch itself about 3.
//
// Arguments come in the fixed order that layer.py hands on.  Every tensor is checked
// (type, shape, device, layout) before the library is called, which checks the rest;
// outputs that are None are allocated on the inputs' device, and the work goes to that
// device's current stream.  Errors become ValueError, or RuntimeError for a launch that
// failed; C++ exceptions (an allocation that fails) become torch's Python errors.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <string>

#include "fp8gg_layer.h"

namespace {

// A refusal, thrown to the entry point and turned into ValueError there.
struct Refused {
  std::string what;
};

[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  throw Refused{buf};
}

using Shape = std::initializer_list<int64_t>;

std::string text(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return c10::toString(t);
  }
}

// The interpreter's lock given up for a scope, however it is left.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// One call's arguments: a cursor over them, the first tensor's device, and the outputs.
class Call {
 public:
  Call(const char* name, PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : name_(name), args_(args) {
    if (n != want) refuse("%s takes %zd arguments, got %zd", name, want, n);
  }

  // The next argument as a tensor; null where it may be missing and is None.
  const at::Tensor* tensor(const char* what, bool optional = false) {
    PyObject* o = args_[at_++];
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", what);
    return &THPVariable_Unpack(o);
  }
  int64_t integer() {
    const long long v = PyLong_AsLongLong(args_[at_++]);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
  }
  double number() {
    const double v = PyFloat_AsDouble(args_[at_++]);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
  }
  bool flag() {
    const int v = PyObject_IsTrue(args_[at_++]);
    if (v < 0) throw python_error();
    return v != 0;
  }
  bool none(Py_ssize_t ahead = 0) const { return args_[at_ + ahead] == Py_None; }

  // Type, rank, place and layout of an input; the first one decides the device.
  void check(const at::Tensor& t, const char* what, at::ScalarType type, int64_t dim, const char* shape) {
    if (t.scalar_type() != type) refuse("%s must be %s, got %s", what, name_of(type), name_of(t.scalar_type()));
    if (t.dim() != dim) refuse("%s must be %s", what, shape);
    place(t, what);
  }
  void check(const at::Tensor& t, const char* what, at::ScalarType type, Shape shape) {
    if (t.scalar_type() != type) refuse("%s must be %s, got %s", what, name_of(type), name_of(t.scalar_type()));
    if (!t.sizes().equals(c10::IntArrayRef(shape.begin(), shape.size())))
      refuse("%s must have shape %s, got %s", what, text(c10::IntArrayRef(shape.begin(), shape.size())).c_str(),
             text(t.sizes()).c_str());
    place(t, what);
  }
  // fp8 codes: uint8 or float8_e4m3fn.
  void check_codes(const at::Tensor& t, const char* what, Shape shape) {
    check(t, what, t.scalar_type() == at::kFloat8_e4m3fn ? at::kFloat8_e4m3fn : at::kByte, shape);
  }
  int float_type(const at::Tensor& t, const char* what) {
    if (t.scalar_type() == at::kBFloat16) return FP8GG_DTYPE_BF16;
    if (t.scalar_type() != at::kFloat) refuse("%s must be bfloat16 or float32, got %s", what, name_of(t.scalar_type()));
    return FP8GG_DTYPE_F32;
  }

  // The next argument as an output: the caller's, checked, or a new one.  float8 buffers
  // come back as the uint8 view that codes are everywhere.
  at::Tensor output(const char* what, at::ScalarType type, Shape shape) {
    const at::Tensor* given = tensor(what, true);
    if (!given) return fresh(type, shape);
    if (type == at::kByte && given->scalar_type() == at::kFloat8_e4m3fn) {
      check(*given, what, at::kFloat8_e4m3fn, shape);
      return given->view(at::kByte);
    }
    check(*given, what, type, shape);
    return *given;
  }
  // A new tensor straight from torch's GPU allocator, on the current device (which place()
  // has set): 0.2 us, where at::empty's way through the dispatcher takes 0.7.
  at::Tensor fresh(at::ScalarType type, Shape shape) {
    static c10::Allocator* const allocator = [this] {
      // past the dispatcher's Python modes: one of them (a tracer's) may be on in the first call
      const c10::impl::ExcludeDispatchKeyGuard no_modes(
          c10::DispatchKeySet({c10::DispatchKey::Python, c10::DispatchKey::PythonTLSSnapshot}));
      return at::empty({1}, at::TensorOptions().dtype(at::kByte).device(device_)).storage().allocator();
    }();
    return at::Tensor(at::detail::empty_generic(c10::IntArrayRef(shape.begin(), shape.size()), allocator,
                                                c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
  }
  // The next argument as a workspace of `need` bytes.  A new one may be released when the
  // call returns: the allocator hands it out again in the stream's order.
  at::Tensor workspace(int64_t need) {
    const at::Tensor* given = tensor("workspace", true);
    if (!given) return need > 0 ? fresh(at::kByte, {need}) : at::Tensor();
    place(*given, "workspace");
    return *given;
  }

  // Makes the library's call on the tensors' device and its current stream, without the
  // interpreter's lock.  The library throws nothing, but a tensor that has no memory (one of
  // a tracer's) throws when it is asked for its address.
  template <typename Library>
  void run(Library library) const {
    void* stream = c10::hip::getCurrentHIPStream(device_.index()).stream();
    fp8gg_status st;
    {
      const Unlocked unlocked;
      st = library(stream);
    }
    if (st == FP8GG_OK) return;
    const std::string what = std::string(name_) + ": " + f8f8bf16_layer_last_error();
    if (st == FP8GG_ERR_HIP) throw std::runtime_error(what);
    throw Refused{what};
  }

 private:
  void place(const at::Tensor& t, const char* what) {
    if (!t.is_cuda()) refuse("%s must be on the GPU", what);
    if (!t.is_contiguous()) refuse("%s must be contiguous", what);
    if (!placed_) {
      device_ = t.device();
      guard_.reset_device(device_);
      placed_ = true;
    } else if (t.device() != device_) {
      refuse("all tensors must be on one device: %s is on %s, not %s", what, t.device().str().c_str(),
             device_.str().c_str());
    }
  }

  const char* name_;
  PyObject* const* args_;
  Py_ssize_t at_ = 0;
  c10::Device device_{c10::DeviceType::CPU};
  c10::OptionalDeviceGuard guard_;       // the tensors' device is the current one for the call
  bool placed_ = false;
};

template <typename T>
T* ptr(const at::Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}
template <typename T>
const T* ptr(const at::Tensor* t) {
  return t ? static_cast<const T*>(t->data_ptr()) : nullptr;
}

// New references in a tuple; an undefined tensor is None.
PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
template <typename... Ts>
PyObject* pack(const Ts&... ts) {
  PyObject* tuple = PyTuple_New(sizeof...(ts));
  if (!tuple) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(tuple, i++, wrap(ts)), ...);
  return tuple;
}

int64_t block_cols(int64_t block, int64_t width) {
  if (block != 0 && block != 128) refuse("block must be 0 (one scale per row) or 128, got %lld", (long long)block);
  if (block && width % 128) refuse("block scaling needs a multiple of 128 columns, got %lld", (long long)width);
  return block ? width / 128 : 0;
}

at::Tensor scales(Call& c, const char* what, int64_t rows, int64_t cols) {
  return cols ? c.output(what, at::kFloat, {rows, cols}) : c.output(what, at::kFloat, {rows});
}

PyObject* rmsnorm_quantize(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_rmsnorm_quantize", args, n, 12);
  const at::Tensor& X = *c.tensor("X");
  c.check(X, "X", at::kBFloat16, 2, "[rows, K]");
  const int64_t rows = X.size(0), K = X.size(1);
  const at::Tensor& weight = *c.tensor("weight");
  const int wt = c.float_type(weight, "weight");
  c.check(weight, "weight", weight.scalar_type(), {K});
  const double eps = c.number();
  const at::Tensor* residual = c.tensor("residual", true);
  if (residual) c.check(*residual, "residual", at::kBFloat16, {rows, K});
  const int64_t block = c.integer();
  const int64_t cols = block_cols(block, K);
  const bool want_y = c.flag(), want_rstd = c.flag();
  const at::Tensor XQ = c.output("XQ", at::kByte, {rows, K});
  const at::Tensor x_scale = scales(c, "x_scale", rows, cols);
  at::Tensor residual_out, Y, rstd;
  if (residual) residual_out = c.output("residual_out", at::kBFloat16, {rows, K});
  else if (c.tensor("residual_out", true)) refuse("residual_out is given without a residual");
  if (want_y || !c.none()) Y = c.output("Y", at::kBFloat16, {rows, K});
  else c.tensor("Y", true);
  if (want_rstd || !c.none()) rstd = c.output("rstd", at::kFloat, {rows});
  else c.tensor("rstd", true);
  c.run([&](void* stream) {
    return f8f8bf16_rmsnorm_quantize(
      ptr<uint16_t>(&X), ptr<uint16_t>(residual), weight.data_ptr(), wt, (float)eps, (int)block, ptr<uint8_t>(XQ),
      ptr<float>(x_scale), ptr<uint16_t>(Y), ptr<uint16_t>(residual_out), ptr<float>(rstd), rows, K, stream);
  });
  return pack(XQ, x_scale, residual_out, Y, rstd);
}

PyObject* rmsnorm_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_rmsnorm_backward", args, n, 8);
  const at::Tensor& dY = *c.tensor("dY");
  c.check(dY, "dY", at::kBFloat16, 2, "[rows, K]");
  const int64_t rows = dY.size(0), K = dY.size(1);
  const at::Tensor& H = *c.tensor("H");
  c.check(H, "H", at::kBFloat16, {rows, K});
  const at::Tensor& weight = *c.tensor("weight");
  const int wt = c.float_type(weight, "weight");
  c.check(weight, "weight", weight.scalar_type(), {K});
  const at::Tensor& rstd = *c.tensor("rstd");
  c.check(rstd, "rstd", at::kFloat, {rows});
  const at::Tensor* dres = c.tensor("dresidual", true);
  if (dres) c.check(*dres, "dresidual", at::kBFloat16, {rows, K});
  const at::Tensor dX = c.output("dX", at::kBFloat16, {rows, K});
  const at::Tensor dweight = c.output("dweight", at::kFloat, {K});
  const at::Tensor ws = c.workspace(f8f8bf16_rmsnorm_backward_workspace(rows, K));
  c.run([&](void* stream) {
    return f8f8bf16_rmsnorm_backward(
      ptr<uint16_t>(&dY), ptr<uint16_t>(&H), weight.data_ptr(), wt, ptr<float>(&rstd), ptr<uint16_t>(dres),
      ptr<uint16_t>(dX), ptr<float>(dweight), ptr<void>(ws), ws.defined() ? (int64_t)ws.nbytes() : 0, rows, K, stream);
  });
  return pack(dX, dweight);
}

// logits: [T, E] of either float type.
const at::Tensor& logits_of(Call& c, int& dtype) {
  const at::Tensor& x = *c.tensor("logits");
  dtype = c.float_type(x, "logits");
  c.check(x, "logits", x.scalar_type(), 2, "[T, E]");
  return x;
}

PyObject* route(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_route", args, n, 15);
  int dtype;
  const at::Tensor& logits = logits_of(c, dtype);
  const int64_t T = logits.size(0), E = logits.size(1), k = c.integer();
  // before anything of that size is allocated
  if (k < 0) refuse("k must not be negative, got %lld", (long long)k);
  if (k > E) refuse("k=%lld exceeds the number of experts, E=%lld", (long long)k, (long long)E);
  const at::Tensor* bias = c.tensor("bias", true);
  if (bias) c.check(*bias, "bias", at::kFloat, {E});
  const int64_t score = c.integer(), n_group = c.integer(), topk_group = c.integer(), group_top = c.integer();
  // here, because the library takes an int
  if (group_top != 1 && group_top != 2) refuse("group_top=%lld must be 1 or 2", (long long)group_top);
  const bool renormalize = c.flag();
  const double scale = c.number();
  const bool plan = c.flag();
  const at::Tensor weights = c.output("weights", at::kFloat, {T, k});
  const at::Tensor ids = c.output("ids", at::kInt, {T, k});
  at::Tensor M_sizes, dst_row, ws;
  if (plan) {
    M_sizes = c.output("M_sizes", at::kLong, {E});
    dst_row = c.output("dst_row", at::kInt, {T, k});
    ws = c.workspace(f8f8bf16_route_workspace(T, E, k));
  } else if (!c.none(0) || !c.none(1)) {
    refuse("M_sizes and dst_row are outputs of the plan, which plan=False leaves out");
  }
  c.run([&](void* stream) {
    return f8f8bf16_route(
      logits.data_ptr(), dtype, ptr<float>(bias), (int)score, n_group, topk_group, (int)group_top, renormalize,
      (float)scale, ptr<float>(weights), ptr<int32_t>(ids), ptr<int64_t>(M_sizes), ptr<int32_t>(dst_row), ptr<void>(ws),
      ws.defined() ? (int64_t)ws.nbytes() : 0, T, E, k, stream);
  });
  return pack(weights, ids, M_sizes, dst_row);
}

PyObject* route_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_route_backward", args, n, 7);
  int dtype;
  const at::Tensor& logits = logits_of(c, dtype);
  const int64_t T = logits.size(0), E = logits.size(1);
  const at::Tensor& ids = *c.tensor("ids");
  c.check(ids, "ids", at::kInt, 2, "[T, k]");
  const int64_t k = ids.size(1);
  c.check(ids, "ids", at::kInt, {T, k});
  const at::Tensor& dweights = *c.tensor("dweights");
  c.check(dweights, "dweights", at::kFloat, {T, k});
  const int64_t score = c.integer();
  const bool renormalize = c.flag();
  const double scale = c.number();
  const at::Tensor dlogits = c.output("dlogits", logits.scalar_type(), {T, E});
  c.run([&](void* stream) {
    return f8f8bf16_route_backward(logits.data_ptr(), dtype, ptr<int32_t>(&ids), ptr<float>(&dweights), (int)score,
                                 renormalize, (float)scale, dlogits.data_ptr(), T, E, k, stream);
  });
  return wrap(dlogits);
}

// dst_row: [T, k], T given or (-1) its own.
const at::Tensor& places_of(Call& c, int64_t T, int64_t& k) {
  const at::Tensor& dst = *c.tensor("dst_row");
  c.check(dst, "dst_row", at::kInt, 2, "[T, k]");
  k = dst.size(1);
  if (T >= 0) c.check(dst, "dst_row", at::kInt, {T, k});
  return dst;
}

// rows: an integer, or T * k for None.
int64_t rows_of(Call& c, int64_t T, int64_t k) {
  if (c.none()) {
    c.tensor("rows", true);
    return T * k;
  }
  const int64_t rows = c.integer();
  if (rows < 0) refuse("rows must not be negative, got %lld", (long long)rows);
  // the library's bound, before anything of that size is allocated
  if (rows > (int64_t(1) << 31) - 256) refuse("rows=%lld is too large", (long long)rows);
  return rows;
}

PyObject* moe_dispatch(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_moe_dispatch", args, n, 6);
  const at::Tensor& XQ = *c.tensor("XQ");
  if (XQ.dim() != 2) refuse("XQ must be [T, K]");
  const int64_t T = XQ.size(0), K = XQ.size(1);
  c.check_codes(XQ, "XQ", {T, K});
  const at::Tensor& xs = *c.tensor("x_scale");
  if (xs.dim() != 1 && xs.dim() != 2) refuse("x_scale must be [T] or [T, columns]");
  const int64_t cols = xs.dim() == 2 ? xs.size(1) : 1;
  if (xs.dim() == 2) c.check(xs, "x_scale", at::kFloat, {T, cols});
  else c.check(xs, "x_scale", at::kFloat, {T});
  int64_t k;
  const at::Tensor& dst = places_of(c, T, k);
  const int64_t R = rows_of(c, T, k);
  const at::Tensor XQs = c.output("XQs", at::kByte, {R, K});
  const at::Tensor out = scales(c, "xs_out", R, xs.dim() == 2 ? cols : 0);
  c.run([&](void* stream) {
    return f8f8bf16_moe_dispatch(ptr<uint8_t>(&XQ), ptr<float>(&xs), cols, ptr<int32_t>(&dst), ptr<uint8_t>(XQs),
                               ptr<float>(out), T, k, R, K, stream);
  });
  return pack(XQs, out);
}

PyObject* moe_combine(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_moe_combine", args, n, 5);
  const at::Tensor& Y = *c.tensor("Y");
  c.check(Y, "Y", at::kBFloat16, 2, "[R, N]");
  const int64_t R = Y.size(0), N = Y.size(1);
  int64_t k;
  const at::Tensor& dst = places_of(c, -1, k);
  const int64_t T = dst.size(0);
  const at::Tensor* weights = c.tensor("weights", true);
  if (weights) c.check(*weights, "weights", at::kFloat, {T, k});
  const at::Tensor* addend = c.tensor("addend", true);
  if (addend) c.check(*addend, "addend", at::kBFloat16, {T, N});
  const at::Tensor out = c.output("out", at::kBFloat16, {T, N});
  c.run([&](void* stream) {
    return f8f8bf16_moe_combine(ptr<uint16_t>(&Y), ptr<int32_t>(&dst), ptr<float>(weights), ptr<uint16_t>(addend),
                              ptr<uint16_t>(out), T, k, R, N, stream);
  });
  return wrap(out);
}

PyObject* moe_combine_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_moe_combine_backward", args, n, 7);
  const at::Tensor& dout = *c.tensor("dout");
  c.check(dout, "dout", at::kBFloat16, 2, "[T, N]");
  const int64_t T = dout.size(0), N = dout.size(1);
  int64_t k;
  const at::Tensor& dst = places_of(c, T, k);
  const at::Tensor* weights = c.tensor("weights", true);
  if (weights) c.check(*weights, "weights", at::kFloat, {T, k});
  const at::Tensor* Y = c.tensor("Y", true);
  const int64_t own = Y && Y->dim() == 2 ? Y->size(0) : -1;
  if (Y) c.check(*Y, "Y", at::kBFloat16, {own, N});
  const bool given = !c.none();
  int64_t R = rows_of(c, T, k);
  if (Y) {
    if (given && R != own) refuse("rows=%lld, but Y has %lld", (long long)R, (long long)own);
    R = own;
  }
  const at::Tensor dY = c.output("dY", at::kBFloat16, {R, N});
  at::Tensor dweights;
  if (Y) dweights = c.output("dweights", at::kFloat, {T, k});
  else if (!c.none()) refuse("dweights needs Y");
  c.run([&](void* stream) {
    return f8f8bf16_moe_combine_backward(ptr<uint16_t>(&dout), ptr<int32_t>(&dst), ptr<float>(weights), ptr<uint16_t>(Y),
                                       ptr<uint16_t>(dY), ptr<float>(dweights), T, k, R, N, stream);
  });
  return pack(dY, dweights);
}

PyObject* silu_mul_quantize(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_silu_mul_quantize", args, n, 7);
  const at::Tensor& H = *c.tensor("H");
  c.check(H, "H", at::kBFloat16, 2, "[rows, 2 I]");
  const int64_t rows = H.size(0), two = H.size(1), I = two / 2;
  if (two % 2) refuse("H must have an even number of columns, got %lld", (long long)two);
  const int64_t block = c.integer();
  const int64_t cols = block_cols(block, I);
  const bool checkpoint = c.flag();
  const at::Tensor AQ = c.output("AQ", at::kByte, {rows, I});
  const at::Tensor a_scale = scales(c, "a_scale", rows, cols);
  at::Tensor HQ, h_scale;
  if (checkpoint || !c.none(0) || !c.none(1)) {
    HQ = c.output("HQ", at::kByte, {rows, two});
    h_scale = c.output("h_scale", at::kFloat, {rows, 2, (I + 127) / 128});
  }
  c.run([&](void* stream) {
    return f8f8bf16_silu_mul_quantize(ptr<uint16_t>(&H), (int)block, ptr<uint8_t>(AQ), ptr<float>(a_scale), ptr<uint8_t>(HQ),
                                    ptr<float>(h_scale), rows, I, stream);
  });
  return pack(AQ, a_scale, HQ, h_scale);
}

PyObject* silu_mul_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_silu_mul_backward", args, n, 4);
  const at::Tensor& dA = *c.tensor("dA");
  c.check(dA, "dA", at::kBFloat16, 2, "[rows, I]");
  const int64_t rows = dA.size(0), I = dA.size(1);
  const at::Tensor& HQ = *c.tensor("HQ");
  c.check_codes(HQ, "HQ", {rows, 2 * I});
  const at::Tensor& h_scale = *c.tensor("h_scale");
  c.check(h_scale, "h_scale", at::kFloat, {rows, 2, (I + 127) / 128});
  const at::Tensor dH = c.output("dH", at::kBFloat16, {rows, 2 * I});
  c.run([&](void* stream) {
    return f8f8bf16_silu_mul_backward(ptr<uint16_t>(&dA), ptr<uint8_t>(&HQ), ptr<float>(&h_scale), ptr<uint16_t>(dH), rows,
                                    I, stream);
  });
  return wrap(dH);
}

PyObject* quantize_k_offsets(PyObject* const* args, Py_ssize_t n) {
  Call c("f8f8bf16_quantize_k_offsets", args, n, 7);
  const at::Tensor& X = *c.tensor("X");
  if (X.dim() != 2) refuse("X must be [R, K]");
  const int64_t R = X.size(0), K = X.size(1);
  const at::Tensor& M_sizes = *c.tensor("M_sizes");
  if (M_sizes.dim() != 1) refuse("M_sizes must be [G]");
  const int64_t G = M_sizes.size(0);
  const at::Tensor* xs = c.tensor("x_scale", true);
  int64_t cols = 0;
  if (xs) {
    c.check_codes(X, "X", {R, K});
    cols = xs->dim() == 1 ? 1 : K / 128;
    if (xs->dim() == 1) c.check(*xs, "x_scale", at::kFloat, {R});
    else c.check(*xs, "x_scale", at::kFloat, {R, cols});
  } else {
    c.check(X, "X", at::kBFloat16, {R, K});
  }
  c.check(M_sizes, "M_sizes", at::kLong, {G});
  const at::Tensor XT = c.output("XT", at::kByte, {K, f8f8bf16_k_offsets_capacity(R, G)});
  const at::Tensor t_scale = c.output("t_scale", at::kFloat, {G, K});
  const at::Tensor k_offsets = c.output("k_offsets", at::kInt, {G});
  const at::Tensor ws = c.workspace(f8f8bf16_quantize_k_offsets_workspace(R, G, K));
  c.run([&](void* stream) {
    return f8f8bf16_quantize_k_offsets(X.data_ptr(), xs ? FP8GG_DTYPE_E4M3 : FP8GG_DTYPE_BF16, ptr<float>(xs), cols,
                                     ptr<int64_t>(&M_sizes), ptr<uint8_t>(XT), ptr<float>(t_scale), ptr<int32_t>(k_offsets),
                                     ptr<void>(ws), ws.defined() ? (int64_t)ws.nbytes() : 0, R, G, K, stream);
  });
  return pack(XT, t_scale, k_offsets);
}

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<rmsnorm_quantize>("rmsnorm_quantize"),
    method<rmsnorm_backward>("rmsnorm_backward"),
    method<route>("route"),
    method<route_backward>("route_backward"),
    method<moe_dispatch>("moe_dispatch"),
    method<moe_combine>("moe_combine"),
    method<moe_combine_backward>("moe_combine_backward"),
    method<silu_mul_quantize>("silu_mul_quantize"),
    method<silu_mul_backward>("silu_mul_backward"),
    method<quantize_k_offsets>("quantize_k_offsets"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding() { return PyModule_Create(&module); }
