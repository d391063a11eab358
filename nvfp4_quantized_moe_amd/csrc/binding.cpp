// The Python calls of the operators around the expert FFN, from their checked
// arguments to the C entry point: tensor checks, output allocations and the
// launch. A call's smallest kernels run for 3 to 6 us; marshalled in Python it
// took 8.3 us for the gate of 64 tokens (13 for the norms, whose ten tensors
// are each looked at), here 4.8.
//
// Tensors in, pointers and the current stream out, as the rest of the binding:
// every input a contiguous tensor of the current device, shapes checked, given
// outputs checked for their size, everything else left to the library's own
// checks. Refused tensors raise ValueError, a nonzero status NVFP4Error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <climits>
#include <initializer_list>
#include <optional>
#include <string>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "nvfp4moe.h"

namespace {

PyObject* g_get_device;  // () -> index of the current device
PyObject* g_get_stream;  // (index) -> address of its current stream
PyObject* g_error;       // NVFP4Error(status, name of the call)

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte, kI8 = at::kChar;

[[noreturn]] void refuse(const char* name, const std::string& why) {
  PyErr_Format(PyExc_ValueError, "%s: %s", name, why.c_str());
  throw python_error();
}
std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + ")";
}

long long py_long(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int32_t to_i32(long long v, const char* name) {
  if (v < INT_MIN || v > INT_MAX) refuse(name, std::to_string(v) + " does not fit 32 bits");
  return (int32_t)v;
}
int32_t py_i32(PyObject* o, const char* name) { return to_i32(py_long(o), name); }
float py_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}

const at::Tensor* given(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw python_error();
  }
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = given(o, name);
  if (!t) refuse(name, "expected a tensor, got None");
  return *t;
}

// One call: the device it runs on, and its launch.
class Call {
 public:
  explicit Call(const char* name) : name_(name) {}

  int device() {
    if (device_ < 0) {
      PyObject* d = PyObject_CallNoArgs(g_get_device);
      if (!d) throw python_error();
      device_ = (int)PyLong_AsLong(d);
      Py_DECREF(d);
    }
    return device_;
  }

  // t is a contiguous tensor of this type on the current device
  const at::Tensor& here(const at::Tensor& t, at::ScalarType type, const char* name) {
    if (!t.is_cuda() || t.scalar_type() != type || !t.is_contiguous())
      refuse(name, std::string("expected a contiguous CUDA ") + c10::toString(type) + " tensor, got " +
                       c10::toString(t.scalar_type()) + " on " + t.device().str());
    if (t.get_device() != device())
      refuse(name, "on " + t.device().str() + ", but the current device is cuda:" + std::to_string(device()));
    return t;
  }
  // the same, BF16 or float32
  const at::Tensor& floats(const at::Tensor& t, const char* name) {
    const at::ScalarType type = t.scalar_type();
    if (type != kBf16 && type != kF32)
      refuse(name, std::string("expected BF16 or float32, got ") + c10::toString(type));
    return here(t, type, name);
  }
  void shaped(const at::Tensor& t, std::initializer_list<int64_t> shape, const char* name) {
    if (t.sizes() != at::IntArrayRef(shape))
      refuse(name, "expected shape " + text(shape) + ", got " + text(t.sizes()));
  }
  // an optional input of exactly this type and shape; its address
  template <typename P>
  P* input(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, const char* name) {
    const at::Tensor* t = given(o, name);
    if (!t) return nullptr;
    here(*t, type, name);
    shaped(*t, shape, name);
    return static_cast<P*>(t->data_ptr());
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)device())));
  }

  template <typename Launch>
  void run(Launch launch) {
    PyObject* index = PyLong_FromLong(device());
    PyObject* address = index ? PyObject_CallOneArg(g_get_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!address) throw python_error();
    void* stream = PyLong_AsVoidPtr(address);
    Py_DECREF(address);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = launch(stream);
    Py_END_ALLOW_THREADS
    if (status == NVFP4_OK) return;
    PyObject* error = PyObject_CallFunction(g_error, "is", status, name_);
    if (error) {
      PyErr_SetObject(g_error, error);
      Py_DECREF(error);
    }
    throw python_error();
  }

 private:
  const char* name_;
  int device_ = -1;
};

// An output: the caller's tensor, of this type and large enough, or a new one.
class Out {
 public:
  Out(Call& call, PyObject* o, at::IntArrayRef shape, at::ScalarType type, const char* name) {
    const at::Tensor* t = given(o, name);
    if (!t) {
      fresh_ = call.make(shape, type);
      at_ = fresh_.data_ptr();
      return;
    }
    call.here(*t, type, name);
    const int64_t n = c10::multiply_integers(shape);
    if (t->numel() < n)
      refuse(name, "needs at least " + std::to_string(n) + " elements, got " + std::to_string(t->numel()));
    given_ = o;
    at_ = t->data_ptr();
    bytes_ = (size_t)t->numel() * t->element_size();
  }
  template <typename P>
  P* at() const {
    return static_cast<P*>(at_);
  }
  size_t bytes() const { return given_ ? bytes_ : fresh_.nbytes(); }
  PyObject* take() const {  // a new reference
    if (!given_) return THPVariable_Wrap(fresh_);
    Py_INCREF(given_);
    return given_;
  }

 private:
  at::Tensor fresh_;
  PyObject* given_ = nullptr;
  void* at_ = nullptr;
  size_t bytes_ = 0;
};
// A workspace: of at least `need` bytes when new; a given one is checked by the library.
Out workspace(Call& call, PyObject* o, size_t need) {
  return o == Py_None ? Out(call, o, {(int64_t)std::max<size_t>(need, 256)}, kU8, "ws")
                      : Out(call, o, {0}, kU8, "ws");
}

struct Matrix {
  int64_t rows, cols;
};
Matrix matrix(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(name, "expected 2 dimensions, got shape " + text(t.sizes()));
  to_i32(t.size(0), name);
  to_i32(t.size(1), name);
  return {t.size(0), t.size(1)};
}
int32_t code(const at::Tensor& t) { return t.scalar_type() == kBf16 ? NVFP4_DT_BF16 : NVFP4_DT_F32; }

PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
  return r;
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// Sequences of cu_seqlens int32 [B + 1] (None: one).
struct Seqs {
  const int32_t* cu;
  int32_t B;
};
Seqs sequences(Call& call, PyObject* o) {
  const at::Tensor* t = given(o, "cu_seqlens");
  if (!t) return {nullptr, 1};
  call.here(*t, kI32, "cu_seqlens");
  if (t->dim() != 1 || t->numel() < 2)
    refuse("cu_seqlens", "expected [B + 1] with B >= 1, got shape " + text(t->sizes()));
  return {static_cast<const int32_t*>(t->data_ptr()), to_i32(t->numel() - 1, "cu_seqlens")};
}

PyObject* gate_topk(PyObject* const* a) {
  Call call("moe_gate_topk");
  const at::Tensor& logits = call.floats(needed(a[0], "logits"), "logits");
  const auto [T, E] = matrix(logits, "logits");
  const int32_t k = py_i32(a[1], "k"), score = py_i32(a[2], "score");
  const float* bias = call.input<float>(a[3], kF32, {E}, "bias");
  const uint8_t* mask = call.input<uint8_t>(a[4], kU8, {T}, "token_mask");
  const int32_t n_group = py_i32(a[5], "n_group"), topk_group = py_i32(a[6], "topk_group");
  const int32_t renormalize = py_i32(a[7], "renormalize");
  const float scale = py_float(a[8]);
  const int64_t cols = std::max(k, 0);  // a negative k is the library's to refuse
  const Out ids(call, a[9], {T, cols}, kI32, "topk_ids"), w(call, a[10], {T, cols}, kF32, "topk_w");
  call.run([&, T = (int32_t)T, E = (int32_t)E](void* stream) {
    return moe_gate_topk(logits.data_ptr(), code(logits), bias, mask, T, E, k, score, n_group, topk_group, renormalize,
                         scale, ids.at<int32_t>(), w.at<float>(), stream);
  });
  return tuple({ids.take(), w.take()});
}

PyObject* balance_loss(PyObject* const* a) {
  Call call("moe_balance_loss");
  const at::Tensor& logits = call.floats(needed(a[0], "logits"), "logits");
  const auto [T, E] = matrix(logits, "logits");
  const at::Tensor& ids = call.here(needed(a[1], "topk_ids"), kI32, "topk_ids");
  const int64_t k = matrix(ids, "topk_ids").cols;
  call.shaped(ids, {T, k}, "topk_ids");
  const int32_t score = py_i32(a[2], "score");
  const uint8_t* mask = call.input<uint8_t>(a[3], kU8, {T}, "token_mask");
  const Seqs seq = sequences(call, a[4]);
  const Out loss(call, a[5], {2}, kF32, "loss"), counts(call, a[6], {seq.B, E}, kI32, "counts");
  const Out tokens(call, a[7], {(int64_t)seq.B + 2}, kI32, "tokens");
  const Out ws = workspace(call, a[8], moe_balance_loss_ws_bytes((int32_t)T, (int32_t)E, seq.B));
  call.run([&, T = (int32_t)T, E = (int32_t)E](void* stream) {
    return moe_balance_loss(logits.data_ptr(), code(logits), static_cast<const int32_t*>(ids.data_ptr()), mask, seq.cu,
                            seq.B, T, E, (int32_t)k, score, loss.at<float>(), counts.at<int32_t>(),
                            tokens.at<int32_t>(), ws.at<void>(), ws.bytes(), stream);
  });
  return tuple({loss.take(), counts.take(), tokens.take()});
}

PyObject* gate_backward(PyObject* const* a) {
  Call call("moe_gate_backward");
  const at::Tensor& logits = call.floats(needed(a[0], "logits"), "logits");
  const auto [T, E] = matrix(logits, "logits");
  const at::Tensor& ids = call.here(needed(a[1], "topk_ids"), kI32, "topk_ids");
  const int64_t k = matrix(ids, "topk_ids").cols;
  call.shaped(ids, {T, k}, "topk_ids");
  const int32_t score = py_i32(a[2], "score"), renormalize = py_i32(a[3], "renormalize");
  const float scale = py_float(a[4]);
  const uint8_t* mask = call.input<uint8_t>(a[5], kU8, {T}, "token_mask");
  const float* d_w = call.input<float>(a[6], kF32, {T, k}, "d_topk_w");
  const float* d_loss = call.input<float>(a[7], kF32, {2}, "d_loss");
  Seqs seq = {nullptr, 1};
  const int32_t *counts = nullptr, *tokens = nullptr;
  if (d_loss) {
    seq = sequences(call, a[10]);
    if (a[8] == Py_None || a[9] == Py_None) refuse("d_loss", "needs counts and tokens of moe_balance_loss");
    counts = Out(call, a[8], {seq.B, E}, kI32, "counts").at<int32_t>();
    tokens = Out(call, a[9], {(int64_t)seq.B + 2}, kI32, "tokens").at<int32_t>();
  }
  const Out d_logits(call, a[11], {T, E}, logits.scalar_type(), "d_logits");
  call.run([&, T = (int32_t)T, E = (int32_t)E](void* stream) {
    return moe_gate_backward(logits.data_ptr(), code(logits), static_cast<const int32_t*>(ids.data_ptr()), mask, T, E,
                             (int32_t)k, score, renormalize, scale, d_w, d_loss, counts, tokens, seq.cu, seq.B,
                             d_logits.at<void>(), stream);
  });
  return d_logits.take();
}

// A gate float32 [H] (channels) or [T, 1] (tokens), and its MOE_GATE_*.
struct Gate {
  const float* at;
  int32_t mode;
};
Gate gate_of(Call& call, PyObject* o, int64_t T, int64_t H) {
  const at::Tensor* t = given(o, "gate");
  if (!t) return {nullptr, MOE_GATE_NONE};
  const float* p = static_cast<const float*>(call.here(*t, kF32, "gate").data_ptr());
  if (t->sizes() == at::IntArrayRef({H})) return {p, MOE_GATE_CHANNEL};
  if (t->sizes() == at::IntArrayRef({T, 1})) return {p, MOE_GATE_TOKEN};
  refuse("gate", "expected shape " + text({H}) + " or " + text({T, 1}) + ", got " + text(t->sizes()));
}

PyObject* block_norm(PyObject* const* a) {
  Call call("moe_block_norm");
  const at::Tensor& x = call.floats(needed(a[0], "x"), "x");
  const auto [T, H] = matrix(x, "x");
  at::ScalarType res_type = x.scalar_type();
  const at::Tensor* residual = given(a[1], "residual");
  if (residual) {
    call.floats(*residual, "residual");
    call.shaped(*residual, {T, H}, "residual");
    res_type = residual->scalar_type();
  } else if (const at::Tensor* out = given(a[8], "residual_out")) {
    res_type = call.floats(*out, "residual_out").scalar_type();
  }
  const float* w_pre = call.input<float>(a[2], kF32, {H}, "w_pre");
  const float* w_post = call.input<float>(a[3], kF32, {H}, "w_post");
  const Gate gate = gate_of(call, a[4], T, H);
  const float scale = py_float(a[5]), eps = py_float(a[6]);
  const float* gs = call.input<float>(a[7], kF32, {1}, "gs");
  const Out residual_out(call, a[8], {T, H}, res_type, "residual_out");
  std::optional<Out> y, y_q, y_sf;
  if (w_pre) y.emplace(call, a[9], at::IntArrayRef({T, H}), x.scalar_type(), "y");
  if (gs) {
    y_q.emplace(call, a[10], at::IntArrayRef({T, H / 2}), kU8, "y_q");
    y_sf.emplace(call, a[11], at::IntArrayRef({T, H / 16}), kU8, "y_sf");
  }
  call.run([&, T = (int32_t)T, H = (int32_t)H](void* stream) {
    return moe_block_norm(x.data_ptr(), code(x), residual ? residual->data_ptr() : nullptr,
                          res_type == kBf16 ? NVFP4_DT_BF16 : NVFP4_DT_F32, T, H, w_pre, w_post, gate.at, gate.mode,
                          scale, eps, residual_out.at<void>(), y ? y->at<void>() : nullptr, gs,
                          gs ? y_q->at<uint8_t>() : nullptr, gs ? y_sf->at<uint8_t>() : nullptr, stream);
  });
  PyObject* second = y ? y->take() : none();
  if (!gs) return tuple({residual_out.take(), second});
  return tuple({residual_out.take(), second, y_q->take(), y_sf->take()});
}

PyObject* block_norm_backward(PyObject* const* a) {
  Call call("moe_block_norm_backward");
  const at::Tensor& x = call.floats(needed(a[2], "x"), "x");
  const auto [T, H] = matrix(x, "x");
  const at::Tensor& residual_out = call.floats(needed(a[3], "residual_out"), "residual_out");
  call.shaped(residual_out, {T, H}, "residual_out");
  const at::ScalarType res_type = residual_out.scalar_type();
  const void* d_y = call.input<void>(a[0], x.scalar_type(), {T, H}, "d_y");
  const void* d_res_out = call.input<void>(a[1], res_type, {T, H}, "d_residual_out");
  const float* w_pre = call.input<float>(a[4], kF32, {H}, "w_pre");
  const float* w_post = call.input<float>(a[5], kF32, {H}, "w_post");
  const Gate gate = gate_of(call, a[6], T, H);
  const float scale = py_float(a[7]), eps = py_float(a[8]);
  const Out d_x(call, a[9], {T, H}, x.scalar_type(), "d_x");
  const Out d_residual(call, a[10], {T, H}, res_type, "d_residual");
  std::optional<Out> d_w_pre, d_w_post, d_gate;
  if (w_pre) d_w_pre.emplace(call, a[11], at::IntArrayRef({H}), kF32, "d_w_pre");
  if (w_post) d_w_post.emplace(call, a[12], at::IntArrayRef({H}), kF32, "d_w_post");
  if (gate.mode == MOE_GATE_CHANNEL) d_gate.emplace(call, a[13], at::IntArrayRef({H}), kF32, "d_gate");
  if (gate.mode == MOE_GATE_TOKEN) d_gate.emplace(call, a[13], at::IntArrayRef({T, 1}), kF32, "d_gate");
  const Out ws = workspace(call, a[14], moe_block_norm_backward_ws_bytes((int32_t)T, (int32_t)H));
  call.run([&, T = (int32_t)T, H = (int32_t)H](void* stream) {
    return moe_block_norm_backward(d_y, d_res_out, x.data_ptr(), code(x), residual_out.data_ptr(), code(residual_out),
                                   T, H, w_pre, w_post, gate.at, gate.mode, scale, eps, d_x.at<void>(),
                                   d_residual.at<void>(), d_w_pre ? d_w_pre->at<float>() : nullptr,
                                   d_w_post ? d_w_post->at<float>() : nullptr, d_gate ? d_gate->at<float>() : nullptr,
                                   ws.at<void>(), ws.bytes(), stream);
  });
  const auto grad = [](const std::optional<Out>& o) { return o ? o->take() : none(); };
  return tuple({d_x.take(), d_residual.take(), grad(d_w_pre), grad(d_w_post), grad(d_gate)});
}

PyObject* quantize_rows(PyObject* const* a) {
  Call call("int8_quantize_rows");
  const at::Tensor& x = call.floats(needed(a[0], "x"), "x");
  const auto [M, K] = matrix(x, "x");
  const Out q(call, a[1], {M, K}, kI8, "q"), scale(call, a[2], {M}, kF32, "scale");
  call.run([&, M = (int32_t)M, K = (int32_t)K](void* stream) {
    return int8_quantize_rows(x.data_ptr(), code(x), M, K, q.at<int8_t>(), scale.at<float>(), stream);
  });
  return tuple({q.take(), scale.take()});
}

PyObject* gemm(PyObject* const* a) {
  Call call("int8_gemm");
  const at::Tensor& a_q = call.here(needed(a[0], "a_q"), kI8, "a_q");
  const at::Tensor& b_q = call.here(needed(a[2], "b_q"), kI8, "b_q");
  const auto [M, K] = matrix(a_q, "a_q");
  const int64_t N = matrix(b_q, "b_q").rows;
  call.shaped(b_q, {N, K}, "b_q");
  needed(a[1], "a_scale");
  needed(a[3], "b_scale");
  const float* a_scale = call.input<float>(a[1], kF32, {M}, "a_scale");
  const float* b_scale = call.input<float>(a[3], kF32, {N}, "b_scale");
  const int32_t epilogue = py_i32(a[4], "epilogue");
  const int64_t n_out = epilogue == NVFP4_EPI_SILU_MUL ? N / 2 : N;
  const void* add = call.input<void>(a[5], kBf16, {M, n_out}, "add");
  const Out d(call, a[6], {M, n_out}, kBf16, "d");
  std::optional<Out> ws;
  const size_t need = a[7] == Py_None ? int8_gemm_ws_bytes((int32_t)M, (int32_t)N, (int32_t)K) : 1;
  if (need) ws = workspace(call, a[7], need);
  call.run([&, M = (int32_t)M, N = (int32_t)N, K = (int32_t)K](void* stream) {
    return int8_gemm(static_cast<const int8_t*>(a_q.data_ptr()), a_scale, static_cast<const int8_t*>(b_q.data_ptr()),
                     b_scale, M, N, K, epilogue, add, d.at<void>(), ws ? ws->at<void>() : nullptr,
                     ws ? ws->bytes() : 0, stream);
  });
  return d.take();
}

PyObject* ffn(PyObject* const* a) {  // weights (whose attributes may have been set since they were made), x, add, out, ws
  Call call("int8_ffn_forward");
  const at::Tensor& w1 = call.here(needed(a[0], "weights.w1_q"), kI8, "weights.w1_q");
  const at::Tensor& w2 = call.here(needed(a[2], "weights.w2_q"), kI8, "weights.w2_q");
  const auto [H, I] = matrix(w2, "weights.w2_q");
  call.shaped(w1, {2 * I, H}, "weights.w1_q");
  needed(a[1], "weights.w1_scale");
  needed(a[3], "weights.w2_scale");
  const float* w1_scale = call.input<float>(a[1], kF32, {2 * I}, "weights.w1_scale");
  const float* w2_scale = call.input<float>(a[3], kF32, {H}, "weights.w2_scale");
  const at::Tensor& x = call.here(needed(a[4], "x"), kBf16, "x");
  const int64_t T = matrix(x, "x").rows;
  call.shaped(x, {T, H}, "x");
  const void* add = call.input<void>(a[5], kBf16, {T, H}, "add");
  const Out out(call, a[6], {T, H}, kBf16, "out");
  const Out ws = workspace(call, a[7], int8_ffn_ws_bytes((int32_t)T, (int32_t)H, (int32_t)I));
  call.run([&, T = (int32_t)T, H = (int32_t)H, I = (int32_t)I](void* stream) {
    return int8_ffn_forward(static_cast<const int8_t*>(w1.data_ptr()), w1_scale,
                            static_cast<const int8_t*>(w2.data_ptr()), w2_scale, x.data_ptr(), T, H, I, add,
                            out.at<void>(), ws.at<void>(), ws.bytes(), stream);
  });
  return out.take();
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  return F(args);
  END_HANDLE_TH_ERRORS
}
// (get_device, get_stream, error): what the package looks the device up with, and its exception
PyObject* set_up(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "expected 3 arguments");
    return nullptr;
  }
  PyObject** const to[3] = {&g_get_device, &g_get_stream, &g_error};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(args[i]);
    Py_XDECREF(*to[i]);
    *to[i] = args[i];
  }
  return none();
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {
    method<set_up>("set_up"),
    method<entry<gate_topk, 11>>("gate_topk"),
    method<entry<balance_loss, 9>>("balance_loss"),
    method<entry<gate_backward, 12>>("gate_backward"),
    method<entry<block_norm, 12>>("block_norm"),
    method<entry<block_norm_backward, 15>>("block_norm_backward"),
    method<entry<quantize_rows, 3>>("quantize_rows"),
    method<entry<gemm, 8>>("gemm"),
    method<entry<ffn, 8>>("ffn"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
