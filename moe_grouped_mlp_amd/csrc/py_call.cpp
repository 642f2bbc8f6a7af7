// Python's way into the calls of api_step.cpp (module moe_grouped_mlp_amd._call).
//
// A decoding step's calls are as long as their marshalling: through ctypes, with
// the checks in Python, moe_quantize_fp8 of 16 rows takes the host 6.6 us, of
// which the launch is 2.5.  Here the checks read the tensors' fields directly.
// They see to what the C ABI cannot: that a tensor is contiguous device memory
// of the type and at least the size that the call reads or writes, on the device
// the call runs on.  Arguments come by position from the functions of
// binding.py, which have the names, defaults and documentation.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <limits>
#include <string>
#include <vector>

#include "../../include/moe_gmlp.h"

namespace {

using Size = __int128;   // holds any product of three 32-bit sizes

PyObject* g_check = nullptr;        // binding._check(name, status): raises
PyObject* g_raw_stream = nullptr;   // device -> the current stream's handle

struct Raised {};   // a Python exception is set

enum : unsigned { kF32 = 1, kBF16 = 2, kF64 = 4, kI32 = 8, kU8 = 16, kE4M3 = 32, kBool = 64, kI8 = 128,
                  kCodes = kU8 | kE4M3, kMask = kU8 | kBool };

struct TypeName {
  unsigned bit;
  at::ScalarType type;
  const char* name;
};
constexpr TypeName kTypes[] = {
    {kF32, at::kFloat, "torch.float32"},   {kBF16, at::kBFloat16, "torch.bfloat16"},
    {kF64, at::kDouble, "torch.float64"},  {kI32, at::kInt, "torch.int32"},
    {kU8, at::kByte, "torch.uint8"},       {kE4M3, at::kFloat8_e4m3fn, "torch.float8_e4m3fn"},
    {kBool, at::kBool, "torch.bool"},      {kI8, at::kChar, "torch.int8"}};

unsigned type_bit(at::ScalarType t) {
  for (const TypeName& n : kTypes)
    if (n.type == t) return n.bit;
  return 0;
}

Size blocks(Size n) { return (n + MOE_FP8_BLOCK - 1) / MOE_FP8_BLOCK; }

// One call's arguments, taken in order; the first is the device.
class Args {
 public:
  Args(const char* fn, PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : fn_(fn), a_(a) {
    if (n != want) fail(PyExc_TypeError, std::string(fn) + ": " + std::to_string(want) + " arguments are needed");
    dev_ = i32();
  }
  [[noreturn]] static void fail(PyObject* type, const std::string& text) {
    PyErr_SetString(type, text.c_str());
    throw Raised{};
  }
  [[noreturn]] void refuse(const std::string& text) const { fail(PyExc_ValueError, fn_ + (": " + text)); }

  PyObject* next() { return a_[at_++]; }
  PyObject* peek() const { return a_[at_]; }
  int64_t i64() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  int32_t i32() {
    const int64_t v = i64();
    if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
      fail(PyExc_OverflowError, fn_ + (": " + std::to_string(v) + " does not fit in 32 bits"));
    return static_cast<int32_t>(v);
  }
  double f64() { return number(next()); }
  float f32() { return static_cast<float>(f64()); }
  uint32_t u32() {
    const int64_t v = i64();
    if (v < 0 || v > std::numeric_limits<uint32_t>::max())
      fail(PyExc_OverflowError, fn_ + (": " + std::to_string(v) + " does not fit in 32 bits without a sign"));
    return static_cast<uint32_t>(v);
  }
  bool truth() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) throw Raised{};
    return v != 0;
  }
  // The next argument's memory: null for None, else a tensor of one of the
  // types with n elements at least.
  template <typename T = void>
  T* buf(const char* name, unsigned types, Size n, size_t* bytes = nullptr) {
    PyObject* o = next();
    if (bytes) *bytes = 0;
    if (o == Py_None) return nullptr;
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if ((type_bit(t.scalar_type()) & types) && t.numel() >= n && here(t)) {
        if (bytes) *bytes = t.nbytes();
        return static_cast<T*>(t.data_ptr());
      }
    }
    std::string of;
    for (const TypeName& k : kTypes)
      if (k.bit & types) of += (of.empty() ? "" : " or ") + std::string(k.name);
    refuse(std::string(name) + " must be a contiguous tensor of type " + of + " with at least " +
           std::to_string(static_cast<long long>(n)) + " elements on the current device (cuda:" +
           std::to_string(dev_) + ")");
  }
  // A list of gradients and (out not None) of where to put them.
  std::vector<moe_tensor> list(PyObject* tensors, PyObject* out) {
    std::vector<moe_tensor> v;
    each(tensors, [&](size_t i, const at::Tensor& t) {
      const unsigned type = type_bit(t.scalar_type());
      if (!(type & (kF32 | kBF16))) refuse("tensor " + std::to_string(i) + " must be bfloat16 or float32");
      at_home(t);
      v.push_back({t.data_ptr(), nullptr, t.numel(), type == kF32 ? MOE_TYPE_F32 : MOE_TYPE_BF16});
    });
    if (out == Py_None) return v;
    size_t n = 0;
    const char* other = "out must have a tensor of each one's type and size";
    each(out, [&](size_t i, const at::Tensor& t) {
      if (i >= v.size() || t.numel() != v[i].numel || type_bit(t.scalar_type()) != (v[i].type == MOE_TYPE_F32 ? kF32 : kBF16))
        refuse(other);
      at_home(t);
      v[i].out = t.data_ptr();
      ++n;
    });
    if (n != v.size()) refuse(other);
    return v;
  }
  // A list that goes with params (n tensors): f(i, tensor), for None entries too
  // (null) where they may be.
  template <typename F>
  void along(PyObject* seq, const char* name, size_t n, bool none, F&& f) {
    size_t got = 0;
    each(
        seq,
        [&](size_t i, const at::Tensor* t) {
          if (i >= n) refuse(std::string(name) + " must have an entry for each of params");
          if (t) at_home(*t);
          f(i, t);
          ++got;
        },
        none);
    if (got != n) refuse(std::string(name) + " must have an entry for each of params");
  }
  // moe_adamw's lists.
  std::vector<moe_adamw_tensor> adamw_list(int32_t* state_type) {
    std::vector<moe_adamw_tensor> v;
    PyObject *params = next(), *grads = next(), *m = next(), *vv = next(), *master = next(), *m_scale = next(), *v_scale = next(),
             *decay = next();
    each(params, [&](size_t i, const at::Tensor& t) {
      const unsigned type = type_bit(t.scalar_type());
      if (!(type & (kF32 | kBF16))) refuse("params[" + std::to_string(i) + "] must be bfloat16 or float32");
      at_home(t);
      moe_adamw_tensor a{};
      a.param = t.data_ptr();
      a.numel = t.numel();
      a.param_type = type == kF32 ? MOE_TYPE_F32 : MOE_TYPE_BF16;
      v.push_back(a);
    });
    const size_t n = v.size();
    auto of = [&](const char* name, size_t i, const at::Tensor& t, unsigned types, int64_t numel) {
      if (!(type_bit(t.scalar_type()) & types) || t.numel() != numel)
        refuse(std::string(name) + "[" + std::to_string(i) + "] is of another type or size than params[" + std::to_string(i) + "] takes");
    };
    along(grads, "grads", n, false, [&](size_t i, const at::Tensor* t) {
      of("grads", i, *t, kF32 | kBF16, v[i].numel);
      v[i].grad = t->data_ptr();
      v[i].grad_type = type_bit(t->scalar_type()) == kF32 ? MOE_TYPE_F32 : MOE_TYPE_BF16;
    });
    // the states' type is that of the scales being there
    const bool fp8 = m_scale != Py_None;
    if (fp8 != (v_scale != Py_None)) refuse("m_scale and v_scale go together");
    *state_type = fp8 ? MOE_STATE_FP8 : MOE_STATE_F32;
    const unsigned state = fp8 ? kCodes : kF32;
    along(m, "m", n, false, [&](size_t i, const at::Tensor* t) {
      of("m", i, *t, state, v[i].numel);
      v[i].m = t->data_ptr();
    });
    along(vv, "v", n, false, [&](size_t i, const at::Tensor* t) {
      of("v", i, *t, state, v[i].numel);
      v[i].v = t->data_ptr();
    });
    if (master != Py_None)
      along(master, "master", n, true, [&](size_t i, const at::Tensor* t) {
        if (!t) return;
        of("master", i, *t, kF32, v[i].numel);
        if (v[i].param_type != MOE_TYPE_BF16) refuse("master[" + std::to_string(i) + "] is of a parameter that is float32 itself");
        v[i].master = static_cast<float*>(t->data_ptr());
      });
    if (fp8) {
      along(m_scale, "m_scale", n, false, [&](size_t i, const at::Tensor* t) {
        of("m_scale", i, *t, kF32, static_cast<int64_t>(blocks(v[i].numel)));
        v[i].m_scale = static_cast<float*>(t->data_ptr());
      });
      along(v_scale, "v_scale", n, false, [&](size_t i, const at::Tensor* t) {
        of("v_scale", i, *t, kF32, static_cast<int64_t>(blocks(v[i].numel)));
        v[i].v_scale = static_cast<float*>(t->data_ptr());
      });
    }
    if (PyNumber_Check(decay) && !PySequence_Check(decay)) {
      const float d = static_cast<float>(number(decay));
      for (moe_adamw_tensor& t : v) t.weight_decay = d;
    } else {
      PyObject* fast = PySequence_Fast(decay, "weight_decay must be a number or a list of them");
      if (!fast) throw Raised{};
      const Drop drop{fast};
      if (PySequence_Fast_GET_SIZE(fast) != static_cast<Py_ssize_t>(n)) refuse("weight_decay must have an entry for each of params");
      for (size_t i = 0; i < n; ++i) v[i].weight_decay = static_cast<float>(number(PySequence_Fast_GET_ITEM(fast, static_cast<Py_ssize_t>(i))));
    }
    return v;
  }
  void* stream() {
    PyObject* s = next();
    if (PyLong_Check(s)) return pointer(s);
    if (s != Py_None) {   // a Stream object: of the current device
      PyObject* d = PyObject_GetAttrString(s, "device_index");
      if (!d) throw Raised{};
      const long on = PyLong_AsLong(d);
      Py_DECREF(d);
      if (on == -1 && PyErr_Occurred()) throw Raised{};
      if (on != dev_) refuse("the stream is of another device (cuda:" + std::to_string(on) + ")");
    }
    PyObject* h = s == Py_None ? PyObject_CallOneArg(g_raw_stream, a_[0]) : PyObject_GetAttrString(s, "cuda_stream");
    if (!h) throw Raised{};
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
  }

 private:
  // (a view with a pending negation, say x.imag of a conjugate, is no plain memory)
  bool here(const at::Tensor& t) const { return t.get_device() == dev_ && t.is_contiguous() && !t.is_neg(); }
  void at_home(const at::Tensor& t) const {
    if (!here(t))
      refuse("the tensors must be contiguous and on the current device (cuda:" + std::to_string(dev_) + ")");
  }
  struct Drop {
    PyObject* o;
    ~Drop() { Py_DECREF(o); }
  };
  static double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  // f(i, tensor) for a list of tensors; none: f(i, pointer), null for None.
  template <typename F>
  void each(PyObject* seq, F&& f) {
    each(seq, [&](size_t i, const at::Tensor* t) { f(i, *t); }, false);
  }
  template <typename F>
  void each(PyObject* seq, F&& f, bool none) {
    PyObject* fast = PySequence_Fast(seq, "");
    if (!fast) {
      PyErr_Clear();
      refuse("a list of tensors is needed");
    }
    const Drop drop{fast};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(fast, i);
      const bool is = THPVariable_Check(o);
      if (!is && !(none && o == Py_None)) refuse("a list of tensors is needed");
      f(static_cast<size_t>(i), is ? &THPVariable_Unpack(o) : nullptr);
    }
  }
  static void* pointer(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
  }
  const char* fn_;
  PyObject* const* a_;
  int at_ = 0;
  int dev_ = 0;

 public:
  const char* name() const { return fn_; }
};

// The call itself, without the interpreter's lock; a status is raised.
template <typename A>
PyObject* call(Args& p, moe_status (*f)(const A*, void*), const A& a) {
  void* s = p.stream();
  moe_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f(&a, s);
  Py_END_ALLOW_THREADS
  if (st == MOE_OK) Py_RETURN_NONE;
  return PyObject_CallFunction(g_check, "si", p.name(), static_cast<int>(st));
}

// No C++ exception leaves a function of the module.
template <typename F>
PyObject* guarded(const char* fn, F&& f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::bad_alloc&) {
    PyErr_NoMemory();
  } catch (const std::exception& e) {
    PyErr_Format(PyExc_ValueError, "%s: %s", fn, e.what());
  } catch (...) {
    PyErr_Format(PyExc_RuntimeError, "%s: unknown exception", fn);
  }
  return nullptr;
}

PyObject* quantize_fp8(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_quantize_fp8";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 15);
    moe_quant_fp8_args a{};
    a.mode = p.i32();
    a.batch = p.i32();
    a.rows = p.i32();
    a.cols = p.i32();
    a.x_stride = p.i64();
    const Size B = a.batch, R = a.rows, C = a.cols, n = B * R * C;
    const Size rows = blocks(C) * R, cols = blocks(R) * C, tiles = blocks(R) * blocks(C);
    const Size ns = a.mode == MOE_QUANT_TILE ? tiles : a.mode == MOE_QUANT_COL ? cols : rows;
    a.x = p.buf("x", kBF16, a.x_stride && B ? (B - 1) * a.x_stride + R * C : n);
    a.q = p.buf<uint8_t>("q", kCodes, n);
    a.s = p.buf<float>("s", kF32, B * ns);
    a.qT = p.buf<uint8_t>("qT", kCodes, n);
    a.sT = p.buf<float>("sT", kF32, B * (a.mode == MOE_QUANT_TILE ? tiles : cols));
    a.pow2 = p.truth();
    a.live = p.buf<int32_t>("live", kI32, B);
    a.row_end = p.buf<int32_t>("row_end", kI32, 1);
    return call(p, moe_quantize_fp8, a);
  });
}

PyObject* grouped_gemm_fp8(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_grouped_gemm_fp8";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 22);
    moe_gemm_fp8_args a{};
    a.E = p.i32();
    a.N = p.i32();
    a.K = p.i32();
    a.M_cap = p.i64();
    a.b_stride = p.i64();
    a.b_s_stride = p.i64();
    a.ldc = p.i64();
    a.c_type = p.i32();
    a.max_rows = p.i32();
    a.cu_margin = p.i32();
    a.fp8_sums = p.truth();
    const Size E = a.E, N = a.N, K = a.K, M = a.M_cap, nk = N * K, ns = blocks(N) * blocks(K);
    a.split_sizes = p.buf<int32_t>("split_sizes", kI32, E);
    a.padded_offsets = p.buf<int32_t>("padded_offsets", kI32, E + 1);
    a.a = p.buf<uint8_t>("a", kCodes, M * K);
    a.a_s = p.buf<float>("a_s", kF32, M * blocks(K));
    a.b = p.buf<uint8_t>("b", kCodes, (E - 1) * (a.b_stride ? a.b_stride : nk) + nk);
    a.b_s = p.buf<float>("b_s", kF32, (E - 1) * (a.b_s_stride ? a.b_s_stride : ns) + ns);
    a.c = p.buf("c", a.c_type == MOE_TYPE_F32 ? kF32 : kBF16, (M - 1) * (a.ldc ? a.ldc : N) + N);
    a.err_flag = p.buf<int32_t>("err_flag", kI32, 1);
    a.workspace = p.buf("workspace", kU8, 0, &a.workspace_bytes);
    return call(p, moe_grouped_gemm_fp8, a);
  });
}

PyObject* grouped_wgrad_fp8(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_grouped_wgrad_fp8";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 18);
    moe_wgrad_fp8_args a{};
    a.E = p.i32();
    a.P = p.i32();
    a.Q = p.i32();
    a.M_cap = p.i64();
    a.c_type = p.i32();
    a.accumulate = p.truth();
    a.cu_margin = p.i32();
    a.fp8_sums = p.truth();
    const Size E = a.E, P = a.P, Q = a.Q, M = a.M_cap;
    a.split_sizes = p.buf<int32_t>("split_sizes", kI32, E);
    a.padded_offsets = p.buf<int32_t>("padded_offsets", kI32, E + 1);
    a.a = p.buf<uint8_t>("a", kCodes, P * M);
    a.a_s = p.buf<float>("a_s", kF32, P * blocks(M));
    a.b = p.buf<uint8_t>("b", kCodes, Q * M);
    a.b_s = p.buf<float>("b_s", kF32, Q * blocks(M));
    a.c = p.buf("c", a.c_type == MOE_TYPE_F32 ? kF32 : kBF16, E * P * Q);
    a.err_flag = p.buf<int32_t>("err_flag", kI32, 1);
    return call(p, moe_grouped_wgrad_fp8, a);
  });
}

PyObject* router_loss(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_router_loss";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 15);
    moe_router_loss_args a{};
    a.T = p.i32();
    a.E = p.i32();
    a.k = p.i32();
    a.balance_coef = p.f32();
    a.z_coef = p.f32();
    const Size T = a.T;
    a.logits = p.buf<float>("logits", kF32, T * a.E);
    a.expert_idx = p.buf<int32_t>("expert_idx", kI32, T * a.k);
    a.token_mask = p.buf<uint8_t>("token_mask", kMask, T);
    a.counts = p.buf<int32_t>("counts", kI32, a.E);
    a.n_tokens = p.buf<int32_t>("n_tokens", kI32, 1);
    a.prob_mean = p.buf<float>("prob_mean", kF32, a.E);
    a.loss = p.buf<float>("loss", kF32, 2);
    a.workspace = p.buf("workspace", kU8, 0, &a.workspace_bytes);
    return call(p, moe_router_loss, a);
  });
}

PyObject* router_bwd(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_router_bwd";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 15);
    moe_router_bwd_args a{};
    a.T = p.i32();
    a.E = p.i32();
    a.k = p.i32();
    a.balance_coef = p.f32();
    a.z_coef = p.f32();
    const Size T = a.T;
    a.logits = p.buf<float>("logits", kF32, T * a.E);
    a.expert_idx = p.buf<int32_t>("expert_idx", kI32, T * a.k);
    a.token_mask = p.buf<uint8_t>("token_mask", kMask, T);
    a.dprobs = p.buf<float>("dprobs", kF32, T * a.k);
    a.dloss = p.buf<float>("dloss", kF32, 2);
    a.counts = p.buf<int32_t>("counts", kI32, a.E);
    a.n_tokens = p.buf<int32_t>("n_tokens", kI32, 1);
    a.dlogits = p.buf<float>("dlogits", kF32, T * a.E);
    return call(p, moe_router_bwd, a);
  });
}

PyObject* grad_sumsq(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_grad_sumsq";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 5);
    moe_grad_args a{};
    const std::vector<moe_tensor> v = p.list(p.next(), Py_None);
    a.tensors = v.data();
    a.n_tensors = static_cast<int32_t>(v.size());
    a.sumsq = p.buf<double>("sumsq", kF64, 1);
    a.workspace = p.buf("workspace", kU8, 0, &a.workspace_bytes);
    return call(p, moe_grad_sumsq, a);
  });
}

PyObject* grad_clip(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_grad_clip";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 8);
    moe_grad_args a{};
    PyObject* tensors = p.next();
    const std::vector<moe_tensor> v = p.list(tensors, p.next());
    a.tensors = v.data();
    a.n_tensors = static_cast<int32_t>(v.size());
    a.max_norm = p.f32();
    a.sumsq = p.buf<double>("sumsq", kF64, 1);
    a.norm = p.buf<float>("norm", kF32, 1);
    a.err_flag = p.buf<int32_t>("err_flag", kI32, 1);
    return call(p, moe_grad_clip, a);
  });
}

// The type of a tensor that may have two.
int32_t type_of(PyObject* o) {
  return THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kBFloat16 ? MOE_TYPE_BF16 : MOE_TYPE_F32;
}

PyObject* router_gate(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_router_gate";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 18);
    moe_gate_args a{};
    a.T = p.i32();
    a.E = p.i32();
    a.k = p.i32();
    a.score = p.i32();
    a.n_groups = p.i32();
    a.topk_groups = p.i32();
    a.group_top = p.i32();
    a.renorm = p.truth();
    a.scale = p.f32();
    a.ld = p.i64();
    const Size T = a.T;
    a.logits_type = type_of(p.peek());
    a.logits = p.buf("logits", kF32 | kBF16, T > 0 ? (T - 1) * (a.ld ? a.ld : a.E) + a.E : 0);
    a.bias = p.buf<float>("bias", kF32, a.E);
    a.token_mask = p.buf<uint8_t>("token_mask", kMask, T);
    a.expert_idx = p.buf<int32_t>("expert_idx", kI32, T * a.k);
    a.probs = p.buf<float>("probs", kF32, T * a.k);
    a.counts = p.buf<int32_t>("counts", kI32, a.E);
    return call(p, moe_router_gate, a);
  });
}

PyObject* router_gate_bwd(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_router_gate_bwd";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 15);
    moe_gate_bwd_args a{};
    a.T = p.i32();
    a.E = p.i32();
    a.k = p.i32();
    a.score = p.i32();
    a.renorm = p.truth();
    a.scale = p.f32();
    a.accumulate = p.truth();
    a.ld = p.i64();
    a.ld_d = p.i64();
    const Size T = a.T;
    a.logits_type = type_of(p.peek());
    a.logits = p.buf("logits", kF32 | kBF16, T > 0 ? (T - 1) * (a.ld ? a.ld : a.E) + a.E : 0);
    a.expert_idx = p.buf<int32_t>("expert_idx", kI32, T * a.k);
    a.dprobs = p.buf<float>("dprobs", kF32, T * a.k);
    a.dlogits = p.buf("dlogits", a.logits_type == MOE_TYPE_F32 ? kF32 : kBF16, T > 0 ? (T - 1) * (a.ld_d ? a.ld_d : a.E) + a.E : 0);
    return call(p, moe_router_gate_bwd, a);
  });
}

PyObject* router_bias_update(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_router_bias_update";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 7);
    moe_bias_update_args a{};
    a.E = p.i32();
    a.rate = p.f32();
    a.reset = p.truth();
    a.counts = p.buf<int32_t>("counts", kI32, a.E);
    a.bias = p.buf<float>("bias", kF32, a.E);
    return call(p, moe_router_bias_update, a);
  });
}

PyObject* adamw(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_adamw";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 22);
    moe_adamw_args a{};
    const std::vector<moe_adamw_tensor> v = p.adamw_list(&a.state_type);
    a.tensors = v.data();
    a.n_tensors = static_cast<int32_t>(v.size());
    a.lr = p.f64();
    a.beta1 = p.f64();
    a.beta2 = p.f64();
    a.eps = p.f64();
    a.step = p.i32();
    a.max_norm = p.f64();
    a.stochastic = p.truth();
    a.seed = p.u32();
    a.sumsq = p.buf<double>("sumsq", kF64, 1);
    a.step_dev = p.buf<int32_t>("step_dev", kI32, 1);
    a.lr_dev = p.buf<float>("lr_dev", kF32, 1);
    a.err_flag = p.buf<int32_t>("err_flag", kI32, 1);
    return call(p, moe_adamw, a);
  });
}

PyObject* quantize_int8(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_quantize_int8";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 9);
    moe_quant_int8_args a{};
    a.rows = p.i32();
    a.cols = p.i32();
    a.x_stride = p.i64();
    const Size R = a.rows, C = a.cols;
    a.x = p.buf("x", kBF16, R > 0 ? (R - 1) * (a.x_stride ? a.x_stride : C) + C : 0);
    a.q = p.buf<int8_t>("q", kI8, R * C);
    a.s = p.buf<float>("s", kF32, R);
    a.row_end = p.buf<int32_t>("row_end", kI32, 1);
    return call(p, moe_quantize_int8, a);
  });
}

PyObject* grouped_gemm_int8(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  constexpr const char* fn = "moe_grouped_gemm_int8";
  return guarded(fn, [&] {
    Args p(fn, args, n_args, 21);
    moe_gemm_int8_args a{};
    a.E = p.i32();
    a.N = p.i32();
    a.K = p.i32();
    a.M_cap = p.i64();
    a.b_stride = p.i64();
    a.b_s_stride = p.i64();
    a.ldc = p.i64();
    a.c_type = p.i32();
    a.max_rows = p.i32();
    a.cu_margin = p.i32();
    const Size E = a.E, N = a.N, K = a.K, M = a.M_cap, nk = N * K;
    a.split_sizes = p.buf<int32_t>("split_sizes", kI32, E);
    a.padded_offsets = p.buf<int32_t>("padded_offsets", kI32, E + 1);
    a.a = p.buf<int8_t>("a", kI8, M * K);
    a.a_s = p.buf<float>("a_s", kF32, M);
    a.b = p.buf<int8_t>("b", kI8, (E - 1) * (a.b_stride ? a.b_stride : nk) + nk);
    a.b_s = p.buf<float>("b_s", kF32, (E - 1) * (a.b_s_stride ? a.b_s_stride : N) + N);
    a.c = p.buf("c", a.c_type == MOE_TYPE_F32 ? kF32 : kBF16, (M - 1) * (a.ldc ? a.ldc : N) + N);
    a.err_flag = p.buf<int32_t>("err_flag", kI32, 1);
    a.workspace = p.buf("workspace", kU8, 0, &a.workspace_bytes);
    return call(p, moe_grouped_gemm_int8, a);
  });
}

PyObject* setup(PyObject*, PyObject* args) {
  PyObject *check, *raw_stream;
  if (!PyArg_ParseTuple(args, "OO", &check, &raw_stream)) return nullptr;
  Py_INCREF(check);
  Py_INCREF(raw_stream);
  Py_XDECREF(g_check);
  Py_XDECREF(g_raw_stream);
  g_check = check;
  g_raw_stream = raw_stream;
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(quantize_fp8), FAST(grouped_gemm_fp8), FAST(grouped_wgrad_fp8), FAST(router_loss),
                          FAST(router_bwd),   FAST(grad_sumsq),       FAST(grad_clip),
                          FAST(router_gate),  FAST(router_gate_bwd),  FAST(router_bias_update), FAST(adamw),
                          FAST(quantize_int8), FAST(grouped_gemm_int8),
                          {"setup", setup, METH_VARARGS, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&kModule); }
