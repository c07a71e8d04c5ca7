// host_ops.cpp - the Python module behind ops.py: checks tensors, allocates outputs and
// workspaces with torch and calls the C entry points of libmoe_ffn.so on the tensors' device
// and its current stream. No arithmetic happens here. The calls are short (a one-row norm is
// 2 us on the GPU), so their host side is what a caller waits for: written in Python over
// ctypes it took 8 to 9 us for the norm or the dropout.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "moe_ffn.h"

namespace {

PyObject* g_error = nullptr;      // the exception class: called with (status, message)

struct Refusal {
  int status;
  std::string message;
};
[[noreturn]] void refuse(const std::string& message) { throw Refusal{MOE_INVALID_ARG, message}; }

PyObject* raise(const Refusal& r) {
  if (!g_error) {
    PyErr_SetString(PyExc_RuntimeError, r.message.c_str());
    return nullptr;
  }
  PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.message.c_str());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}
std::string typed_on(const at::Tensor& x) {
  return std::string(c10::toString(x.scalar_type())) + " tensor on " + x.device().str();
}

// ------------------------------------------------------------------ arguments
const at::Tensor& cuda_tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided)
    refuse(std::string(what) + " must be a CUDA tensor");
  if (t.is_neg()) refuse(std::string(what) + " is a lazily negated view: call resolve_neg()");
  // The C ABI reads a null pointer as an argument that was not given. A wrapper subclass or a
  // fake tensor says it is on the device and has none of its memory.
  if (!t.has_storage() || (t.numel() > 0 && !t.storage().data()))
    refuse(std::string(what) + " has no memory of its own (a wrapper or a fake tensor)");
  return t;
}

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_FP16;
    case at::kFloat: return MOE_DTYPE_FP32;
    default: refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
  }
}

int choice(PyObject* o, const char* a, const char* b, const char* what) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, a) == 0) return 0;
    if (PyUnicode_CompareWithASCIIString(o, b) == 0) return 1;
  }
  refuse(std::string(what) + " must be \"" + a + "\" or \"" + b + "\"");
}
int norm_kind(PyObject* o) {
  static_assert(MOE_NORM_LAYER == 0 && MOE_NORM_RMS == 1, "order of the choice");
  return choice(o, "layer", "rms", "kind");
}
int activation(PyObject* o) {
  static_assert(MOE_ACT_SILU == 0 && MOE_ACT_GELU == 1, "order of the choice");
  return choice(o, "silu", "gelu", "activation");
}

double number(PyObject* o, const char* what) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(what) + " must be a number");
  }
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse("a flag must be a truth value");
  }
  return v != 0;
}

// t as (rows, cols) with unit column stride and rows that neither overlap nor run backwards:
// a view where its strides allow it, otherwise laid out anew.
at::Tensor as_rows(const at::Tensor& t, const char* what) {
  if (t.dim() == 0) refuse(std::string(what) + " must have at least one dimension");
  if (t.size(-1) == 0) refuse(std::string(what) + " has an empty last dimension");
  at::Tensor r = t.dim() == 2 ? t : t.reshape({-1, t.size(-1)});
  if ((r.size(1) > 1 && r.stride(1) != 1) || (r.size(0) > 1 && r.stride(0) < r.size(1)))
    r = r.contiguous();
  return r;
}

void check_like(const at::Tensor& t, const at::Tensor& x, const char* what) {
  if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type() ||
      t.get_device() != x.get_device())
    refuse(std::string(what) + " must be a " + shape_text(x.sizes()) + " " + typed_on(x));
}

at::Tensor empty_as(const at::Tensor& x) { return at::empty(x.sizes(), x.options()); }
at::Tensor bytes_on(const at::Tensor& x, size_t n) {
  return at::empty({static_cast<int64_t>(n)}, x.options().dtype(at::kByte));
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// Call a C entry point with the current stream of x's device, which is made current; other
// Python threads may run meanwhile (a full launch queue blocks).
template <typename F>
void launch(const at::Tensor& x, F call) {
  const c10::cuda::CUDAGuard guard(x.device());
  void* stream = c10::cuda::getCurrentCUDAStream(x.get_device()).stream();
  int status;
  std::string message;
  Py_BEGIN_ALLOW_THREADS
  status = call(stream);
  if (status != MOE_OK) message = moe_last_error();     // of this host thread
  Py_END_ALLOW_THREADS
  if (status != MOE_OK) throw Refusal{status, message};
}

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
template <typename... Ts>
PyObject* wrap_all(const Ts&... ts) {
  PyObject* items[] = {wrap(ts)...};
  constexpr Py_ssize_t n = sizeof...(Ts);
  PyObject* tuple = PyTuple_New(n);
  bool ok = tuple != nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) ok = ok && items[i];
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (ok)
      PyTuple_SET_ITEM(tuple, i, items[i]);
    else
      Py_XDECREF(items[i]);
  }
  if (!ok) {
    Py_XDECREF(tuple);
    return nullptr;
  }
  return tuple;
}

// One entry point: `body` runs below autograd (these calls record nothing); refusals become
// the module's exception, torch's errors torch's.
template <typename F>
PyObject* entry(Py_ssize_t given, Py_ssize_t wanted, F body) {
  HANDLE_TH_ERRORS
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    const at::AutoDispatchBelowADInplaceOrView below_autograd;
    return body();
  } catch (const Refusal& r) {
    return raise(r);
  }
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ norm
at::Tensor norm_vector(PyObject* o, const at::Tensor& x, int64_t cols, const char* what) {
  if (o == Py_None) return at::Tensor();
  const at::Tensor& t = cuda_tensor(o, what);
  if (t.dim() != 1 || t.size(0) != cols || t.get_device() != x.get_device() ||
      (t.scalar_type() != x.scalar_type() && t.scalar_type() != at::kFloat))
    refuse(std::string(what) + " must be a (" + std::to_string(cols) +
           ",) tensor of x's type or fp32 on " + x.device().str());
  return t.is_contiguous() ? t : t.contiguous();
}

// norm_forward(x, weight, bias, eps, kind, save)
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t given) {
  return entry(given, 6, [&]() -> PyObject* {
    const at::Tensor& x = cuda_tensor(a[0], "x");
    const int dt = dtype_of(x), kind = norm_kind(a[4]);
    const at::Tensor x2 = as_rows(x, "x");
    const int64_t rows = x2.size(0), cols = x2.size(1);
    const at::Tensor weight = norm_vector(a[1], x, cols, "weight");
    const at::Tensor bias = norm_vector(a[2], x, cols, "bias");
    const double eps = number(a[3], "eps");
    if (kind == MOE_NORM_RMS && bias.defined()) refuse("an RMS norm has no bias");
    if (weight.defined() && bias.defined() && weight.scalar_type() != bias.scalar_type())
      refuse("weight and bias must have the same type");
    const int wdt = weight.defined() ? dtype_of(weight) : bias.defined() ? dtype_of(bias) : dt;
    const at::Tensor y = empty_as(x);
    at::Tensor mean, rstd;
    const bool save = truth(a[5]);
    if (save) {
      rstd = at::empty({rows}, x.options().dtype(at::kFloat));
      if (kind == MOE_NORM_LAYER) mean = at::empty({rows}, x.options().dtype(at::kFloat));
    }
    launch(x, [&](void* stream) {
      return moe_norm_forward(kind, dt, wdt, rows, cols, x2.data_ptr(), x2.stride(0), ptr(weight),
                              ptr(bias), eps, y.data_ptr(), cols,
                              static_cast<float*>(ptr(mean)), static_cast<float*>(ptr(rstd)),
                              stream);
    });
    return save ? wrap_all(y, mean, rstd) : wrap(y);
  });
}

const at::Tensor& saved_stat(PyObject* o, const at::Tensor& x, int64_t rows, const char* what) {
  const at::Tensor& t = cuda_tensor(o, what);
  if (t.dim() != 1 || t.size(0) != rows || t.scalar_type() != at::kFloat ||
      t.get_device() != x.get_device() || !t.is_contiguous())
    refuse(std::string(what) + " must be the contiguous fp32 (" + std::to_string(rows) +
           ",) tensor of norm_forward");
  return t;
}

// norm_backward(dy, x, weight, mean, rstd, kind, bias, need_dx, need_dweight, grad_fp32)
// grad_fp32: None, or whether dbias (without a weight) is fp32 instead of x's type
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t given) {
  return entry(given, 10, [&]() -> PyObject* {
    const at::Tensor& x = cuda_tensor(a[1], "x");
    const at::Tensor& dy = cuda_tensor(a[0], "dy");
    const int dt = dtype_of(x), kind = norm_kind(a[5]);
    check_like(dy, x, "dy");
    const at::Tensor x2 = as_rows(x, "x"), dy2 = as_rows(dy, "dy");
    const int64_t rows = x2.size(0), cols = x2.size(1);
    const at::Tensor weight = norm_vector(a[2], x, cols, "weight");
    const bool want_bias = truth(a[6]);
    if (kind == MOE_NORM_RMS && want_bias) refuse("an RMS norm has no bias");
    const at::Tensor& rstd = saved_stat(a[4], x, rows, "rstd");
    float* mean = nullptr;
    if (kind == MOE_NORM_LAYER)
      mean = static_cast<float*>(saved_stat(a[3], x, rows, "mean").data_ptr());
    const at::ScalarType wtype = weight.defined()                         ? weight.scalar_type()
                                 : a[9] != Py_None && truth(a[9]) ? at::kFloat
                                                                          : x.scalar_type();
    at::Tensor dx, dweight, dbias, ws;
    if (truth(a[7])) dx = empty_as(x);
    if (truth(a[8]) && weight.defined()) dweight = empty_as(weight);
    if (want_bias) dbias = at::empty({cols}, x.options().dtype(wtype));
    size_t bytes = 0;
    if (dweight.defined() || dbias.defined()) {
      bytes = moe_norm_workspace_bytes(kind, rows, cols);
      ws = bytes_on(x, bytes < 16 ? 16 : bytes);
    }
    const int wdt = wtype == at::kFloat ? MOE_DTYPE_FP32 : dt;
    launch(x, [&](void* stream) {
      return moe_norm_backward(kind, dt, wdt, rows, cols, dy2.data_ptr(), dy2.stride(0),
                               x2.data_ptr(), x2.stride(0), ptr(weight), mean,
                               static_cast<const float*>(rstd.data_ptr()), ptr(dx), cols,
                               ptr(dweight), ptr(dbias), ptr(ws), bytes, stream);
    });
    return wrap_all(dx, dweight, dbias);
  });
}

// ------------------------------------------------------------------ gated feed-forward
// Rows the tensor maps can describe: 16-byte aligned rows and base.
at::Tensor map_rows(const at::Tensor& t, const char* what) {
  at::Tensor r = as_rows(t, what);
  if (reinterpret_cast<uintptr_t>(r.data_ptr()) % 16 || (r.size(0) > 1 && r.stride(0) % 8))
    r = r.clone(at::MemoryFormat::Contiguous);
  return r;
}

struct FfnWeights {
  const at::Tensor &w1, &w3, &w2;
  int64_t d, f;
};
FfnWeights ffn_weights(const at::Tensor& x, PyObject* p1, PyObject* p3, PyObject* p2) {
  const at::Tensor& w1 = cuda_tensor(p1, "W1");
  FfnWeights w{w1, cuda_tensor(p3, "W3"), cuda_tensor(p2, "W2"), 0, 0};
  if (x.dim() < 1 || w1.dim() != 2) refuse("x needs a last dimension d and W1 the shape (f, d)");
  w.d = x.size(-1);
  w.f = w1.size(0);
  const auto check = [&](const at::Tensor& t, int64_t r, int64_t c, const char* what) {
    if (t.dim() != 2 || t.size(0) != r || t.size(1) != c || t.scalar_type() != x.scalar_type() ||
        t.get_device() != x.get_device() || !t.is_contiguous())
      refuse(std::string(what) + " must be a contiguous (" + std::to_string(r) + ", " +
             std::to_string(c) + ") " + typed_on(x));
  };
  check(w.w1, w.f, w.d, "W1");
  check(w.w3, w.f, w.d, "W3");
  check(w.w2, w.d, w.f, "W2");
  return w;
}

// gated_ffn_forward(x, W1, W3, W2, activation, save)
PyObject* gated_ffn_forward(PyObject*, PyObject* const* a, Py_ssize_t given) {
  return entry(given, 6, [&]() -> PyObject* {
    const at::Tensor& x = cuda_tensor(a[0], "x");
    const FfnWeights w = ffn_weights(x, a[1], a[2], a[3]);
    const int dt = dtype_of(x), act = activation(a[4]);
    const at::Tensor x2 = map_rows(x, "x");
    const int64_t T = x2.size(0);
    const at::Tensor out = empty_as(x);
    at::Tensor gate, up;
    const bool save = truth(a[5]);
    if (save) {
      gate = at::empty({T, w.f}, x.options().dtype(at::kFloat));
      up = at::empty({T, w.f}, x.options().dtype(at::kFloat));
    }
    const size_t bytes = moe_gated_ffn_workspace_bytes(T, w.d, w.f, 0);
    const at::Tensor ws = bytes_on(x, bytes);
    launch(x, [&](void* stream) {
      return moe_gated_ffn_forward(act, dt, T, w.d, w.f, x2.data_ptr(), x2.stride(0),
                                   w.w1.data_ptr(), w.w3.data_ptr(), w.w2.data_ptr(),
                                   out.data_ptr(), w.d, static_cast<float*>(ptr(gate)),
                                   static_cast<float*>(ptr(up)), ws.data_ptr(), bytes, stream);
    });
    return save ? wrap_all(out, gate, up) : wrap(out);
  });
}

const at::Tensor& saved_rows(PyObject* o, const at::Tensor& x, int64_t T, int64_t f,
                             const char* what) {
  const at::Tensor& t = cuda_tensor(o, what);
  if (t.dim() != 2 || t.size(0) != T || t.size(1) != f || t.scalar_type() != at::kFloat ||
      t.get_device() != x.get_device() || !t.is_contiguous())
    refuse(std::string(what) + " must be the contiguous fp32 (" + std::to_string(T) +
           ", " + std::to_string(f) + ") tensor of gated_ffn_forward");
  return t;
}

// gated_ffn_backward(dout, x, W1, W3, W2, gate, up, activation, need_x, need_W1, need_W3, need_W2)
PyObject* gated_ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t given) {
  return entry(given, 12, [&]() -> PyObject* {
    const at::Tensor& x = cuda_tensor(a[1], "x");
    const at::Tensor& dout = cuda_tensor(a[0], "dout");
    const FfnWeights w = ffn_weights(x, a[2], a[3], a[4]);
    const int dt = dtype_of(x), act = activation(a[7]);
    check_like(dout, x, "dout");
    const at::Tensor x2 = map_rows(x, "x"), dout2 = map_rows(dout, "dout");
    const int64_t T = x2.size(0);
    const at::Tensor& gate = saved_rows(a[5], x, T, w.f, "gate");
    const at::Tensor& up = saved_rows(a[6], x, T, w.f, "up");
    at::Tensor dx, d1, d3, d2;
    if (truth(a[8])) dx = empty_as(x);
    if (truth(a[9])) d1 = empty_as(w.w1);
    if (truth(a[10])) d3 = empty_as(w.w3);
    if (truth(a[11])) d2 = empty_as(w.w2);
    const size_t bytes = moe_gated_ffn_workspace_bytes(T, w.d, w.f, 1);
    const at::Tensor ws = bytes_on(x, bytes);
    launch(x, [&](void* stream) {
      return moe_gated_ffn_backward(act, dt, T, w.d, w.f, dout2.data_ptr(), dout2.stride(0),
                                    x2.data_ptr(), x2.stride(0), w.w1.data_ptr(),
                                    w.w3.data_ptr(), w.w2.data_ptr(),
                                    static_cast<const float*>(gate.data_ptr()),
                                    static_cast<const float*>(up.data_ptr()), ptr(dx), w.d,
                                    ptr(d1), ptr(d3), ptr(d2), ws.data_ptr(), bytes, stream);
    });
    return wrap_all(dx, d1, d3, d2);
  });
}

// ------------------------------------------------------------------ dropout
// dropout_add(x, residual, p, rng)
PyObject* dropout_add(PyObject*, PyObject* const* a, Py_ssize_t given) {
  return entry(given, 4, [&]() -> PyObject* {
    const at::Tensor& x = cuda_tensor(a[0], "x");
    const int dt = dtype_of(x);
    if (x.dim() == 0) refuse("x must have at least one dimension");
    const double p = number(a[2], "p");
    if (!(p >= 0.0 && p <= 1.0)) refuse("p must lie in [0, 1]");      // also of an empty tensor
    const uint64_t* rng = nullptr;
    if (!(p == 0.0 && a[3] == Py_None)) {
      const at::Tensor& r = cuda_tensor(a[3], "rng");
      if (r.dim() != 1 || r.size(0) != 2 || r.get_device() != x.get_device() ||
          (r.scalar_type() != at::kLong && r.scalar_type() != at::kUInt64) || !r.is_contiguous())
        refuse("rng must be a contiguous int64 (2,) tensor (seed, offset) on " +
               x.device().str());
      rng = static_cast<const uint64_t*>(r.data_ptr());
    }
    at::Tensor res;
    if (a[1] != Py_None) {
      res = cuda_tensor(a[1], "residual");
      check_like(res, x, "residual");
    }
    const at::Tensor out = empty_as(x);
    if (x.numel() == 0) return wrap(out);
    at::Tensor x2 = x;
    // one line of all elements, whatever the shape, where everything is contiguous
    int64_t rows = 1, cols = x.numel(), ldx = cols, ldr = cols;
    if (!x.is_contiguous() || (res.defined() && !res.is_contiguous())) {
      x2 = as_rows(x, "x");
      if (res.defined()) res = as_rows(res, "residual");
      rows = x2.size(0);
      cols = x2.size(1);
      ldx = x2.stride(0);
      ldr = res.defined() ? res.stride(0) : 0;
    }
    launch(x, [&](void* stream) {
      return moe_dropout_forward(dt, rows, cols, x2.data_ptr(), ldx, ptr(res), ldr, p, rng,
                                 out.data_ptr(), cols, stream);
    });
    return wrap(out);
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {
    {"norm_forward", FAST(norm_forward), nullptr},
    {"norm_backward", FAST(norm_backward), nullptr},
    {"gated_ffn_forward", FAST(gated_ffn_forward), nullptr},
    {"gated_ffn_backward", FAST(gated_ffn_backward), nullptr},
    {"dropout_add", FAST(dropout_add), nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_moe_host", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_host(void) { return PyModule_Create(&kModule); }
