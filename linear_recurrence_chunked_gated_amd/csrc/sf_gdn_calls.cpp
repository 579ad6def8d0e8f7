// Python calls of the layer's operators: checks of torch tensors, allocation
// of the outputs, and the C-ABI call, in one native step.
//
// A decoding step makes several of these calls per layer, each of a few
// microseconds on the GPU, so what the host spends on one counts: with the
// same checks and marshalling in Python (ctypes) a call took 9 to 10 us, of
// which the launch itself is about 3.  The C ABI stays the interface; bind()
// takes the addresses of its entry points in the library that the package has
// loaded, so this module is not linked against it.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>

#include <string>
#include <vector>

#include "../../include/sf_gdn.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct Entries {
  decltype(&sf_gdn_recurrent_step) recurrent_step;
  decltype(&sf_gdn_shortconv_step) shortconv_step;
  decltype(&sf_gdn_gated_norm_fwd) gated_norm_fwd;
  decltype(&sf_gdn_gated_norm_bwd) gated_norm_bwd;
  decltype(&sf_gdn_gated_norm_bwd_workspace_size) gated_norm_bwd_workspace_size;
  decltype(&sf_gdn_residual_norm_fwd) residual_norm_fwd;
  decltype(&sf_gdn_residual_norm_bwd) residual_norm_bwd;
  decltype(&sf_gdn_residual_norm_bwd_workspace_size) residual_norm_bwd_workspace_size;
  decltype(&sf_gdn_decay_chunk_fwd) decay_chunk_fwd;
  decltype(&sf_gdn_decay_chunk_fwd_workspace_size) decay_chunk_fwd_workspace_size;
  decltype(&sf_gdn_decay_chunk_bwd) decay_chunk_bwd;
  decltype(&sf_gdn_decay_chunk_bwd_workspace_size) decay_chunk_bwd_workspace_size;
  decltype(&sf_gdn_decay_step) decay_step;
  decltype(&sf_gdn_qk_norm_rotary_fwd) qk_norm_rotary_fwd;
  decltype(&sf_gdn_qk_norm_rotary_bwd) qk_norm_rotary_bwd;
  decltype(&sf_gdn_qk_norm_rotary_bwd_workspace_size) qk_norm_rotary_bwd_workspace_size;
} g_abi;
PyObject* g_fail = nullptr;  // fail(status, call): raises the package's error

// A Python exception on its way out of the checks.  type null: it is set.
struct Error {
  PyObject* type;
  std::string text;
};
[[noreturn]] void value_error(const std::string& s) { throw Error{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw Error{PyExc_TypeError, s}; }

std::string text(IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}
std::string text(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return "torch.float32";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Double: return "torch.float64";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Byte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (o == Py_None) value_error(std::string(name) + " is required");
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor* optional(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}

void need_type(const Tensor& t, const char* name, ScalarType dtype, IntArrayRef shape,
               c10::Device dev) {
  if (t.device() != dev)
    value_error(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
  if (t.scalar_type() != dtype)
    type_error(std::string(name) + " has dtype " + text(t.scalar_type()) + ", expected " + text(dtype));
  if (t.sizes() != shape)
    value_error(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
}
void need(const Tensor& t, const char* name, ScalarType dtype, IntArrayRef shape, c10::Device dev) {
  need_type(t, name, dtype, shape, dev);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}
void need(const Tensor* t, const char* name, ScalarType dtype, IntArrayRef shape, c10::Device dev) {
  if (t) need(*t, name, dtype, shape, dev);
}

c10::Device device_of(const Tensor& t, const char* name) {
  if (!t.is_cuda())
    value_error(std::string("tensors must be on a GPU device (") + name + " is on " + t.device().str() + ")");
  return t.device();
}
int dtype_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::Float) return SF_DTYPE_F32;
  if (t.scalar_type() == ScalarType::BFloat16) return SF_DTYPE_BF16;
  type_error(std::string(name) + " must be bfloat16 or float32, got " + text(t.scalar_type()));
}

// Elements between the token rows of t, whose last `inner` dimensions are a
// row and contiguous, and whose leading ones may lie apart at one stride (a
// slice of wider rows).  0: contiguous, or at most one row.
int64_t token_rows(const Tensor& t, const char* name, int inner) {
  if (t.is_contiguous() || t.numel() == 0) return 0;
  const auto sizes = t.sizes(), strides = t.strides();
  int64_t width = 1;
  int d = (int)t.dim() - 1;
  for (int i = 0; i < inner; ++i, --d) {
    if (sizes[d] != 1 && strides[d] != width)
      value_error(std::string(name) + ": each token's row must be contiguous");
    width *= sizes[d];
  }
  int64_t row = 0, rows = 1;  // stride of the innermost dimension with rows, rows inside d
  for (; d >= 0; --d) {
    if (sizes[d] == 1) continue;
    if (rows == 1)
      row = strides[d];
    else if (strides[d] != row * rows)
      value_error(std::string(name) + ": the rows of all leading dimensions must lie at one stride, "
                  "got strides " + text(strides) + " of shape " + text(sizes));
    rows *= sizes[d];
  }
  if (rows > 1 && row < width) value_error(std::string(name) + ": token rows must not overlap");
  return rows > 1 ? row : 0;
}

Tensor new_like(const Tensor& t, IntArrayRef shape) { return at::empty(shape, t.options()); }
Tensor new_f32(const Tensor& t, int64_t n) { return at::empty({n}, t.options().dtype(ScalarType::Float)); }

const void* ptr(const Tensor& t) { return t.data_ptr(); }
const void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* out(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
const float* f32(const Tensor* t) { return (const float*)ptr(t); }
const int* i32(const Tensor* t) { return (const int*)ptr(t); }

// Tensors that a call has written: autograd counts that as a
// change in place and refuses values it kept of them.  (Tensors of inference
// mode have no count.)
void written(std::initializer_list<const Tensor*> ts) {
  for (const Tensor* t : ts)
    if (t && t->defined() && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// Arguments of one call, in the wrapper's order.
struct Args {
  PyObject* const* a;
  Py_ssize_t n;
  void count(Py_ssize_t want) const {
    if (n != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
  }
  PyObject* operator[](int i) const { return a[i]; }
  long long integer(int i) const {
    const long long v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) throw Error{nullptr, ""};
    return v;
  }
  int small(int i) const {
    const long long v = integer(i);
    if (v < INT_MIN || v > INT_MAX) value_error("argument out of range");
    return (int)v;
  }
  float real(int i) const {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Error{nullptr, ""};
    return (float)v;
  }
  bool truth(int i) const {
    const int v = PyObject_IsTrue(a[i]);
    if (v < 0) throw Error{nullptr, ""};
    return v;
  }
  void* stream(int i) const {
    void* p = PyLong_AsVoidPtr(a[i]);
    if (!p && PyErr_Occurred()) throw Error{nullptr, ""};
    return p;
  }
};

int fits(int64_t v, const char* name) {
  if (v > INT_MAX) value_error(std::string(name) + " is too large");
  return (int)v;
}

// The C-ABI call `f` with `dev` current and the interpreter free; its failure
// as the package's exception.
template <typename F> void run(c10::Device dev, const char* name, F f) {
  sf_status st;
  {
    const c10::DeviceGuard guard(dev);
    Py_BEGIN_ALLOW_THREADS;
    st = f();
    Py_END_ALLOW_THREADS;
  }
  if (st == SF_OK) return;
  PyObject* r = PyObject_CallFunction(g_fail, "is", (int)st, name);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
  throw Error{nullptr, ""};
}

PyObject* wrap(const Tensor* t) {
  if (!t || !t->defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}
PyObject* tuple(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Error{nullptr, ""};
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw Error{nullptr, ""};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Nothing thrown in `F` leaves the module as anything but a Python exception.
template <PyObject* (*F)(const Args&)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(Args{a, n});
  } catch (const Error& e) {
    if (e.type) PyErr_SetString(e.type, e.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown failure");
  }
  return nullptr;
}

// n_seq of a batch over a pool.
int batch(const Tensor* slots, const Tensor* seq_start, int64_t n_slots, c10::Device dev) {
  int64_t n = n_slots;
  if (slots) {
    if (slots->dim() != 1) value_error("slots must have one dimension");
    n = slots->size(0);
    need(*slots, "slots", ScalarType::Int, {n}, dev);
  }
  if (seq_start) {
    if (seq_start->dim() != 1 || seq_start->size(0) < 1)
      value_error("seq_start must be one-dimensional, n_seq + 1 offsets");
    if (!slots) n = seq_start->size(0) - 1;
    need(*seq_start, "seq_start", ScalarType::Int, {n + 1}, dev);
  }
  return fits(n, "n_seq");
}

// q, k, v, alpha, beta, state, slots, seq_start, o, update, stream -> o
PyObject* recurrent_step(const Args& a) {
  a.count(11);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
               &alpha = tensor(a[3], "alpha"), &beta = tensor(a[4], "beta"),
               &state = tensor(a[5], "state");
  const Tensor *slots = optional(a[6], "slots"), *seq_start = optional(a[7], "seq_start"),
               *o = optional(a[8], "o");
  const c10::Device dev = device_of(q, "q");
  const ScalarType dt = q.scalar_type();
  sf_step_shape s{};
  s.dtype = dtype_code(q, "q");
  if (q.dim() != 3 || v.dim() != 3 || state.dim() != 4)
    value_error("q and v must be [n_tok, heads, D], state [n_slots, Hv, Dv, Dk]");
  const int64_t N = q.size(0), Hk = q.size(1), Dk = q.size(2), Hv = v.size(1), Dv = v.size(2),
                slots_n = state.size(0);
  need_type(k, "k", dt, {N, Hk, Dk}, dev);
  need_type(v, "v", dt, {N, Hv, Dv}, dev);
  s.q_stride = token_rows(q, "q", 2);
  s.k_stride = token_rows(k, "k", 2);
  s.v_stride = token_rows(v, "v", 2);
  need(alpha, "alpha", ScalarType::Float, {N, Hv}, dev);
  need(beta, "beta", ScalarType::Float, {N, Hv}, dev);
  need(state, "state", ScalarType::Float, {slots_n, Hv, Dv, Dk}, dev);
  s.n_seq = batch(slots, seq_start, slots_n, dev);
  s.n_tok = fits(N, "n_tok");
  s.n_slots = fits(slots_n, "n_slots");
  s.Hk = fits(Hk, "Hk");
  s.Hv = fits(Hv, "Hv");
  s.Dk = fits(Dk, "Dk");
  s.Dv = fits(Dv, "Dv");
  s.update = a.truth(9);
  void* st = a.stream(10);
  need(o, "o", dt, {N, Hv, Dv}, dev);
  const Tensor made = o ? Tensor() : new_like(v, {N, Hv, Dv});
  if (!o) o = &made;
  run(dev, "sf_gdn_recurrent_step", [&] {
    return g_abi.recurrent_step(&s, ptr(q), ptr(k), ptr(v), f32(&alpha), f32(&beta), i32(slots),
                                i32(seq_start), (float*)out(&state), out(o), st);
  });
  written({s.update ? &state : nullptr, o});
  return wrap(o);
}

// x, w, state, slots, seq_start, act, y, update, stream -> y
PyObject* shortconv_step(const Args& a) {
  a.count(9);
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &state = tensor(a[2], "state");
  const Tensor *slots = optional(a[3], "slots"), *seq_start = optional(a[4], "seq_start"),
               *y = optional(a[6], "y");
  const c10::Device dev = device_of(x, "x");
  if (x.dim() != 2 || w.dim() != 2 || state.dim() != 3)
    value_error("x must be [n_tok, C], w [C, W], state [n_slots, W-1, C]");
  const ScalarType dt = x.scalar_type();
  const int64_t N = x.size(0), C = x.size(1), W = w.size(1), slots_n = state.size(0);
  sf_conv_step_shape s{};
  s.dtype = dtype_code(x, "x");
  s.x_stride = token_rows(x, "x", 1);
  need(w, "w", ScalarType::Float, {C, W}, dev);
  need(state, "state", dt, {slots_n, W - 1, C}, dev);
  s.n_seq = batch(slots, seq_start, slots_n, dev);
  s.n_tok = fits(N, "n_tok");
  s.n_slots = fits(slots_n, "n_slots");
  s.C = fits(C, "C");
  s.W = fits(W, "W");
  s.act = a.small(5);
  s.update = a.truth(7);
  void* st = a.stream(8);
  need(y, "y", dt, {N, C}, dev);
  const Tensor made = y ? Tensor() : new_like(x, {N, C});
  if (!y) y = &made;
  run(dev, "sf_gdn_shortconv_step", [&] {
    return g_abi.shortconv_step(&s, ptr(x), f32(&w), i32(slots), i32(seq_start), out(&state),
                                out(y), st);
  });
  written({s.update ? &state : nullptr, y});
  return wrap(y);
}

// The gated norm's shape from x [..., H, D] and a gate like it.
sf_gated_norm_shape gated_shape(const Tensor& x, const Tensor* gate, const Tensor* w, float eps,
                                float scale, int act, c10::Device dev) {
  if (x.dim() < 3) value_error("expected [..., H, D], got shape " + text(x.sizes()));
  sf_gated_norm_shape s{};
  const int64_t D = x.size(-1), H = x.size(-2);
  s.dtype = dtype_code(x, "x");
  s.N = 1;
  for (int64_t d = 0; d < x.dim() - 2; ++d) s.N *= x.size(d);
  s.H = fits(H, "H");
  s.D = fits(D, "D");
  s.act = act;
  s.eps = eps;
  s.scale = scale;
  s.x_stride = token_rows(x, "x", 2);
  if (gate) {
    need_type(*gate, "gate", x.scalar_type(), x.sizes(), dev);
    s.gate_stride = token_rows(*gate, "gate", 2);
  }
  need(w, "w", ScalarType::Float, {D}, dev);
  return s;
}

// x, gate, w, eps, scale, act, y, stream -> y
PyObject* gated_norm_fwd(const Args& a) {
  a.count(8);
  const Tensor& x = tensor(a[0], "x");
  const Tensor *gate = optional(a[1], "gate"), *w = optional(a[2], "w"), *y = optional(a[6], "y");
  const c10::Device dev = device_of(x, "x");
  const sf_gated_norm_shape s = gated_shape(x, gate, w, a.real(3), a.real(4), a.small(5), dev);
  void* st = a.stream(7);
  need(y, "y", x.scalar_type(), x.sizes(), dev);
  const Tensor made = y ? Tensor() : new_like(x, x.sizes());
  if (!y) y = &made;
  run(dev, "sf_gdn_gated_norm_fwd",
      [&] { return g_abi.gated_norm_fwd(&s, ptr(x), ptr(gate), f32(w), out(y), st); });
  written({y});
  return wrap(y);
}

// The caller's workspace if it is large enough, else a new one.
Tensor workspace(const Tensor* given, size_t bytes, const Tensor& like) {
  if (given) need(*given, "workspace", ScalarType::Byte, {given->numel()}, like.device());
  if (given && (size_t)given->numel() >= bytes) return *given;
  if (bytes == 0) return Tensor();
  const auto opt = like.options().dtype(ScalarType::Byte);
  Tensor t = at::empty({(int64_t)bytes}, opt);
  if ((uintptr_t)t.data_ptr() % 256) {
    t = at::empty({(int64_t)bytes + 256}, opt);
    t = t.narrow(0, (256 - (int64_t)((uintptr_t)t.data_ptr() % 256)) % 256, (int64_t)bytes);
  }
  return t;
}
size_t bytes_of(const Tensor& t) { return t.defined() ? (size_t)t.numel() : 0; }

// Three (four) optional outputs out of `grads`, None or a tuple.
void unpack(PyObject* grads, Py_ssize_t n, PyObject** g) {
  for (Py_ssize_t i = 0; i < n; ++i) g[i] = Py_None;
  if (grads == Py_None) return;
  if (!PyTuple_Check(grads) || PyTuple_GET_SIZE(grads) != n)
    type_error("grads must be a tuple of " + std::to_string(n) + " outputs");
  for (Py_ssize_t i = 0; i < n; ++i) g[i] = PyTuple_GET_ITEM(grads, i);
}

// x, gate, w, dy, eps, scale, act, grads, want_dw, workspace, stream
//   -> dx, dgate, dw, workspace
PyObject* gated_norm_bwd(const Args& a) {
  a.count(11);
  const Tensor &x = tensor(a[0], "x"), &dy = tensor(a[3], "dy");
  const Tensor *gate = optional(a[1], "gate"), *w = optional(a[2], "w"),
               *given = optional(a[9], "workspace");
  const c10::Device dev = device_of(x, "x");
  const ScalarType dt = x.scalar_type();
  const sf_gated_norm_shape s = gated_shape(x, gate, w, a.real(4), a.real(5), a.small(6), dev);
  need(dy, "dy", dt, x.sizes(), dev);
  const bool want_dw = a.truth(8) && w;
  PyObject* g[3];
  unpack(a[7], 3, g);
  Tensor dx, dgate, dw, ws;
  if (a[7] == Py_None) {
    dx = new_like(x, x.sizes());
    if (gate) dgate = new_like(x, x.sizes());
    if (want_dw) dw = new_f32(x, s.D);
  } else {
    dx = tensor(g[0], "dx");
    need(dx, "dx", dt, x.sizes(), dev);
    if (gate) {
      dgate = tensor(g[1], "dgate");
      need(dgate, "dgate", dt, x.sizes(), dev);
    } else if (g[1] != Py_None) {
      value_error("dgate without gate");
    }
    if (want_dw) {
      dw = tensor(g[2], "dw");
      need(dw, "dw", ScalarType::Float, {s.D}, dev);
    }
  }
  if (want_dw) {
    size_t bytes = 0;
    run(dev, "sf_gdn_gated_norm_bwd_workspace_size",
        [&] { return g_abi.gated_norm_bwd_workspace_size(&s, &bytes); });
    ws = workspace(given, bytes, x);
  }
  void* st = a.stream(10);
  run(dev, "sf_gdn_gated_norm_bwd", [&] {
    return g_abi.gated_norm_bwd(&s, ptr(x), ptr(gate), f32(w), ptr(dy), dx.data_ptr(),
                                dgate.defined() ? dgate.data_ptr() : nullptr,
                                dw.defined() ? (float*)dw.data_ptr() : nullptr,
                                ws.defined() ? ws.data_ptr() : nullptr, bytes_of(ws), st);
  });
  written({&dx, &dgate, &dw, &ws});
  return tuple({&dx, &dgate, &dw, &ws});
}

sf_residual_norm_shape residual_shape(const Tensor& x, const char* name, float scale, float eps) {
  sf_residual_norm_shape s{};
  s.dtype = dtype_code(x, name);
  if (x.dim() < 1) value_error(std::string(name) + " must be [..., C]");
  const int64_t C = x.size(-1);
  s.C = fits(C, "C");
  s.N = C ? x.numel() / C : 0;
  s.eps = eps;
  s.scale = scale;
  return s;
}

// x, r, w, s, scale, eps, h, y, stream -> y, h
PyObject* residual_norm_fwd(const Args& a) {
  a.count(9);
  const Tensor& x = tensor(a[0], "x");
  const Tensor *r = optional(a[1], "r"), *w = optional(a[2], "w"), *s = optional(a[3], "s"),
               *h = optional(a[6], "h"), *y = optional(a[7], "y");
  const c10::Device dev = device_of(x, "x");
  const ScalarType dt = x.scalar_type();
  const sf_residual_norm_shape sh = residual_shape(x, "x", a.real(4), a.real(5));
  void* st = a.stream(8);
  need(x, "x", dt, x.sizes(), dev);
  need(w, "w", ScalarType::Float, {sh.C}, dev);
  need(s, "s", ScalarType::Float, {sh.C}, dev);
  need(r, "r", dt, x.sizes(), dev);
  if (!r && (s || h)) value_error("s and h need r");
  need(h, "h", dt, x.sizes(), dev);
  need(y, "y", dt, x.sizes(), dev);
  const Tensor made_h = r && !h ? new_like(x, x.sizes()) : Tensor();
  const Tensor made_y = y ? Tensor() : new_like(x, x.sizes());
  if (r && !h) h = &made_h;
  if (!y) y = &made_y;
  run(dev, "sf_gdn_residual_norm_fwd", [&] {
    return g_abi.residual_norm_fwd(&sh, ptr(x), ptr(r), f32(s), f32(w), out(h), out(y), st);
  });
  written({y, h});
  return tuple({y, r ? h : &x});
}

// h, r, w, s, dy, dh, scale, eps, grads, want_dr, want_dw, want_ds, workspace, stream
//   -> dx, dr, dw, ds, workspace
PyObject* residual_norm_bwd(const Args& a) {
  a.count(14);
  const Tensor &h = tensor(a[0], "h"), &dy = tensor(a[4], "dy");
  const Tensor *w = optional(a[2], "w"), *s = optional(a[3], "s"), *dh = optional(a[5], "dh"),
               *given = optional(a[12], "workspace"), *r = nullptr;
  const c10::Device dev = device_of(h, "h");
  const ScalarType dt = h.scalar_type();
  const sf_residual_norm_shape sh = residual_shape(h, "h", a.real(6), a.real(7));
  need(h, "h", dt, h.sizes(), dev);
  need(dy, "dy", dt, h.sizes(), dev);
  need(dh, "dh", dt, h.sizes(), dev);
  need(w, "w", ScalarType::Float, {sh.C}, dev);
  need(s, "s", ScalarType::Float, {sh.C}, dev);
  const bool want_dr = a.truth(9), want_dw = a.truth(10) && w, want_ds = a.truth(11) && s;
  if (want_ds) {
    r = &tensor(a[1], "r");
    need(*r, "r", dt, h.sizes(), dev);
  }
  PyObject* g[4];
  unpack(a[8], 4, g);
  Tensor dx, dr, dw, ds, ws;
  if (a[8] == Py_None) {
    dx = new_like(h, h.sizes());
    if (want_dr) dr = new_like(h, h.sizes());
    if (want_dw) dw = new_f32(h, sh.C);
    if (want_ds) ds = new_f32(h, sh.C);
  } else {
    dx = tensor(g[0], "dx");
    need(dx, "dx", dt, h.sizes(), dev);
    if (want_dr) {
      dr = tensor(g[1], "dr");
      need(dr, "dr", dt, h.sizes(), dev);
    }
    if (want_dw) {
      dw = tensor(g[2], "dw");
      need(dw, "dw", ScalarType::Float, {sh.C}, dev);
    }
    if (want_ds) {
      ds = tensor(g[3], "ds");
      need(ds, "ds", ScalarType::Float, {sh.C}, dev);
    }
  }
  if (want_dw || want_ds) {
    size_t bytes = 0;
    run(dev, "sf_gdn_residual_norm_bwd_workspace_size",
        [&] { return g_abi.residual_norm_bwd_workspace_size(&sh, &bytes); });
    ws = workspace(given, bytes, h);
  }
  void* st = a.stream(13);
  run(dev, "sf_gdn_residual_norm_bwd", [&] {
    return g_abi.residual_norm_bwd(&sh, ptr(h), ptr(r), f32(s), f32(w), ptr(dy), ptr(dh),
                                   dx.data_ptr(), dr.defined() ? dr.data_ptr() : nullptr,
                                   dw.defined() ? (float*)dw.data_ptr() : nullptr,
                                   ds.defined() ? (float*)ds.data_ptr() : nullptr,
                                   ws.defined() ? ws.data_ptr() : nullptr, bytes_of(ws), st);
  });
  written({&dx, &dr, &dw, &ds, &ws});
  return tuple({&dx, &dr, &dw, &ds, &ws});
}

// The decay chunk's shape from q, k [B, T, Hk, D], v [B, T, Hv, D], or from
// packed rows [n_tok, H, D] with seq_start (without it: one sequence).
struct DecayChunk {
  sf_decay_shape s{};
  int64_t n_seq, Hv, Dv, Dk;
};
DecayChunk decay_chunk(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& decay,
                       const Tensor* seq_start, double scale, c10::Device dev) {
  DecayChunk c;
  const ScalarType dt = q.scalar_type();
  c.s.dtype = dtype_code(q, "q");
  if ((q.dim() != 3 && q.dim() != 4) || v.dim() != q.dim())
    value_error("q and v must be [B, T, heads, D], or [n_tok, heads, D] packed");
  if (seq_start && q.dim() != 3) value_error("packed sequences (seq_start) are [n_tok, heads, D]");
  c.Dk = q.size(-1);
  c.Dv = v.size(-1);
  c.Hv = v.size(-2);
  const int64_t Hk = q.size(-2);
  std::vector<int64_t> want(q.sizes().begin(), q.sizes().end());
  need_type(k, "k", dt, want, dev);
  want[want.size() - 2] = c.Hv;
  want.back() = c.Dv;
  need_type(v, "v", dt, want, dev);
  need(decay, "decay", ScalarType::Float, {c.Hv}, dev);
  c.s.q_stride = token_rows(q, "q", 2);
  c.s.k_stride = token_rows(k, "k", 2);
  c.s.v_stride = token_rows(v, "v", 2);
  int64_t n_tok = q.size(0);
  if (q.dim() == 4) {
    c.n_seq = q.size(0);
    if (q.size(1) && c.n_seq > INT_MAX / q.size(1)) value_error("n_tok is too large");
    n_tok *= q.size(1);
  } else {
    c.n_seq = seq_start ? batch(nullptr, seq_start, 0, dev) : 1;
  }
  c.s.n_seq = fits(c.n_seq, "n_seq");
  c.s.n_tok = fits(n_tok, "n_tok");
  c.s.Hk = fits(Hk, "Hk");
  c.s.Hv = fits(c.Hv, "Hv");
  c.s.Dk = fits(c.Dk, "Dk");
  c.s.Dv = fits(c.Dv, "Dv");
  c.s.scale = (float)scale;
  return c;
}

// q, k, v, decay, S_in, seq_start, scale, o, S_out, workspace, stream -> o, S_out, workspace
PyObject* decay_chunk_fwd(const Args& a) {
  a.count(11);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
               &decay = tensor(a[3], "decay");
  const Tensor *S_in = optional(a[4], "S_in"), *seq_start = optional(a[5], "seq_start"),
               *o = optional(a[7], "o"), *S_out = optional(a[8], "S_out"),
               *given = optional(a[9], "workspace");
  const c10::Device dev = device_of(q, "q");
  const DecayChunk c = decay_chunk(q, k, v, decay, seq_start, a.real(6), dev);
  void* st = a.stream(10);
  need(S_in, "S_in", ScalarType::Float, {c.n_seq, c.Hv, c.Dv, c.Dk}, dev);
  need(o, "o", q.scalar_type(), v.sizes(), dev);
  need(S_out, "S_out", ScalarType::Float, {c.n_seq, c.Hv, c.Dv, c.Dk}, dev);
  const Tensor made_o = o ? Tensor() : new_like(v, v.sizes());
  const Tensor made_S = S_out ? Tensor() : at::empty({c.n_seq, c.Hv, c.Dv, c.Dk},
                                                     v.options().dtype(ScalarType::Float));
  if (!o) o = &made_o;
  if (!S_out) S_out = &made_S;
  size_t bytes = 0;
  run(dev, "sf_gdn_decay_chunk_fwd_workspace_size",
      [&] { return g_abi.decay_chunk_fwd_workspace_size(&c.s, &bytes); });
  const Tensor ws = workspace(given, bytes, q);
  run(dev, "sf_gdn_decay_chunk_fwd", [&] {
    return g_abi.decay_chunk_fwd(&c.s, ptr(q), ptr(k), ptr(v), f32(&decay), i32(seq_start), f32(S_in),
                                 out(o), (float*)out(S_out), ws.defined() ? ws.data_ptr() : nullptr,
                                 bytes_of(ws), st);
  });
  written({o, S_out, &ws});
  return tuple({o, S_out, &ws});
}

// q, k, v, decay, S_in, dO, dS_out, seq_start, scale, grads, want_dS_in, workspace, stream
//   -> dq, dk, dv, dS_in, workspace
PyObject* decay_chunk_bwd(const Args& a) {
  a.count(13);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
               &decay = tensor(a[3], "decay"), &dO = tensor(a[5], "dO");
  const Tensor *S_in = optional(a[4], "S_in"), *dS_out = optional(a[6], "dS_out"),
               *seq_start = optional(a[7], "seq_start"), *given = optional(a[11], "workspace");
  const c10::Device dev = device_of(q, "q");
  const DecayChunk c = decay_chunk(q, k, v, decay, seq_start, a.real(8), dev);
  const ScalarType dt = q.scalar_type();
  const std::vector<int64_t> state{c.n_seq, c.Hv, c.Dv, c.Dk};
  void* st = a.stream(12);
  need(S_in, "S_in", ScalarType::Float, state, dev);
  need(dO, "dO", dt, v.sizes(), dev);
  need(dS_out, "dS_out", ScalarType::Float, state, dev);
  const bool want = a.truth(10);
  PyObject* g[4];
  unpack(a[9], 4, g);
  Tensor dq, dk, dv, dS;
  if (a[9] == Py_None) {
    dq = new_like(q, q.sizes());
    dk = new_like(k, k.sizes());
    dv = new_like(v, v.sizes());
    if (want) dS = at::empty(state, v.options().dtype(ScalarType::Float));
  } else {
    dq = tensor(g[0], "dq");
    need(dq, "dq", dt, q.sizes(), dev);
    dk = tensor(g[1], "dk");
    need(dk, "dk", dt, k.sizes(), dev);
    dv = tensor(g[2], "dv");
    need(dv, "dv", dt, v.sizes(), dev);
    if (want) {
      dS = tensor(g[3], "dS_in");
      need(dS, "dS_in", ScalarType::Float, state, dev);
    }
  }
  size_t bytes = 0;
  run(dev, "sf_gdn_decay_chunk_bwd_workspace_size",
      [&] { return g_abi.decay_chunk_bwd_workspace_size(&c.s, &bytes); });
  const Tensor ws = workspace(given, bytes, q);
  run(dev, "sf_gdn_decay_chunk_bwd", [&] {
    return g_abi.decay_chunk_bwd(&c.s, ptr(q), ptr(k), ptr(v), f32(&decay), i32(seq_start), f32(S_in),
                                 ptr(dO), f32(dS_out), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                 dS.defined() ? (float*)dS.data_ptr() : nullptr,
                                 ws.defined() ? ws.data_ptr() : nullptr, bytes_of(ws), st);
  });
  written({&dq, &dk, &dv, &dS, &ws});
  return tuple({&dq, &dk, &dv, &dS, &ws});
}

// q, k, v, decay, state, slots, seq_start, o, update, scale, stream -> o
PyObject* decay_step(const Args& a) {
  a.count(11);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
               &decay = tensor(a[3], "decay"), &state = tensor(a[4], "state");
  const Tensor *slots = optional(a[5], "slots"), *seq_start = optional(a[6], "seq_start"),
               *o = optional(a[7], "o");
  const c10::Device dev = device_of(q, "q");
  const ScalarType dt = q.scalar_type();
  sf_decay_step_shape s{};
  s.dtype = dtype_code(q, "q");
  if (q.dim() != 3 || v.dim() != 3 || state.dim() != 4)
    value_error("q and v must be [n_tok, heads, D], state [n_slots, Hv, Dv, Dk]");
  const int64_t N = q.size(0), Hk = q.size(1), Dk = q.size(2), Hv = v.size(1), Dv = v.size(2),
                slots_n = state.size(0);
  need_type(k, "k", dt, {N, Hk, Dk}, dev);
  need_type(v, "v", dt, {N, Hv, Dv}, dev);
  s.q_stride = token_rows(q, "q", 2);
  s.k_stride = token_rows(k, "k", 2);
  s.v_stride = token_rows(v, "v", 2);
  need(decay, "decay", ScalarType::Float, {Hv}, dev);
  need(state, "state", ScalarType::Float, {slots_n, Hv, Dv, Dk}, dev);
  s.n_seq = batch(slots, seq_start, slots_n, dev);
  s.n_tok = fits(N, "n_tok");
  s.n_slots = fits(slots_n, "n_slots");
  s.Hk = fits(Hk, "Hk");
  s.Hv = fits(Hv, "Hv");
  s.Dk = fits(Dk, "Dk");
  s.Dv = fits(Dv, "Dv");
  s.update = a.truth(8);
  s.scale = a.real(9);
  void* st = a.stream(10);
  need(o, "o", dt, {N, Hv, Dv}, dev);
  const Tensor made = o ? Tensor() : new_like(v, {N, Hv, Dv});
  if (!o) o = &made;
  run(dev, "sf_gdn_decay_step", [&] {
    return g_abi.decay_step(&s, ptr(q), ptr(k), ptr(v), f32(&decay), i32(slots), i32(seq_start),
                            (float*)out(&state), out(o), st);
  });
  written({s.update ? &state : nullptr, o});
  return wrap(o);
}

// The rotary call's shape from q [..., Hq, D], k [..., Hk, D].
sf_rotary_shape rotary_shape(const Tensor& q, const Tensor& k, const Tensor* pos, const Tensor* freq,
                             const Tensor* wq, const Tensor* wk, c10::Device dev) {
  if (q.dim() < 3 || k.dim() != q.dim())
    value_error("q and k must be [..., heads, D], got shapes " + text(q.sizes()) + " and " + text(k.sizes()));
  sf_rotary_shape s{};
  const int64_t D = q.size(-1), Hq = q.size(-2), Hk = k.size(-2);
  s.dtype = dtype_code(q, "q");
  std::vector<int64_t> want(q.sizes().begin(), q.sizes().end());
  want[want.size() - 2] = Hk;
  need_type(k, "k", q.scalar_type(), want, dev);
  s.N = 1;
  for (int64_t d = 0; d < q.dim() - 2; ++d) s.N *= q.size(d);
  s.T = q.size(-3);
  s.Hq = fits(Hq, "Hq");
  s.Hk = fits(Hk, "Hk");
  s.D = fits(D, "D");
  s.q_stride = token_rows(q, "q", 2);
  s.k_stride = token_rows(k, "k", 2);
  want.resize(want.size() - 2);
  need(pos, "pos", ScalarType::Int, want, dev);
  if (freq) {
    if (freq->dim() != 1) value_error("freq must have one dimension");
    s.F = fits(freq->size(0), "F");
    need(*freq, "freq", ScalarType::Float, {freq->size(0)}, dev);
  }
  need(wq, "wq", ScalarType::Float, {D}, dev);
  need(wk, "wk", ScalarType::Float, {D}, dev);
  return s;
}

// q, k, pos, freq, wq, wk, eps, q_scale, k_scale, neighbours, first, yq, yk, stream -> yq, yk
PyObject* qk_norm_rotary_fwd(const Args& a) {
  a.count(14);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const Tensor *pos = optional(a[2], "pos"), *freq = optional(a[3], "freq"), *wq = optional(a[4], "wq"),
               *wk = optional(a[5], "wk"), *yq = optional(a[11], "yq"), *yk = optional(a[12], "yk");
  const c10::Device dev = device_of(q, "q");
  sf_rotary_shape s = rotary_shape(q, k, pos, freq, wq, wk, dev);
  s.eps = a.real(6);
  s.q_scale = a.real(7);
  s.k_scale = a.real(8);
  s.neighbours = a.truth(9);
  s.first = a.small(10);
  void* st = a.stream(13);
  need(yq, "yq", q.scalar_type(), q.sizes(), dev);
  need(yk, "yk", q.scalar_type(), k.sizes(), dev);
  const Tensor made_q = yq ? Tensor() : new_like(q, q.sizes());
  const Tensor made_k = yk ? Tensor() : new_like(k, k.sizes());
  if (!yq) yq = &made_q;
  if (!yk) yk = &made_k;
  run(dev, "sf_gdn_qk_norm_rotary_fwd", [&] {
    return g_abi.qk_norm_rotary_fwd(&s, ptr(q), ptr(k), i32(pos), f32(freq), f32(wq), f32(wk), out(yq),
                                    out(yk), st);
  });
  written({yq, yk});
  return tuple({yq, yk});
}

// q, k, pos, freq, wq, wk, dyq, dyk, eps, q_scale, k_scale, neighbours, first, grads, want_dw,
// workspace, stream -> dq, dk, dwq, dwk, workspace
PyObject* qk_norm_rotary_bwd(const Args& a) {
  a.count(17);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &dyq = tensor(a[6], "dyq"),
               &dyk = tensor(a[7], "dyk");
  const Tensor *pos = optional(a[2], "pos"), *freq = optional(a[3], "freq"), *wq = optional(a[4], "wq"),
               *wk = optional(a[5], "wk"), *given = optional(a[15], "workspace");
  const c10::Device dev = device_of(q, "q");
  const ScalarType dt = q.scalar_type();
  sf_rotary_shape s = rotary_shape(q, k, pos, freq, wq, wk, dev);
  s.eps = a.real(8);
  s.q_scale = a.real(9);
  s.k_scale = a.real(10);
  s.neighbours = a.truth(11);
  s.first = a.small(12);
  void* st = a.stream(16);
  need(dyq, "dyq", dt, q.sizes(), dev);
  need(dyk, "dyk", dt, k.sizes(), dev);
  const bool want_dw = a.truth(14);
  PyObject* g[4];
  unpack(a[13], 4, g);
  Tensor dq, dk, dwq, dwk, ws;
  if (a[13] == Py_None) {
    dq = new_like(q, q.sizes());
    dk = new_like(k, k.sizes());
    if (want_dw && wq) dwq = new_f32(q, s.D);
    if (want_dw && wk) dwk = new_f32(q, s.D);
  } else {
    dq = tensor(g[0], "dq");
    need(dq, "dq", dt, q.sizes(), dev);
    dk = tensor(g[1], "dk");
    need(dk, "dk", dt, k.sizes(), dev);
    if (want_dw && wq) {
      dwq = tensor(g[2], "dwq");
      need(dwq, "dwq", ScalarType::Float, {s.D}, dev);
    }
    if (want_dw && wk) {
      dwk = tensor(g[3], "dwk");
      need(dwk, "dwk", ScalarType::Float, {s.D}, dev);
    }
  }
  if (dwq.defined() || dwk.defined()) {
    size_t bytes = 0;
    run(dev, "sf_gdn_qk_norm_rotary_bwd_workspace_size",
        [&] { return g_abi.qk_norm_rotary_bwd_workspace_size(&s, &bytes); });
    ws = workspace(given, bytes, q);
  }
  run(dev, "sf_gdn_qk_norm_rotary_bwd", [&] {
    return g_abi.qk_norm_rotary_bwd(&s, ptr(q), ptr(k), i32(pos), f32(freq), f32(wq), f32(wk),
                                    ptr(dyq), ptr(dyk), dq.data_ptr(), dk.data_ptr(),
                                    dwq.defined() ? (float*)dwq.data_ptr() : nullptr,
                                    dwk.defined() ? (float*)dwk.data_ptr() : nullptr,
                                    ws.defined() ? ws.data_ptr() : nullptr, bytes_of(ws), st);
  });
  written({&dq, &dk, &dwq, &dwk, &ws});
  return tuple({&dq, &dk, &dwq, &dwk, &ws});
}

// bind(fail, addresses of the entry points in the order of Entries)
PyObject* bind(const Args& a) {
  constexpr Py_ssize_t n = sizeof(Entries) / sizeof(void*);
  a.count(n + 1);
  void* p[n];
  for (Py_ssize_t i = 0; i < n; ++i) p[i] = a.stream((int)i + 1);
  memcpy(&g_abi, p, sizeof(p));
  Py_XDECREF(g_fail);
  g_fail = a[0];
  Py_INCREF(g_fail);
  Py_RETURN_NONE;
}

#define CALL(f) {#f, (PyCFunction)(void (*)(void))entry<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(bind),           CALL(recurrent_step),    CALL(shortconv_step),
                         CALL(gated_norm_fwd), CALL(gated_norm_bwd),    CALL(residual_norm_fwd),
                         CALL(residual_norm_bwd), CALL(decay_chunk_fwd), CALL(decay_chunk_bwd),
                         CALL(decay_step), CALL(qk_norm_rotary_fwd), CALL(qk_norm_rotary_bwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  // the digest of the header whose structs it passes; the library has its own
  if (m && PyModule_AddStringConstant(m, "INTERFACE", SF_GDN_INTERFACE) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
