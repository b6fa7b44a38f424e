// CPython binding of the block operators and the int8 ones (moe_block.h, moe_int8.h): checks the tensors of a
// call and passes their addresses on. A call of a few microseconds on the GPU costs
// more in Python attribute lookups (shape, type, layout, device, address of up to
// 13 tensors) than on the device, so the checks are made here; _block.py and _int8.py
// hold the entry points with their defaults and documentation.
//
// Every function takes its tensors (or None), its scalars and the stream (an
// integer, or None for the current stream of the tensors' GPU), and returns the
// moe_status, or -1 - d if GPU d has to be made current first. ValueError: a tensor
// of the wrong shape, type, layout or device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/moe_int8.h"

namespace {

// libmoe's entry points (set by init) and torch's current device and stream
decltype(&moe_grouped_mm) f_grouped_mm;
decltype(&moe_grouped_mm_backward) f_grouped_mm_backward;
decltype(&moe_linear) f_linear;
decltype(&moe_linear_backward) f_linear_backward;
decltype(&moe_block_norm) f_block_norm;
decltype(&moe_block_norm_backward) f_block_norm_backward;
decltype(&moe_combine_backward) f_combine_backward;
decltype(&moe_layer_norm) f_layer_norm;
decltype(&moe_layer_norm_backward) f_layer_norm_backward;
decltype(&moe_quant_rows) f_quant_rows;
decltype(&moe_linear_w8a8) f_linear_w8a8;
decltype(&moe_layer_w8a8) f_layer_w8a8;
PyObject* g_get_device = nullptr;   // () -> current device
PyObject* g_get_stream = nullptr;   // (device) -> current raw stream
bool g_has_gpu = false;

struct Refused {};   // a Python exception is set

[[noreturn]] void refuse(const std::string& text) {
  PyErr_SetString(PyExc_ValueError, text.c_str());
  throw Refused{};
}

std::string shape_text(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

using at::ScalarType;
constexpr ScalarType kBf = ScalarType::BFloat16, kHf = ScalarType::Half, kF32 = ScalarType::Float,
                     kI32 = ScalarType::Int, kI8 = ScalarType::Char;

int type_code(ScalarType t) {
  return t == kBf ? MOE_BF16 : t == kHf ? MOE_FP16 : t == kI8 ? MOE_INT8 : MOE_F32;
}

// The operands of one call: the tensors are borrowed from the argument array.
class Call {
 public:
  Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, const char* fn) : args_(args) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", fn, want, n);
      throw Refused{};
    }
  }
  // Operand i, or NULL for None; its layout and device are checked.
  const at::Tensor* tensor(int i, const char* name) {
    PyObject* o = args_[i];
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " is no tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    const int d = t.is_cuda() ? static_cast<int>(t.get_device()) : -1;
    if (d < 0 && !t.is_cpu()) refuse(std::string(name) + " is neither on a GPU nor on the CPU");
    if (device_ == kNone) device_ = d;
    else if (d != device_)
      refuse(std::string(name) + " is on another device than the operands before it");
    return &t;
  }
  const at::Tensor& need(int i, const char* name) {
    const at::Tensor* t = tensor(i, name);
    if (!t) refuse(std::string(name) + " is missing");
    return *t;
  }
  double number(int i) {
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
  }
  int32_t integer(int i, const char* name) {
    const long v = PyLong_AsLong(args_[i]);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
    return static_cast<int32_t>(v);
  }
  // The stream in argument i. False: another GPU has to be made current first
  // (`device()` names it).
  bool stream(int i, void** s) {
    PyObject* o = args_[i];
    if (device_ < 0 && g_has_gpu) refuse("tensors on the CPU; a GPU is needed");
    if (device_ >= 0) {
      PyObject* cur = PyObject_CallNoArgs(g_get_device);
      if (!cur) throw Refused{};
      const long c = PyLong_AsLong(cur);
      Py_DECREF(cur);
      if (c == -1 && PyErr_Occurred()) throw Refused{};
      if (c != device_) return false;
    }
    *s = nullptr;
    if (o == Py_None && device_ < 0) return true;
    PyObject* v = o;
    if (o == Py_None) {
      PyObject* d = PyLong_FromLong(device_);
      if (!d) throw Refused{};
      v = PyObject_CallOneArg(g_get_stream, d);
      Py_DECREF(d);
      if (!v) throw Refused{};
    } else {
      Py_INCREF(v);
    }
    *s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw Refused{};
    return true;
  }
  int device() const { return device_; }

 private:
  static constexpr int kNone = -2;
  PyObject* const* args_;
  int device_ = kNone;
};

void want(const at::Tensor* t, const char* name, std::initializer_list<int64_t> shape,
          std::initializer_list<ScalarType> types) {
  if (!t) return;
  if (!t->sizes().equals(c10::IntArrayRef(shape.begin(), shape.size())))
    refuse(std::string(name) + " has shape " + shape_text(t->sizes()) + ", the call needs " +
           shape_text(c10::IntArrayRef(shape.begin(), shape.size())));
  for (const ScalarType s : types)
    if (t->scalar_type() == s) return;
  std::string text =
      std::string(name) + " is " + c10::toString(t->scalar_type()) + ", the call needs";
  for (const ScalarType s : types) text += std::string(" ") + c10::toString(s);
  refuse(text);
}

// An empty tensor has no address and stands as a non-null one that nothing reads:
// NULL means that the operand is not there.
void* ptr(const at::Tensor* t) {
  if (!t) return nullptr;
  void* p = t->data_ptr();
  return p ? p : reinterpret_cast<void*>(16);
}
void* ptr(const at::Tensor& t) { return ptr(&t); }
size_t bytes(const at::Tensor* t) { return t ? t->nbytes() : 0; }

ScalarType half_of(const at::Tensor& t, const char* name) {
  const ScalarType s = t.scalar_type();
  if (s != kBf && s != kHf)
    refuse(std::string(name) + " is " + c10::toString(s) + "; bfloat16 or float16 is needed");
  return s;
}

int32_t dim32(int64_t v, const char* what) {
  if (v > INT32_MAX) refuse(std::string(what) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}

// x [*, K], w [E, N, K] or [N, K]
moe_mm_shape product_shape(const at::Tensor& x, const at::Tensor& w, bool grouped, int32_t act,
                           ScalarType t) {
  if (x.dim() != 2 || w.dim() != (grouped ? 3 : 2))
    refuse("x has shape " + shape_text(x.sizes()) + ", w " + shape_text(w.sizes()));
  const int64_t K = w.size(-1), N = w.size(-2);
  if (x.size(1) != K)
    refuse("x has " + std::to_string(x.size(1)) + " columns, w contracts " + std::to_string(K));
  if (w.scalar_type() != t) refuse("w is of another type than x");
  moe_mm_shape s = {};
  s.K = dim32(K, "K");
  s.N = dim32(N, "N");
  s.E = grouped ? dim32(w.size(0), "E") : 1;
  s.topk = 1;
  s.dtype = type_code(t);
  s.act = act;
  return s;
}
int64_t out_width(const moe_mm_shape& s) { return s.act == MOE_ACT_SWIGLU ? s.N / 2 : s.N; }

void gather_shape(moe_mm_shape& s, const at::Tensor& x, const at::Tensor& offsets,
                  const at::Tensor* slot, int32_t topk) {
  want(&offsets, "expert_offsets", {s.E + int64_t{1}}, {kI32});
  if (slot) {
    want(slot, "sorted_slot", {s.rows}, {kI32});
    s.x_rows = dim32(x.size(0), "x's rows");
    s.topk = topk;
  } else if (x.size(0) != s.rows) {
    refuse("x has " + std::to_string(x.size(0)) + " rows, the call needs " +
           std::to_string(s.rows));
  }
}

// r [T, H], weights of one half type
moe_layer_norm_shape layer_norm_shape(const at::Tensor& r, const at::Tensor* y, const at::Tensor& w,
                                      double eps) {
  if (r.dim() != 2)
    refuse("the residual stream has shape " + shape_text(r.sizes()) + "; [T, H] is needed");
  moe_layer_norm_shape s = {};
  s.T = dim32(r.size(0), "T");
  s.H = dim32(r.size(1), "H");
  s.dtype = type_code(half_of(w, "w"));
  s.r_dtype = type_code(r.scalar_type());
  s.y_dtype = y ? type_code(y->scalar_type()) : s.dtype;
  s.eps = static_cast<float>(eps);
  return s;
}

template <class F>
PyObject* guard(F f) {
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
// Calls an entry point without the interpreter's lock: a launch can wait for room in
// the queue, and the argument array keeps the tensors alive.
template <class F, class... A>
PyObject* run(F f, A... args) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f(args...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}
PyObject* other_device(const Call& c) { return PyLong_FromLong(-1 - c.device()); }

// x, w, expert_offsets, sorted_slot, z, y, topk, act, stream
PyObject* grouped_mm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 9, "grouped_mm");
    const at::Tensor &x = c.need(0, "x"), &w = c.need(1, "w"), &off = c.need(2, "expert_offsets");
    const at::Tensor *slot = c.tensor(3, "sorted_slot"), *z = c.tensor(4, "z");
    const at::Tensor& y = c.need(5, "y");
    const ScalarType t = half_of(x, "x");
    moe_mm_shape s = product_shape(x, w, true, c.integer(7, "act"), t);
    if (y.dim() != 2) refuse("y has shape " + shape_text(y.sizes()));
    s.rows = dim32(y.size(0), "rows");
    want(&y, "y", {s.rows, out_width(s)}, {t, kF32});
    want(z, "z", {s.rows, s.N}, {t});
    gather_shape(s, x, off, slot, c.integer(6, "topk"));
    void* st;
    if (!c.stream(8, &st)) return other_device(c);
    return run(f_grouped_mm, &s, ptr(x), ptr(w), static_cast<int32_t*>(ptr(off)),
               static_cast<int32_t*>(ptr(slot)), ptr(z), ptr(y), type_code(y.scalar_type()), st);
  });
}

// dy, x, w, z, expert_offsets, sorted_slot, dx, dw, ws, topk, act, stream
PyObject* grouped_mm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 12, "grouped_mm_backward");
    const at::Tensor &dy = c.need(0, "dy"), &x = c.need(1, "x"), &w = c.need(2, "w");
    const at::Tensor* z = c.tensor(3, "z");
    const at::Tensor& off = c.need(4, "expert_offsets");
    const at::Tensor *slot = c.tensor(5, "sorted_slot"), *dx = c.tensor(6, "dx"),
                     *dw = c.tensor(7, "dw"), *ws = c.tensor(8, "ws");
    const ScalarType t = half_of(x, "x");
    moe_mm_shape s = product_shape(x, w, true, c.integer(10, "act"), t);
    if (dy.dim() != 2) refuse("dy has shape " + shape_text(dy.sizes()));
    s.rows = dim32(dy.size(0), "rows");
    want(&dy, "dy", {s.rows, out_width(s)}, {t});
    want(z, "z", {s.rows, s.N}, {t});
    want(dx, "dx", {s.rows, s.K}, {t, kF32});
    want(dw, "dw", {s.E, s.N, s.K}, {t, kF32});
    gather_shape(s, x, off, slot, c.integer(9, "topk"));
    void* st;
    if (!c.stream(11, &st)) return other_device(c);
    return run(f_grouped_mm_backward, &s, ptr(dy), ptr(x), ptr(w), ptr(z),
               static_cast<int32_t*>(ptr(off)), static_cast<int32_t*>(ptr(slot)), ptr(dx),
               dx ? type_code(dx->scalar_type()) : s.dtype, ptr(dw),
               dw ? type_code(dw->scalar_type()) : s.dtype, ptr(ws), bytes(ws), st);
  });
}

// x, w, bias, residual, z, y, act, stream
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 8, "linear");
    const at::Tensor &x = c.need(0, "x"), &w = c.need(1, "w");
    const at::Tensor *bias = c.tensor(2, "bias"), *res = c.tensor(3, "residual"),
                     *z = c.tensor(4, "z");
    const at::Tensor& y = c.need(5, "y");
    const ScalarType t = half_of(x, "x");
    moe_mm_shape s = product_shape(x, w, false, c.integer(6, "act"), t);
    s.rows = dim32(x.size(0), "rows");
    want(bias, "bias", {s.N}, {t});
    want(&y, "y", {s.rows, out_width(s)}, {t, kF32});
    want(res, "residual", {s.rows, out_width(s)}, {y.scalar_type()});
    want(z, "z", {s.rows, s.N}, {t});
    void* st;
    if (!c.stream(7, &st)) return other_device(c);
    return run(f_linear, &s, ptr(x), ptr(w), ptr(bias), ptr(res), ptr(z), ptr(y),
               type_code(y.scalar_type()), st);
  });
}

// dy, x, w, z, dx, dw, dbias, ws, act, stream
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 10, "linear_backward");
    const at::Tensor &dy = c.need(0, "dy"), &x = c.need(1, "x"), &w = c.need(2, "w");
    const at::Tensor *z = c.tensor(3, "z"), *dx = c.tensor(4, "dx"), *dw = c.tensor(5, "dw"),
                     *db = c.tensor(6, "dbias"), *ws = c.tensor(7, "ws");
    const ScalarType t = half_of(x, "x");
    moe_mm_shape s = product_shape(x, w, false, c.integer(8, "act"), t);
    s.rows = dim32(x.size(0), "rows");
    want(&dy, "dy", {s.rows, out_width(s)}, {t, kF32});
    want(z, "z", {s.rows, s.N}, {t});
    want(dx, "dx", {s.rows, s.K}, {t, kF32});
    want(dw, "dw", {s.N, s.K}, {t, kF32});
    if (dw) want(db, "dbias", {s.N}, {dw->scalar_type()});
    else want(db, "dbias", {s.N}, {t, kF32});
    const at::Tensor* grad = dw ? dw : db;
    void* st;
    if (!c.stream(9, &st)) return other_device(c);
    return run(f_linear_backward, &s, ptr(dy), type_code(dy.scalar_type()), ptr(x), ptr(w), ptr(z),
               ptr(dx), dx ? type_code(dx->scalar_type()) : s.dtype, ptr(dw), ptr(db),
               grad ? type_code(grad->scalar_type()) : s.dtype, ptr(ws), bytes(ws), st);
  });
}

// T, H, the half type of a norm's weights, gate and h (the first of `order` that
// has one; bfloat16 if all are float32), the gate's kind by its shape: [H] channel,
// [T, 1] token, [T, H] element.
moe_norm_shape norm_shape(const at::Tensor& r, const at::Tensor* y, const at::Tensor* gate,
                          std::initializer_list<const at::Tensor*> order, double scale, double eps,
                          ScalarType* half) {
  if (r.dim() != 2)
    refuse("the residual stream has shape " + shape_text(r.sizes()) + "; [T, H] is needed");
  moe_norm_shape s = {};
  s.T = dim32(r.size(0), "T");
  s.H = dim32(r.size(1), "H");
  *half = kBf;
  for (const at::Tensor* t : order) {
    if (!t || t->scalar_type() == kF32) continue;
    *half = half_of(*t, "an operand");
    break;
  }
  if (gate) {
    const auto g = gate->sizes();
    if (g.size() == 1 && g[0] == s.H) s.gate = MOE_GATE_CHANNEL;
    else if (g.size() == 2 && g[0] == s.T && g[1] == 1) s.gate = MOE_GATE_TOKEN;
    else if (g.size() == 2 && g[0] == s.T && g[1] == s.H) s.gate = MOE_GATE_ELEMENT;
    else
      refuse("gate has shape " + shape_text(g) + "; (" + std::to_string(s.H) + ",), (" +
             std::to_string(s.T) + ", 1) or (" + std::to_string(s.T) + ", " + std::to_string(s.H) +
             ") is needed");
    if (gate->scalar_type() != *half) refuse("gate is of another type than the weights");
  }
  s.dtype = type_code(*half);
  s.r_dtype = type_code(r.scalar_type());
  s.y_dtype = y ? type_code(y->scalar_type()) : s.dtype;
  s.scale = static_cast<float>(scale);
  s.eps = static_cast<float>(eps);
  return s;
}

// r, y, w_post, gate, w_pre, r_out, h, scale, eps, stream
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 10, "block_norm");
    const at::Tensor& r = c.need(0, "r");
    const at::Tensor *y = c.tensor(1, "y"), *wp = c.tensor(2, "w_post"), *g = c.tensor(3, "gate"),
                     *wn = c.tensor(4, "w_pre"), *ro = c.tensor(5, "r_out"), *h = c.tensor(6, "h");
    ScalarType t;
    const moe_norm_shape s = norm_shape(r, y, g, {wp, wn, g, h, &r, y}, c.number(7),
                                        c.number(8), &t);
    want(&r, "r", {s.T, s.H}, {t, kF32});
    want(y, "y", {s.T, s.H}, {t, kF32});
    want(ro, "r_out", {s.T, s.H}, {r.scalar_type()});
    want(h, "h", {s.T, s.H}, {t});
    want(wp, "w_post", {s.H}, {t});
    want(wn, "w_pre", {s.H}, {t});
    void* st;
    if (!c.stream(9, &st)) return other_device(c);
    return run(f_block_norm, &s, ptr(r), ptr(y), ptr(wp), ptr(g), ptr(wn), ptr(ro),
               ptr(h), st);
  });
}

// r_out, dr_out, dh, y, w_post, gate, w_pre, dr, dy, dw_post, dw_pre, dgate, ws,
// scale, eps, stream
PyObject* block_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 16, "block_norm_backward");
    const at::Tensor& r = c.need(0, "r_out");
    const at::Tensor *dro = c.tensor(1, "dr_out"), *dh = c.tensor(2, "dh"), *y = c.tensor(3, "y"),
                     *wp = c.tensor(4, "w_post"), *g = c.tensor(5, "gate"),
                     *wn = c.tensor(6, "w_pre");
    const at::Tensor& dr = c.need(7, "dr");
    const at::Tensor *dy = c.tensor(8, "dy"), *dwp = c.tensor(9, "dw_post"),
                     *dwn = c.tensor(10, "dw_pre"), *dg = c.tensor(11, "dgate"),
                     *ws = c.tensor(12, "ws");
    ScalarType t;
    const moe_norm_shape s = norm_shape(r, y, g, {wp, wn, g, dh, &r, y}, c.number(13),
                                        c.number(14), &t);
    want(&r, "r_out", {s.T, s.H}, {t, kF32});
    want(dro, "dr_out", {s.T, s.H}, {r.scalar_type()});
    want(dh, "dh", {s.T, s.H}, {t});
    want(y, "y", {s.T, s.H}, {t, kF32});
    want(wp, "w_post", {s.H}, {t});
    want(wn, "w_pre", {s.H}, {t});
    want(&dr, "dr", {s.T, s.H}, {r.scalar_type()});
    if (y) want(dy, "dy", {s.T, s.H}, {y->scalar_type()});
    want(dwp, "dw_post", {s.H}, {kF32});
    want(dwn, "dw_pre", {s.H}, {kF32});
    if (g && dg) {
      if (!dg->sizes().equals(g->sizes())) refuse("dgate has another shape than gate");
      if (dg->scalar_type() != (s.gate == MOE_GATE_ELEMENT ? t : kF32))
        refuse("dgate is float32 for a channel or token gate, of gate's type for an element gate");
    }
    void* st;
    if (!c.stream(15, &st)) return other_device(c);
    return run(f_block_norm_backward, &s, ptr(r), ptr(dro), ptr(dh), ptr(y), ptr(wp), ptr(g),
               ptr(wn), ptr(dr), ptr(dy), static_cast<float*>(ptr(dwp)),
               static_cast<float*>(ptr(dwn)), ptr(dg), ptr(ws), bytes(ws), st);
  });
}

// dout, y, slot_pos, topk_ids, topk_w, dy, dtopk_w, dlogits, stream
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 9, "combine_backward");
    const at::Tensor& dout = c.need(0, "dout");
    const at::Tensor* y = c.tensor(1, "y");
    const at::Tensor& pos = c.need(2, "slot_pos");
    const at::Tensor* ids = c.tensor(3, "topk_ids");
    const at::Tensor& w = c.need(4, "topk_w");
    const at::Tensor *dy = c.tensor(5, "dy"), *dw = c.tensor(6, "dtopk_w"),
                     *dl = c.tensor(7, "dlogits");
    if (w.dim() != 2 || dout.dim() != 2)
      refuse("topk_w has shape " + shape_text(w.sizes()) + ", dout " + shape_text(dout.sizes()));
    const int64_t T = w.size(0), k = w.size(1), H = dout.size(1);
    want(&dout, "dout", {T, H}, {kF32});
    want(y, "y", {T * k, H}, {kF32});
    want(&w, "topk_w", {T, k}, {kF32});
    if (pos.numel() != T * k || pos.scalar_type() != kI32)
      refuse("slot_pos holds " + std::to_string(pos.numel()) + " values, the call needs " +
             std::to_string(T * k) + " of int32");
    want(ids, "topk_ids", {T, k}, {kI32});
    want(dy, "dy", {T * k, H}, {kBf, kHf, kF32});
    want(dw, "dtopk_w", {T, k}, {kF32});
    int64_t E = k;
    if (dl) {
      if (dl->dim() != 2) refuse("dlogits has shape " + shape_text(dl->sizes()));
      E = dl->size(1);
      want(dl, "dlogits", {T, E}, {kF32});
    }
    void* st;
    if (!c.stream(8, &st)) return other_device(c);
    return run(f_combine_backward, static_cast<float*>(ptr(dout)), static_cast<float*>(ptr(y)),
               static_cast<int32_t*>(ptr(pos)), static_cast<int32_t*>(ptr(ids)),
               static_cast<float*>(ptr(w)), dim32(T, "T"), dim32(H, "H"), dim32(E, "E"),
               dim32(k, "k"), ptr(dy), dy ? type_code(dy->scalar_type()) : MOE_F32,
               static_cast<float*>(ptr(dw)), static_cast<float*>(ptr(dl)), st);
  });
}

// r, y, w, b, r_out, h, eps, stream
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 8, "layer_norm");
    const at::Tensor& r = c.need(0, "r");
    const at::Tensor* y = c.tensor(1, "y");
    const at::Tensor& w = c.need(2, "w");
    const at::Tensor *b = c.tensor(3, "b"), *ro = c.tensor(4, "r_out");
    const at::Tensor& h = c.need(5, "h");
    const moe_layer_norm_shape s = layer_norm_shape(r, y, w, c.number(6));
    const ScalarType t = w.scalar_type();
    want(&r, "r", {s.T, s.H}, {t, kF32});
    want(y, "y", {s.T, s.H}, {t, kF32});
    want(&w, "w", {s.H}, {t});
    want(b, "b", {s.H}, {t});
    want(ro, "r_out", {s.T, s.H}, {r.scalar_type()});
    want(&h, "h", {s.T, s.H}, {t});
    void* st;
    if (!c.stream(7, &st)) return other_device(c);
    return run(f_layer_norm, &s, ptr(r), ptr(y), ptr(w), ptr(b), ptr(ro), ptr(h), st);
  });
}

// r_out, dr_out, dh, w, dr, dw, db, ws, eps, stream
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 10, "layer_norm_backward");
    const at::Tensor& r = c.need(0, "r_out");
    const at::Tensor* dro = c.tensor(1, "dr_out");
    const at::Tensor &dh = c.need(2, "dh"), &w = c.need(3, "w"), &dr = c.need(4, "dr");
    const at::Tensor *dw = c.tensor(5, "dw"), *db = c.tensor(6, "db"), *ws = c.tensor(7, "ws");
    const moe_layer_norm_shape s = layer_norm_shape(r, nullptr, w, c.number(8));
    const ScalarType t = w.scalar_type();
    want(&r, "r_out", {s.T, s.H}, {t, kF32});
    want(dro, "dr_out", {s.T, s.H}, {r.scalar_type()});
    want(&dh, "dh", {s.T, s.H}, {t});
    want(&w, "w", {s.H}, {t});
    want(&dr, "dr", {s.T, s.H}, {r.scalar_type()});
    want(dw, "dw", {s.H}, {kF32});
    want(db, "db", {s.H}, {kF32});
    void* st;
    if (!c.stream(9, &st)) return other_device(c);
    return run(f_layer_norm_backward, &s, ptr(r), ptr(dro), ptr(dh), ptr(w), ptr(dr),
               static_cast<float*>(ptr(dw)), static_cast<float*>(ptr(db)), ptr(ws), bytes(ws), st);
  });
}

// x, q, scale, stream
PyObject* quant_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 4, "quant_rows");
    const at::Tensor &x = c.need(0, "x"), &q = c.need(1, "q"), &s = c.need(2, "scale");
    if (x.dim() != 2) refuse("x has shape " + shape_text(x.sizes()) + "; [rows, K] is needed");
    const int64_t rows = x.size(0), K = x.size(1);
    want(&x, "x", {rows, K}, {kBf, kHf, kF32});
    want(&q, "q", {rows, K}, {kI8});
    want(&s, "scale", {rows}, {kF32});
    void* st;
    if (!c.stream(3, &st)) return other_device(c);
    return run(f_quant_rows, ptr(x), type_code(x.scalar_type()), dim32(rows, "rows"),
               dim32(K, "K"), static_cast<int8_t*>(ptr(q)), static_cast<float*>(ptr(s)), st);
  });
}

// x, x_scale, w, w_scale, bias, residual, y, ws, act, stream
PyObject* linear_w8a8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 10, "linear_w8a8");
    const at::Tensor& x = c.need(0, "x");
    const at::Tensor* xs = c.tensor(1, "x_scale");
    const at::Tensor &w = c.need(2, "w"), &u = c.need(3, "w_scale");
    const at::Tensor *bias = c.tensor(4, "bias"), *res = c.tensor(5, "residual");
    const at::Tensor& y = c.need(6, "y");
    const at::Tensor* ws = c.tensor(7, "ws");
    if (x.dim() != 2 || w.dim() != 2)
      refuse("x has shape " + shape_text(x.sizes()) + ", w " + shape_text(w.sizes()));
    moe_w8_shape s = {};
    s.rows = dim32(x.size(0), "rows");
    s.K = dim32(x.size(1), "K");
    s.N = dim32(w.size(0), "N");
    s.act = c.integer(8, "act");
    s.x_dtype = type_code(x.scalar_type());
    s.y_dtype = type_code(y.scalar_type());
    want(&x, "x", {s.rows, s.K}, {kI8, kBf, kHf});
    want(&w, "w", {s.N, s.K}, {kI8});
    want(xs, "x_scale", {s.rows}, {kF32});
    if ((s.x_dtype == MOE_INT8) != (xs != nullptr))
      refuse("x_scale goes with int8 codes in x, and they with it");
    want(&u, "w_scale", {s.N}, {kF32});
    want(bias, "bias", {s.N}, {kF32});
    want(&y, "y", {s.rows, s.act == MOE_ACT_SWIGLU ? s.N / 2 : s.N}, {kBf, kHf, kF32});
    want(res, "residual", {y.size(0), y.size(1)}, {y.scalar_type()});
    void* st;
    if (!c.stream(9, &st)) return other_device(c);
    return run(f_linear_w8a8, &s, ptr(x), static_cast<float*>(ptr(xs)), static_cast<int8_t*>(ptr(w)),
               static_cast<float*>(ptr(u)), static_cast<float*>(ptr(bias)), ptr(res), ptr(y), ptr(ws),
               bytes(ws), st);
  });
}

// logits, x, w13, s13, w2, s2, residual, topk_ids, topk_w, expert_offsets, out, ws, stream
PyObject* layer_w8a8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guard([&]() -> PyObject* {
    Call c(a, n, 13, "layer_w8a8");
    const at::Tensor &L = c.need(0, "logits"), &x = c.need(1, "x"), &w13 = c.need(2, "w13"),
                     &s13 = c.need(3, "s13"), &w2 = c.need(4, "w2"), &s2 = c.need(5, "s2");
    const at::Tensor* res = c.tensor(6, "residual");
    const at::Tensor &ids = c.need(7, "topk_ids"), &w = c.need(8, "topk_w");
    const at::Tensor* off = c.tensor(9, "expert_offsets");
    const at::Tensor &out = c.need(10, "out"), &ws = c.need(11, "ws");
    if (x.dim() != 2 || w13.dim() != 3 || w2.dim() != 3 || ids.dim() != 2)
      refuse("x has shape " + shape_text(x.sizes()) + ", w13 " + shape_text(w13.sizes()) + ", w2 " +
             shape_text(w2.sizes()) + ", topk_ids " + shape_text(ids.sizes()));
    moe_shape s = {};
    s.T = dim32(x.size(0), "T");
    s.H = dim32(x.size(1), "H");
    s.I = dim32(w2.size(2), "I");
    s.E = dim32(w2.size(0), "E");
    s.k = dim32(ids.size(1), "k");
    const int64_t I2 = 2 * static_cast<int64_t>(s.I);
    want(&L, "logits", {s.T, s.E}, {kF32});
    want(&x, "x", {s.T, s.H}, {kBf, kHf});
    want(&w13, "w13", {s.E, I2, s.H}, {kI8});
    want(&s13, "s13", {s.E, I2}, {kF32});
    want(&w2, "w2", {s.E, s.H, s.I}, {kI8});
    want(&s2, "s2", {s.E, s.H}, {kF32});
    want(&ids, "topk_ids", {s.T, s.k}, {kI32});
    want(&w, "topk_w", {s.T, s.k}, {kF32});
    want(off, "expert_offsets", {s.E + int64_t{1}}, {kI32});
    want(&out, "out", {s.T, s.H}, {kBf, kHf, kF32});
    want(res, "residual", {s.T, s.H}, {out.scalar_type()});
    void* st;
    if (!c.stream(12, &st)) return other_device(c);
    return run(f_layer_w8a8, &s, static_cast<float*>(ptr(L)), ptr(x), type_code(x.scalar_type()),
               static_cast<int8_t*>(ptr(w13)), static_cast<float*>(ptr(s13)),
               static_cast<int8_t*>(ptr(w2)), static_cast<float*>(ptr(s2)), ptr(res),
               static_cast<int32_t*>(ptr(ids)), static_cast<float*>(ptr(w)),
               static_cast<int32_t*>(ptr(off)), ptr(out), type_code(out.scalar_type()), ptr(ws),
               bytes(&ws), st);
  });
}

// init(addresses of the entry points in the order of `entry`, get_device, get_stream,
// has_gpu)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** const entry[] = {reinterpret_cast<void**>(&f_grouped_mm),
                          reinterpret_cast<void**>(&f_grouped_mm_backward),
                          reinterpret_cast<void**>(&f_linear),
                          reinterpret_cast<void**>(&f_linear_backward),
                          reinterpret_cast<void**>(&f_block_norm),
                          reinterpret_cast<void**>(&f_block_norm_backward),
                          reinterpret_cast<void**>(&f_combine_backward),
                          reinterpret_cast<void**>(&f_layer_norm),
                          reinterpret_cast<void**>(&f_layer_norm_backward),
                          reinterpret_cast<void**>(&f_quant_rows),
                          reinterpret_cast<void**>(&f_linear_w8a8),
                          reinterpret_cast<void**>(&f_layer_w8a8)};
  constexpr Py_ssize_t kEntries = sizeof(entry) / sizeof(entry[0]);
  if (n != kEntries + 3) {
    PyErr_Format(PyExc_TypeError, "init takes %zd arguments", kEntries + 3);
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    *entry[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  a += kEntries;
  Py_XINCREF(a[0]);
  Py_XINCREF(a[1]);
  g_get_device = a[0];
  g_get_stream = a[1];
  g_has_gpu = PyObject_IsTrue(a[2]) == 1;
  Py_RETURN_NONE;
}

#define METHOD(f)                                                                          \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init),
                         METHOD(grouped_mm),
                         METHOD(grouped_mm_backward),
                         METHOD(linear),
                         METHOD(linear_backward),
                         METHOD(block_norm),
                         METHOD(block_norm_backward),
                         METHOD(combine_backward),
                         METHOD(layer_norm),
                         METHOD(layer_norm_backward),
                         METHOD(quant_rows),
                         METHOD(linear_w8a8),
                         METHOD(layer_w8a8),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_binding() { return PyModule_Create(&module); }
