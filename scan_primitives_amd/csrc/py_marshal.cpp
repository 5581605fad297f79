// py_marshal.cpp: the short way from Python to the linear-attention and state-space
// entry points of libsx_scan.so, for calls whose time is that of getting to the GPU.
//
// Each function takes what the binding's function of the same name takes, in
// order. Where every tensor is a plain one on the current device, of the expected
// type and shape, without a tangent or a lazy sign, and autograd does not record, it allocates
// the results, calls the C entry on the current stream and returns them (or the
// entry's status where that is not zero). Anything else returns None: the binding then goes the long
// way, which converts, records, switches devices and names what is wrong. The two
// ways pass the same arguments to the same entries.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sx_scan.h"

namespace {

// Set once by bind(): the library's entries and torch's own callables.
struct Entries {
  decltype(&sx_decay_attention) decay_attention;
  decltype(&sx_decay_attention_workspace_bytes) decay_attention_bytes;
  decltype(&sx_decay_attention_backward) decay_attention_backward;
  decltype(&sx_decay_attention_backward_workspace_bytes) decay_attention_backward_bytes;
  decltype(&sx_decay_attention_step) decay_attention_step;
  decltype(&sx_head_norm_rotate) head_norm_rotate;
  decltype(&sx_head_norm_rotate_backward) head_norm_rotate_backward;
  decltype(&sx_head_norm_rotate_backward_workspace_bytes) head_norm_rotate_backward_bytes;
  decltype(&sx_causal_conv) causal_conv;
  decltype(&sx_causal_conv_backward) causal_conv_backward;
  decltype(&sx_causal_conv_backward_workspace_bytes) causal_conv_backward_bytes;
  decltype(&sx_causal_conv_step) causal_conv_step;
  decltype(&sx_selective_scan) selective_scan;
  decltype(&sx_selective_scan_workspace_bytes) selective_scan_bytes;
  decltype(&sx_selective_scan_backward) selective_scan_backward;
  decltype(&sx_selective_scan_backward_workspace_bytes) selective_scan_backward_bytes;
  decltype(&sx_selective_scan_step) selective_scan_step;
  decltype(&sx_group_norm) group_norm;
  decltype(&sx_group_norm_workspace_bytes) group_norm_bytes;
  decltype(&sx_group_norm_backward) group_norm_backward;
  decltype(&sx_group_norm_backward_workspace_bytes) group_norm_backward_bytes;
} lib;
constexpr int kEntries = 21;
PyObject* current_device = nullptr;
PyObject* raw_stream = nullptr;

// The operands of one call; `fit` turns false once one of them has to go the long way.
struct Call {
  bool fit = true;
  int index = -1;
  const bool records = c10::GradMode::is_enabled();

  const at::Tensor* take(PyObject* o) {
    if (!fit || !THPVariable_CheckExact(o)) return fit = false, nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || (records && t.requires_grad()) || t._fw_grad(0).defined() || t.is_neg() ||
        (index >= 0 && t.get_device() != index))
      return fit = false, nullptr;
    index = int(t.get_device());
    return &t;
  }
  const at::Tensor* take(PyObject* o, at::ScalarType type, int64_t dim) {
    const at::Tensor* t = take(o);
    if (t && (t->scalar_type() != type || t->dim() != dim)) return fit = false, nullptr;
    return t;
  }
  // None, or a contiguous tensor of a type and shape
  const void* optional(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    if (!fit || o == Py_None) return nullptr;
    const at::Tensor* t = take(o);
    if (!t || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous()) return fit = false, nullptr;
    return t->data_ptr();
  }
  double number(PyObject* o) {
    if (PyFloat_CheckExact(o)) return PyFloat_AS_DOUBLE(o);
    fit = false;
    return 0.0;
  }
  bool here() {
    if (!fit) return false;
    PyObject* now = PyObject_CallNoArgs(current_device);
    fit = now && PyLong_AsLong(now) == index;
    Py_XDECREF(now);
    if (PyErr_Occurred()) PyErr_Clear();
    return fit;
  }
  void* stream() {
    PyObject* i = PyLong_FromLong(index);
    PyObject* s = PyObject_CallOneArg(raw_stream, i);
    Py_DECREF(i);
    void* p = s ? PyLong_AsVoidPtr(s) : nullptr;
    Py_XDECREF(s);
    return p;
  }
};

bool float_type(const at::Tensor& t, sx_dtype* code) {
  if (t.scalar_type() == at::kFloat) return *code = SX_F32, true;
  if (t.scalar_type() == at::kBFloat16) return *code = SX_BF16, true;
  return false;
}

at::Tensor workspace(size_t bytes, const at::Tensor& like) {
  return bytes ? at::empty({int64_t(bytes)}, like.options().dtype(at::kByte)) : at::Tensor();
}
void* data(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject* the_long_way() { Py_RETURN_NONE; }

// A status, or the tuple of results (an undefined tensor is None).
template <typename... T>
PyObject* answer(sx_status st, const T&... results) {
  if (st != SX_OK) return PyLong_FromLong(long(st));
  PyObject* tuple = PyTuple_New(sizeof...(T));
  Py_ssize_t i = 0;
  for (const at::Tensor* t : {&results...}) {
    PyObject* o = t->defined() ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(tuple, i++, o);
  }
  return tuple;
}

// No C++ exception crosses into Python: what fails here (memory, say) fails again the long way, with its message.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const std::exception&) {
    return the_long_way();
  }
}

struct DecayArgs {
  const at::Tensor *q, *k, *v, *g;
  sx_dtype code;
  int64_t heads;
};

bool decay_args(Call& c, PyObject* const* a, int64_t rank, DecayArgs* d) {
  d->q = c.take(a[0]);
  if (!c.fit || d->q->dim() != rank || !float_type(*d->q, &d->code)) return false;
  d->k = c.take(a[1], d->q->scalar_type(), rank);
  d->v = c.take(a[2], d->q->scalar_type(), rank);
  d->g = c.take(a[3]);
  if (!c.fit || d->g->scalar_type() != at::kFloat || (d->g->dim() != 1 && d->g->dim() != rank - 1)) return false;
  d->heads = d->g->size(-1);
  return true;
}

// (q, k, v, log_decay, initial, lengths, scale, return_state)
PyObject* decay_attention(PyObject* const* a, Py_ssize_t n) {
  Call c;
  DecayArgs d;
  if (n != 8 || (a[7] != Py_True && a[7] != Py_False) || !decay_args(c, a, 4, &d)) return the_long_way();
  const int64_t b = d.q->size(0), t = d.q->size(1), dk = d.q->size(3), dv = d.v->size(3);
  const void* initial = c.optional(a[4], at::kFloat, {b, d.heads, dk, dv});
  const void* lengths = c.optional(a[5], at::kInt, {b});
  const double scale = c.number(a[6]);
  if (!c.here()) return the_long_way();
  const at::Tensor out = at::empty({b, t, d.heads, dv}, d.q->options());
  const at::Tensor state = a[7] == Py_True ? at::empty({b, d.heads, dk, dv}, d.g->options()) : at::Tensor();
  const size_t bytes = lib.decay_attention_bytes(d.code, d.q->sizes().data(), d.v->sizes().data(), d.heads);
  const at::Tensor ws = workspace(bytes, *d.q);
  return answer(lib.decay_attention(d.code, d.q->sizes().data(), d.q->strides().data(), d.q->data_ptr(),
                                    d.k->sizes().data(), d.k->strides().data(), d.k->data_ptr(), d.v->sizes().data(),
                                    d.v->strides().data(), d.v->data_ptr(), int(d.g->dim()), d.g->sizes().data(),
                                    d.g->strides().data(), static_cast<const float*>(d.g->data_ptr()),
                                    static_cast<const float*>(initial), static_cast<const int32_t*>(lengths),
                                    float(scale), out.data_ptr(), static_cast<float*>(data(state)), data(ws), bytes,
                                    c.stream()),
                out, state);
}

// (q, k, v, log_decay, grad_out, initial, lengths, scale, grad_state)
PyObject* decay_attention_backward(PyObject* const* a, Py_ssize_t n) {
  Call c;
  DecayArgs d;
  if (n != 9 || !decay_args(c, a, 4, &d)) return the_long_way();
  const int64_t b = d.q->size(0), t = d.q->size(1), dk = d.q->size(3), dv = d.v->size(3);
  const at::Tensor* go = c.take(a[4], d.q->scalar_type(), 4);
  const void* initial = c.optional(a[5], at::kFloat, {b, d.heads, dk, dv});
  const void* lengths = c.optional(a[6], at::kInt, {b});
  const double scale = c.number(a[7]);
  const void* gs = c.optional(a[8], at::kFloat, {b, d.heads, dk, dv});
  if (!c.here() || go->sizes() != at::IntArrayRef({b, t, d.heads, dv})) return the_long_way();
  const at::Tensor gq = at::empty(d.q->sizes(), d.q->options()), gk = at::empty(d.k->sizes(), d.q->options()),
                   gv = at::empty(d.v->sizes(), d.q->options()), gg = at::empty(d.g->sizes(), d.g->options()),
                   gi = at::empty({b, d.heads, dk, dv}, d.g->options());
  const size_t bytes = lib.decay_attention_backward_bytes(d.code, d.q->sizes().data(), d.k->sizes().data(),
                                                          d.v->sizes().data(), d.heads);
  const at::Tensor ws = workspace(bytes, *d.q);
  return answer(
      lib.decay_attention_backward(
          d.code, d.q->sizes().data(), d.q->strides().data(), d.q->data_ptr(), d.k->sizes().data(),
          d.k->strides().data(), d.k->data_ptr(), d.v->sizes().data(), d.v->strides().data(), d.v->data_ptr(),
          int(d.g->dim()), d.g->sizes().data(), d.g->strides().data(), static_cast<const float*>(d.g->data_ptr()),
          go->strides().data(), go->data_ptr(), static_cast<const float*>(gs), static_cast<const float*>(initial),
          static_cast<const int32_t*>(lengths), float(scale), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
          static_cast<float*>(gg.data_ptr()), static_cast<float*>(gi.data_ptr()), data(ws), bytes, c.stream()),
      gq, gk, gv, gg, gi);
}

// (q, k, v, log_decay, state, slots, scale)
PyObject* decay_attention_step(PyObject* const* a, Py_ssize_t n) {
  Call c;
  DecayArgs d;
  if (n != 7 || !decay_args(c, a, 3, &d)) return the_long_way();
  const int64_t b = d.q->size(0), dk = d.q->size(2), dv = d.v->size(2);
  const at::Tensor* state = c.take(a[4], at::kFloat, 4);
  const void* slots = c.optional(a[5], at::kInt, {b});
  const double scale = c.number(a[6]);
  if (!c.here() || state->size(1) != d.heads || state->size(2) != dk || state->size(3) != dv) return the_long_way();
  const at::Tensor out = at::empty({b, d.heads, dv}, d.q->options());
  const sx_status st = lib.decay_attention_step(
      d.code, d.q->sizes().data(), d.q->strides().data(), d.q->data_ptr(), d.k->sizes().data(), d.k->strides().data(),
      d.k->data_ptr(), d.v->sizes().data(), d.v->strides().data(), d.v->data_ptr(), int(d.g->dim()),
      d.g->sizes().data(), d.g->strides().data(), static_cast<const float*>(d.g->data_ptr()), state->size(0),
      state->strides().data(), static_cast<float*>(state->data_ptr()), static_cast<const int32_t*>(slots),
      float(scale), out.data_ptr(), c.stream());
  // autograd tells by the version that a state it saved has been written to (a state of inference mode has none)
  if (st == SX_OK && !state->is_inference()) state->unsafeGetTensorImpl()->bump_version();
  return answer(st, out);
}

struct RotateArgs {
  const at::Tensor *q, *k, *positions, *turns;
  const float *qw, *kw;
  int64_t position_strides[2];
  sx_dtype code;
  double eps;
  int neighbours;
};

// q, k, positions, turns at a[0 ..], the rest from a[rest]: q_weight, k_weight, eps, neighbours
bool rotate_args(Call& c, PyObject* const* a, int rest, RotateArgs* r) {
  r->q = c.take(a[0]);
  if (!c.fit || r->q->dim() != 4 || !float_type(*r->q, &r->code)) return false;
  r->k = c.take(a[1], r->q->scalar_type(), 4);
  r->positions = c.take(a[2]);
  r->turns = c.take(a[3], at::kDouble, 1);
  const int64_t b = r->q->size(0), t = r->q->size(1), d = r->q->size(3);
  r->qw = static_cast<const float*>(c.optional(a[rest], at::kFloat, {d}));
  r->kw = static_cast<const float*>(c.optional(a[rest + 1], at::kFloat, {d}));
  r->eps = c.number(a[rest + 2]);
  r->neighbours = a[rest + 3] == Py_True;
  if (!c.fit || !r->turns->is_contiguous() || (a[rest + 3] != Py_True && a[rest + 3] != Py_False)) return false;
  if (r->positions->scalar_type() != at::kLong && r->positions->scalar_type() != at::kInt) return false;
  if (r->positions->sizes() == at::IntArrayRef({t})) {
    r->position_strides[0] = 0;
    r->position_strides[1] = r->positions->stride(0);
  } else if (r->positions->sizes() == at::IntArrayRef({b, t})) {
    r->position_strides[0] = r->positions->stride(0);
    r->position_strides[1] = r->positions->stride(1);
  } else {
    return false;
  }
  return true;
}

// (q, k, positions, turns, q_weight, k_weight, eps, neighbours)
PyObject* head_norm_rotate(PyObject* const* a, Py_ssize_t n) {
  Call c;
  RotateArgs r;
  if (n != 8 || !rotate_args(c, a, 4, &r) || !c.here()) return the_long_way();
  const at::Tensor oq = at::empty(r.q->sizes(), r.q->options()), ok = at::empty(r.k->sizes(), r.q->options());
  return answer(lib.head_norm_rotate(r.code, r.q->sizes().data(), r.q->strides().data(), r.q->data_ptr(),
                                     r.k->sizes().data(), r.k->strides().data(), r.k->data_ptr(),
                                     r.positions->scalar_type() == at::kLong, r.position_strides,
                                     r.positions->data_ptr(), 2 * r.turns->size(0),
                                     static_cast<const double*>(r.turns->data_ptr()), r.qw, r.kw, float(r.eps),
                                     r.neighbours, oq.data_ptr(), ok.data_ptr(), c.stream()),
                oq, ok);
}

// (q, k, positions, turns, grad_out_q, grad_out_k, q_weight, k_weight, eps, neighbours)
PyObject* head_norm_rotate_backward(PyObject* const* a, Py_ssize_t n) {
  Call c;
  RotateArgs r;
  if (n != 10 || !rotate_args(c, a, 6, &r)) return the_long_way();
  const at::Tensor* gq = c.take(a[4], r.q->scalar_type(), 4);
  const at::Tensor* gk = c.take(a[5], r.q->scalar_type(), 4);
  if (!c.here() || gq->sizes() != r.q->sizes() || gk->sizes() != r.k->sizes()) return the_long_way();
  const auto f32 = r.q->options().dtype(at::kFloat);
  const int64_t d = r.q->size(3);
  const at::Tensor xq = at::empty(r.q->sizes(), r.q->options()), xk = at::empty(r.k->sizes(), r.q->options());
  const at::Tensor wq = r.qw ? at::empty({d}, f32) : at::Tensor(), wk = r.kw ? at::empty({d}, f32) : at::Tensor();
  const size_t bytes =
      r.qw || r.kw ? lib.head_norm_rotate_backward_bytes(r.q->sizes().data(), r.k->sizes().data()) : 0;
  const at::Tensor ws = workspace(bytes, *r.q);
  return answer(
      lib.head_norm_rotate_backward(r.code, r.q->sizes().data(), r.q->strides().data(), r.q->data_ptr(),
                                    r.k->sizes().data(), r.k->strides().data(), r.k->data_ptr(),
                                    r.positions->scalar_type() == at::kLong, r.position_strides,
                                    r.positions->data_ptr(), 2 * r.turns->size(0),
                                    static_cast<const double*>(r.turns->data_ptr()), gq->strides().data(),
                                    gq->data_ptr(), gk->strides().data(), gk->data_ptr(), r.qw, r.kw, float(r.eps),
                                    r.neighbours, xq.data_ptr(), xk.data_ptr(), static_cast<float*>(data(wq)),
                                    static_cast<float*>(data(wk)), data(ws), bytes, c.stream()),
      xq, xk, wq, wk);
}

struct ConvCall {
  const at::Tensor *x, *w;
  const float* bias;
  sx_dtype code;
  int64_t d, taps;
  sx_activation act;
};

// None or "silu"
bool activation(PyObject* o, sx_activation* act) {
  if (o == Py_None) return *act = SX_ACT_NONE, true;
  if (!PyUnicode_CheckExact(o) || PyUnicode_CompareWithASCIIString(o, "silu") != 0) return false;
  return *act = SX_ACT_SILU, true;
}

bool conv_args(Call& c, PyObject* x, PyObject* w, PyObject* bias, PyObject* act, int64_t rank, ConvCall* a) {
  a->x = c.take(x);
  if (!c.fit || a->x->dim() != rank || !float_type(*a->x, &a->code) || !activation(act, &a->act)) return false;
  a->d = a->x->size(-1);
  a->w = c.take(w, at::kFloat, 2);
  if (!c.fit || a->w->size(0) != a->d || !a->w->is_contiguous()) return false;
  a->taps = a->w->size(1);
  a->bias = static_cast<const float*>(c.optional(bias, at::kFloat, {a->d}));
  return c.fit && a->taps > 0;
}
const float* floats(const at::Tensor* t) { return static_cast<const float*>(t->data_ptr()); }

// (x, weight, bias, initial, lengths, activation, return_state)
PyObject* causal_conv(PyObject* const* a, Py_ssize_t n) {
  Call c;
  ConvCall v;
  if (n != 7 || (a[6] != Py_True && a[6] != Py_False) || !conv_args(c, a[0], a[1], a[2], a[5], 3, &v))
    return the_long_way();
  const int64_t b = v.x->size(0);
  const void* initial = c.optional(a[3], v.x->scalar_type(), {b, v.taps - 1, v.d});
  const void* lengths = c.optional(a[4], at::kInt, {b});
  if (!c.here()) return the_long_way();
  const at::Tensor out = at::empty(v.x->sizes(), v.x->options());
  const at::Tensor state = a[6] == Py_True ? at::empty({b, v.taps - 1, v.d}, v.x->options()) : at::Tensor();
  return answer(lib.causal_conv(v.code, v.x->sizes().data(), v.x->strides().data(), v.x->data_ptr(), v.taps,
                                floats(v.w), v.bias, initial, static_cast<const int32_t*>(lengths), v.act,
                                out.data_ptr(), data(state), c.stream()),
                out, state);
}

// (x, weight, grad_out, bias, initial, lengths, activation, grad_state)
PyObject* causal_conv_backward(PyObject* const* a, Py_ssize_t n) {
  Call c;
  ConvCall v;
  if (n != 8 || !conv_args(c, a[0], a[1], a[3], a[6], 3, &v)) return the_long_way();
  const int64_t b = v.x->size(0);
  const at::Tensor* go = c.take(a[2], v.x->scalar_type(), 3);
  const void* initial = c.optional(a[4], v.x->scalar_type(), {b, v.taps - 1, v.d});
  const void* lengths = c.optional(a[5], at::kInt, {b});
  const void* gs = c.optional(a[7], v.x->scalar_type(), {b, v.taps - 1, v.d});
  if (!c.here() || go->sizes() != v.x->sizes()) return the_long_way();
  const at::Tensor gx = at::empty(v.x->sizes(), v.x->options()), gw = at::empty(v.w->sizes(), v.w->options()),
                   gb = v.bias ? at::empty({v.d}, v.w->options()) : at::Tensor(),
                   gi = at::empty({b, v.taps - 1, v.d}, v.x->options());
  const size_t bytes = lib.causal_conv_backward_bytes(v.code, v.x->sizes().data(), v.taps);
  const at::Tensor ws = workspace(bytes, *v.x);
  return answer(lib.causal_conv_backward(v.code, v.x->sizes().data(), v.x->strides().data(), v.x->data_ptr(), v.taps,
                                         floats(v.w), v.bias, initial, static_cast<const int32_t*>(lengths), v.act,
                                         go->strides().data(), go->data_ptr(), gs, gx.data_ptr(),
                                         static_cast<float*>(gw.data_ptr()), static_cast<float*>(data(gb)),
                                         gi.data_ptr(), data(ws), bytes, c.stream()),
                gx, gw, gb, gi);
}

// A pool of contiguous states [pool, rows, cols].
const at::Tensor* pool_arg(Call& c, PyObject* o, at::ScalarType type, int64_t rows, int64_t cols) {
  const at::Tensor* t = c.take(o, type, 3);
  if (!t || t->size(1) != rows || t->size(2) != cols || (cols > 1 && t->stride(2) != 1) ||
      (rows > 1 && t->stride(1) != cols))
    return c.fit = false, nullptr;
  return t;
}
// autograd tells by the version that a state it saved has been written to (a state of inference mode has none)
void written(sx_status st, const at::Tensor* state) {
  if (st == SX_OK && !state->is_inference()) state->unsafeGetTensorImpl()->bump_version();
}

// (x, weight, state, bias, slots, activation)
PyObject* causal_conv_step(PyObject* const* a, Py_ssize_t n) {
  Call c;
  ConvCall v;
  if (n != 6 || !conv_args(c, a[0], a[1], a[3], a[5], 2, &v)) return the_long_way();
  const at::Tensor* state = pool_arg(c, a[2], v.x->scalar_type(), v.taps - 1, v.d);
  const void* slots = c.optional(a[4], at::kInt, {v.x->size(0)});
  if (!c.here()) return the_long_way();
  const at::Tensor out = at::empty(v.x->sizes(), v.x->options());
  const sx_status st = lib.causal_conv_step(v.code, v.x->sizes().data(), v.x->strides().data(), v.x->data_ptr(), v.taps,
                                            floats(v.w), v.bias, v.act, state->size(0), state->stride(0),
                                            state->data_ptr(), static_cast<const int32_t*>(slots), out.data_ptr(),
                                            c.stream());
  written(st, state);
  return answer(st, out);
}

struct ScanCall {
  const at::Tensor *x, *delta, *a, *b, *c, *z;
  const float *skip, *bias;
  sx_dtype code;
  int64_t d, n;
  int softplus;
};

// x, delta, a, b, c at o[0 ..], skip, z, delta_bias, softplus at r[0 ..]
bool scan_args(Call& c, PyObject* const* o, PyObject* const* r, int64_t rank, ScanCall* s) {
  s->x = c.take(o[0]);
  if (!c.fit || s->x->dim() != rank || !float_type(*s->x, &s->code) || (r[3] != Py_True && r[3] != Py_False))
    return false;
  const at::ScalarType type = s->x->scalar_type();
  s->delta = c.take(o[1], type, rank);
  s->a = c.take(o[2], at::kFloat, 2);
  s->b = c.take(o[3], type, rank + 1);
  s->c = c.take(o[4], type, rank + 1);
  s->z = r[1] == Py_None ? nullptr : c.take(r[1], type, rank);
  if (!c.fit) return false;
  s->d = s->x->size(-1);
  s->n = s->b->size(-1);
  if (s->delta->sizes() != s->x->sizes() || (s->z && s->z->sizes() != s->x->sizes()) ||
      s->c->sizes() != s->b->sizes() || s->a->size(0) != s->d || s->a->size(1) != s->n || !s->a->is_contiguous())
    return false;
  s->skip = static_cast<const float*>(c.optional(r[0], at::kFloat, {s->d}));
  s->bias = static_cast<const float*>(c.optional(r[2], at::kFloat, {s->d}));
  s->softplus = r[3] == Py_True;
  return c.fit;
}

// Calls an entry with the operands in their order, then what is left.
template <typename F, typename... T>
sx_status scan_call(F entry, const ScanCall& s, T... rest) {
  return entry(s.code, s.x->sizes().data(), s.x->strides().data(), s.x->data_ptr(), s.delta->strides().data(),
               s.delta->data_ptr(), floats(s.a), s.b->sizes().data(), s.b->strides().data(), s.b->data_ptr(),
               s.c->strides().data(), s.c->data_ptr(), s.skip, s.z ? s.z->strides().data() : nullptr,
               s.z ? s.z->data_ptr() : nullptr, s.bias, s.softplus, rest...);
}

// (x, delta, a, b, c, skip, z, delta_bias, softplus, initial, lengths, return_state)
PyObject* selective_scan(PyObject* const* a, Py_ssize_t n) {
  Call c;
  ScanCall s;
  if (n != 12 || (a[11] != Py_True && a[11] != Py_False) || !scan_args(c, a, a + 5, 3, &s)) return the_long_way();
  const int64_t b = s.x->size(0);
  const void* initial = c.optional(a[9], at::kFloat, {b, s.d, s.n});
  const void* lengths = c.optional(a[10], at::kInt, {b});
  if (!c.here()) return the_long_way();
  const at::Tensor out = at::empty(s.x->sizes(), s.x->options());
  const at::Tensor state = a[11] == Py_True ? at::empty({b, s.d, s.n}, s.a->options()) : at::Tensor();
  const size_t bytes = lib.selective_scan_bytes(s.code, s.x->sizes().data(), s.b->sizes().data());
  const at::Tensor ws = workspace(bytes, *s.x);
  return answer(scan_call(lib.selective_scan, s, static_cast<const float*>(initial),
                          static_cast<const int32_t*>(lengths), out.data_ptr(), static_cast<float*>(data(state)),
                          data(ws), bytes, c.stream()),
                out, state);
}

// (x, delta, a, b, c, grad_out, skip, z, delta_bias, softplus, initial, lengths, grad_state)
PyObject* selective_scan_backward(PyObject* const* a, Py_ssize_t n) {
  Call c;
  ScanCall s;
  if (n != 13 || !scan_args(c, a, a + 6, 3, &s)) return the_long_way();
  const int64_t b = s.x->size(0);
  const at::Tensor* go = c.take(a[5], s.x->scalar_type(), 3);
  const void* initial = c.optional(a[10], at::kFloat, {b, s.d, s.n});
  const void* lengths = c.optional(a[11], at::kInt, {b});
  const void* gs = c.optional(a[12], at::kFloat, {b, s.d, s.n});
  if (!c.here() || go->sizes() != s.x->sizes()) return the_long_way();
  const at::Tensor gx = at::empty(s.x->sizes(), s.x->options()), gd = at::empty(s.x->sizes(), s.x->options()),
                   ga = at::empty(s.a->sizes(), s.a->options()), gb = at::empty(s.b->sizes(), s.x->options()),
                   gc = at::empty(s.b->sizes(), s.x->options()),
                   gskip = s.skip ? at::empty({s.d}, s.a->options()) : at::Tensor(),
                   gz = s.z ? at::empty(s.x->sizes(), s.x->options()) : at::Tensor(),
                   gbias = s.bias ? at::empty({s.d}, s.a->options()) : at::Tensor(),
                   gi = at::empty({b, s.d, s.n}, s.a->options());
  const size_t bytes = lib.selective_scan_backward_bytes(s.code, s.x->sizes().data(), s.b->sizes().data());
  const at::Tensor ws = workspace(bytes, *s.x);
  return answer(scan_call(lib.selective_scan_backward, s, static_cast<const float*>(initial),
                          static_cast<const int32_t*>(lengths), go->strides().data(), go->data_ptr(),
                          static_cast<const float*>(gs), gx.data_ptr(), gd.data_ptr(),
                          static_cast<float*>(ga.data_ptr()), gb.data_ptr(), gc.data_ptr(),
                          static_cast<float*>(data(gskip)), data(gz), static_cast<float*>(data(gbias)),
                          static_cast<float*>(gi.data_ptr()), data(ws), bytes, c.stream()),
                gx, gd, ga, gb, gc, gskip, gz, gbias, gi);
}

// (x, delta, a, b, c, state, slots, skip, z, delta_bias, softplus)
PyObject* selective_scan_step(PyObject* const* a, Py_ssize_t n) {
  Call c;
  ScanCall s;
  if (n != 11 || !scan_args(c, a, a + 7, 2, &s)) return the_long_way();
  const at::Tensor* state = pool_arg(c, a[5], at::kFloat, s.d, s.n);
  const void* slots = c.optional(a[6], at::kInt, {s.x->size(0)});
  if (!c.here()) return the_long_way();
  const at::Tensor out = at::empty(s.x->sizes(), s.x->options());
  const sx_status st = scan_call(lib.selective_scan_step, s, state->size(0), state->stride(0),
                                 static_cast<float*>(state->data_ptr()), static_cast<const int32_t*>(slots),
                                 out.data_ptr(), c.stream());
  written(st, state);
  return answer(st, out);
}

struct NormCall {
  const at::Tensor* x;
  int64_t shape[3], strides[3], groups;
  const float *w, *bias;
  sx_dtype code;
  double eps;
  sx_activation act;
};

// [N, ..., C] as [N, positions, C], where that is a view of channels next to each other
bool positions(const at::Tensor& t, int64_t* shape, int64_t* strides) {
  const int64_t rank = t.dim();
  if (rank < 2 || t.size(-1) == 0 || (t.size(-1) > 1 && t.stride(-1) != 1)) return false;
  shape[0] = t.size(0);
  shape[1] = rank == 2 ? 1 : t.size(1);
  shape[2] = t.size(-1);
  strides[0] = t.stride(0);
  strides[1] = rank == 2 ? shape[2] : t.stride(rank - 2);
  strides[2] = 1;
  for (int64_t i = 2; i < rank - 1; ++i) {
    if (t.stride(i - 1) != t.stride(i) * t.size(i)) return false;
    shape[1] *= t.size(i);
  }
  return true;
}

bool norm_args(Call& c, PyObject* x, PyObject* groups, PyObject* const* r, NormCall* a) {
  a->x = c.take(x);
  if (!c.fit || !float_type(*a->x, &a->code) || !positions(*a->x, a->shape, a->strides) || !PyLong_CheckExact(groups) ||
      !activation(r[3], &a->act))
    return false;
  int over = 0;
  a->groups = PyLong_AsLongLongAndOverflow(groups, &over);
  a->w = static_cast<const float*>(c.optional(r[0], at::kFloat, {a->shape[2]}));
  a->bias = static_cast<const float*>(c.optional(r[1], at::kFloat, {a->shape[2]}));
  a->eps = c.number(r[2]);
  return c.fit && !over;
}

// (x, groups, weight, bias, eps, activation)
PyObject* group_norm(PyObject* const* a, Py_ssize_t n) {
  Call c;
  NormCall v;
  if (n != 6 || !norm_args(c, a[0], a[1], a + 2, &v) || !c.here()) return the_long_way();
  const at::Tensor out = at::empty(v.x->sizes(), v.x->options());
  const size_t bytes = lib.group_norm_bytes(v.code, v.shape, v.groups);
  const at::Tensor ws = workspace(bytes, *v.x);
  return answer(lib.group_norm(v.code, v.shape, v.strides, v.x->data_ptr(), v.groups, v.w, v.bias, float(v.eps), v.act,
                               out.data_ptr(), data(ws), bytes, c.stream()),
                out);
}

// (x, groups, grad_out, weight, bias, eps, activation)
PyObject* group_norm_backward(PyObject* const* a, Py_ssize_t n) {
  Call c;
  NormCall v;
  if (n != 7 || !norm_args(c, a[0], a[1], a + 3, &v)) return the_long_way();
  const at::Tensor* go = c.take(a[2]);
  int64_t gshape[3], gstrides[3];
  if (!c.here() || go->scalar_type() != v.x->scalar_type() || go->sizes() != v.x->sizes() ||
      !positions(*go, gshape, gstrides))
    return the_long_way();
  const auto f32 = v.x->options().dtype(at::kFloat);
  const at::Tensor gx = at::empty(v.x->sizes(), v.x->options()),
                   gw = v.w ? at::empty({v.shape[2]}, f32) : at::Tensor(),
                   gb = v.bias ? at::empty({v.shape[2]}, f32) : at::Tensor();
  const size_t bytes = lib.group_norm_backward_bytes(v.code, v.shape, v.groups);
  const at::Tensor ws = workspace(bytes, *v.x);
  return answer(lib.group_norm_backward(v.code, v.shape, v.strides, v.x->data_ptr(), v.groups, v.w, v.bias,
                                        float(v.eps), v.act, gstrides, go->data_ptr(), gx.data_ptr(),
                                        static_cast<float*>(data(gw)), static_cast<float*>(data(gb)), data(ws), bytes,
                                        c.stream()),
                gx, gw, gb);
}

// (addresses of the entries, torch's current device, its raw stream of a device)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* at = nullptr;
  PyObject *device = nullptr, *stream = nullptr;
  if (!PyArg_ParseTuple(args, "O!OO", &PyTuple_Type, &at, &device, &stream)) return nullptr;
  void* p[kEntries];
  if (PyTuple_GET_SIZE(at) != kEntries)
    return PyErr_Format(PyExc_ValueError, "%d entries are expected", kEntries), nullptr;
  for (int i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(at, i));
    if (PyErr_Occurred()) return nullptr;
  }
  lib = Entries{reinterpret_cast<decltype(lib.decay_attention)>(p[0]),
                reinterpret_cast<decltype(lib.decay_attention_bytes)>(p[1]),
                reinterpret_cast<decltype(lib.decay_attention_backward)>(p[2]),
                reinterpret_cast<decltype(lib.decay_attention_backward_bytes)>(p[3]),
                reinterpret_cast<decltype(lib.decay_attention_step)>(p[4]),
                reinterpret_cast<decltype(lib.head_norm_rotate)>(p[5]),
                reinterpret_cast<decltype(lib.head_norm_rotate_backward)>(p[6]),
                reinterpret_cast<decltype(lib.head_norm_rotate_backward_bytes)>(p[7]),
                reinterpret_cast<decltype(lib.causal_conv)>(p[8]),
                reinterpret_cast<decltype(lib.causal_conv_backward)>(p[9]),
                reinterpret_cast<decltype(lib.causal_conv_backward_bytes)>(p[10]),
                reinterpret_cast<decltype(lib.causal_conv_step)>(p[11]),
                reinterpret_cast<decltype(lib.selective_scan)>(p[12]),
                reinterpret_cast<decltype(lib.selective_scan_bytes)>(p[13]),
                reinterpret_cast<decltype(lib.selective_scan_backward)>(p[14]),
                reinterpret_cast<decltype(lib.selective_scan_backward_bytes)>(p[15]),
                reinterpret_cast<decltype(lib.selective_scan_step)>(p[16]),
                reinterpret_cast<decltype(lib.group_norm)>(p[17]),
                reinterpret_cast<decltype(lib.group_norm_bytes)>(p[18]),
                reinterpret_cast<decltype(lib.group_norm_backward)>(p[19]),
                reinterpret_cast<decltype(lib.group_norm_backward_bytes)>(p[20])};
  Py_INCREF(device);
  Py_INCREF(stream);
  current_device = device;
  raw_stream = stream;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyCFunction method() {
  PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t) = guarded<F>;
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"decay_attention", method<decay_attention>(), METH_FASTCALL, nullptr},
    {"decay_attention_backward", method<decay_attention_backward>(), METH_FASTCALL, nullptr},
    {"decay_attention_step", method<decay_attention_step>(), METH_FASTCALL, nullptr},
    {"head_norm_rotate", method<head_norm_rotate>(), METH_FASTCALL, nullptr},
    {"head_norm_rotate_backward", method<head_norm_rotate_backward>(), METH_FASTCALL, nullptr},
    {"causal_conv", method<causal_conv>(), METH_FASTCALL, nullptr},
    {"causal_conv_backward", method<causal_conv_backward>(), METH_FASTCALL, nullptr},
    {"causal_conv_step", method<causal_conv_step>(), METH_FASTCALL, nullptr},
    {"selective_scan", method<selective_scan>(), METH_FASTCALL, nullptr},
    {"selective_scan_backward", method<selective_scan_backward>(), METH_FASTCALL, nullptr},
    {"selective_scan_step", method<selective_scan_step>(), METH_FASTCALL, nullptr},
    {"group_norm", method<group_norm>(), METH_FASTCALL, nullptr},
    {"group_norm_backward", method<group_norm_backward>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sx_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__sx_marshal() { return PyModule_Create(&module); }
