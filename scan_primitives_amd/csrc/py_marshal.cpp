// py_marshal.cpp: the short way from Python to the linear-attention entry points
// of libsx_scan.so, for calls whose time is that of getting to the GPU.
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
} lib;
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

// (addresses of the eight entries, torch's current device, its raw stream of a device)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* at = nullptr;
  PyObject *device = nullptr, *stream = nullptr;
  if (!PyArg_ParseTuple(args, "O!OO", &PyTuple_Type, &at, &device, &stream)) return nullptr;
  void* p[8];
  if (PyTuple_GET_SIZE(at) != 8) return PyErr_SetString(PyExc_ValueError, "eight entries are expected"), nullptr;
  for (int i = 0; i < 8; ++i) {
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
                reinterpret_cast<decltype(lib.head_norm_rotate_backward_bytes)>(p[7])};
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
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sx_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__sx_marshal() { return PyModule_Create(&module); }
