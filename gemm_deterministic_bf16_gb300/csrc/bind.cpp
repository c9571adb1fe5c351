// bind.cpp -- the native half of block.py: takes PyTorch tensors, checks them,
// allocates results and scratch on the current stream, and makes the C call.
// A decode step calls these operators on a few kilobytes, where a call's time
// is the host's: the same checks in Python cost 20-50 us a call, these 2-3.
//
// Every function is called with positional arguments by the function of the
// same name in block.py, which documents it, and raises ValueError for tensors
// that do not fit and DetFFNError for a status other than OK.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "detffn.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // DetFFNError(status, name)

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  throw Refused();
}
void need(bool ok, const char* what) {
  if (!ok) refuse(what);
}

// The tensor of an argument; null for None.
const Tensor* tensor(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, what);
    throw Refused();
  }
  return &THPVariable_Unpack(o);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int type_of(at::ScalarType t) {
  return t == at::kFloat ? DETFFN_F32 : t == at::kHalf ? DETFFN_F16 : t == at::kBFloat16 ? DETFFN_BF16 : -1;
}

const void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

PyObject* wrap(const Tensor* t) {
  if (!t) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}

void check(int status, const char* name) {
  if (status == DETFFN_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", status, name);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

PyObject* tuple(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Refused();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw Refused();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// A 2-D tensor of contiguous rows, like `lead` where there is one: its row stride.
long long rows(const Tensor* t, const Tensor* lead, const char* what) {
  if (!t) return 0;
  need(t->is_cuda() && t->dim() == 2 && type_of(t->scalar_type()) >= 0 && (t->size(1) == 1 || t->stride(1) == 1), what);
  need(!lead || (t->sizes() == lead->sizes() && t->scalar_type() == lead->scalar_type() &&
                 t->get_device() == lead->get_device()),
       what);
  return t->stride(0);
}
#define ROWS(t, lead) \
  rows(t, lead, #t ": expected a 2-D CUDA tensor of contiguous rows in float32, float16 or bfloat16, with the shape, dtype and device of the call's other rows")

// A parameter of the call: the rows' type or FP32, one type for all.
void param(const Tensor* t, const Tensor& lead, at::ScalarType* type, bool vector, const char* what) {
  if (!t) return;
  need(t->is_cuda() && t->get_device() == lead.get_device() &&
           (t->scalar_type() == lead.scalar_type() || t->scalar_type() == at::kFloat),
       what);
  need(*type == at::ScalarType::Undefined || *type == t->scalar_type(), "w_post, w_pre and gate must have one dtype");
  need(!vector || (t->dim() == 1 && t->size(0) == lead.size(1) && t->is_contiguous()), what);
  *type = t->scalar_type();
}

// Strides of a gate of shape [], [1], [H], [M, 1], [1, H] or [M, H].
void gate_strides(const Tensor* g, long long M, long long H, long long* rs, long long* cs) {
  *rs = *cs = 0;
  if (!g) return;
  need(g->dim() <= 2, "gate: expected [], [1], [H], [M, 1] or [M, H]");
  const long long a = g->dim() == 2 ? g->size(0) : 1, b = g->dim() >= 1 ? g->size(-1) : 1;
  need((a == 1 || a == M) && (b == 1 || b == H), "gate: expected [], [1], [H], [M, 1] or [M, H]");
  if (b > 1) {
    need(g->stride(-1) == 1, "gate: an expanded gate is given in its own shape, with contiguous features");
    *cs = 1;
  }
  if (a > 1) {
    *rs = g->stride(0);
    need(*rs > 0, "gate: an expanded gate is given in its own shape, with contiguous features");
  }
}

void whole(const Tensor& t, int device, at::ScalarType type, at::IntArrayRef shape, const char* what) {
  need(t.is_cuda() && t.is_contiguous() && t.get_device() == device && t.scalar_type() == type && t.sizes() == shape, what);
}
#define WHOLE(t, device, type, ...) \
  whole(t, device, type, __VA_ARGS__, #t ": expected a contiguous CUDA tensor of the call's shape, dtype and device")

void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

// A CUDA tensor beside `like`, from its allocator directly.
Tensor empty(at::IntArrayRef shape, const Tensor& like, at::ScalarType type) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// Results that belong together (a checkpoint's four, the parameters'
// gradients) share an allocation, 256-byte aligned each: an allocation takes
// 0.9 us of a call, a tensor on part of one 0.2.
class Together {
 public:
  void add(Tensor* out, at::IntArrayRef shape, at::ScalarType type) {
    long long n = (long long)c10::elementSize(type);
    for (long long d : shape) n *= d;
    piece_[n_++] = {out, at::DimVector(shape), type, bytes_};
    bytes_ += (n + 255) / 256 * 256;
  }
  void allocate(const Tensor& like) {
    if (n_ == 0) return;
    const Tensor all = empty({bytes_}, like, at::kByte);
    for (int i = 0; i < n_; ++i) {
      const Piece& p = piece_[i];
      *p.out = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                        c10::scalarTypeToTypeMeta(p.type));
      c10::TensorImpl* t = p.out->unsafeGetTensorImpl();
      t->set_storage_offset(p.at / (long long)c10::elementSize(p.type));
      t->set_sizes_contiguous(p.shape);
    }
  }

 private:
  struct Piece {
    Tensor* out;
    at::DimVector shape;
    at::ScalarType type;
    long long at;
  };
  Piece piece_[4];
  int n_ = 0;
  long long bytes_ = 0;
};

#define BODY(n)                                                             \
  HANDLE_TH_ERRORS                                                          \
  if (nargs != (n)) {                                                       \
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");          \
    return nullptr;                                                         \
  }                                                                         \
  try {
#define END_BODY          \
  }                       \
  catch (const Refused&) { \
    return nullptr;       \
  }                       \
  END_HANDLE_TH_ERRORS

// (x, z, w_post, gate, scale, w_pre, eps, out, y)
PyObject* join_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(9)
  const Tensor *x = tensor(a[0], "x"), *z = tensor(a[1], "z"), *w_post = tensor(a[2], "w_post"),
               *gate = tensor(a[3], "gate"), *w_pre = tensor(a[5], "w_pre"), *out = tensor(a[7], "out"),
               *y = tensor(a[8], "y");
  need(x != nullptr, "x must be given");
  const long long ldx = ROWS(x, nullptr), ldz = ROWS(z, x), M = x->size(0), H = x->size(1);
  at::ScalarType pt = at::ScalarType::Undefined;
  param(w_post, *x, &pt, true, "w_post: expected a contiguous [H] tensor of the rows' dtype or float32");
  param(w_pre, *x, &pt, true, "w_pre: expected a contiguous [H] tensor of the rows' dtype or float32");
  param(gate, *x, &pt, false, "gate: expected the rows' dtype or float32");
  long long rs, cs;
  gate_strides(gate, M, H, &rs, &cs);
  const c10::cuda::CUDAGuard guard(x->device());
  Tensor o, v;
  if (z && !out) out = &(o = empty({M, H}, *x, x->scalar_type()));
  if (w_pre && !y) y = &(v = empty({M, H}, *x, x->scalar_type()));
  const long long ldo = ROWS(out, x), ldy = ROWS(y, x);
  const int dt = type_of(x->scalar_type());
  check(detffn_join_forward(ptr(x), ldx, ptr(z), ldz, ptr(w_post), ptr(gate), rs, cs, (float)number(a[4]), ptr(w_pre),
                            (float)number(a[6]), const_cast<void*>(ptr(out)), ldo, const_cast<void*>(ptr(y)), ldy, M, H,
                            dt, pt == at::ScalarType::Undefined ? dt : type_of(pt), stream_of(x->get_device())),
        "detffn_join_forward");
  return tuple({out, y});
  END_BODY
}

// (r, z, dr, dy, w_post, gate, scale, w_pre, eps, dx, dz, ws)
PyObject* join_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(12)
  const Tensor *r = tensor(a[0], "r"), *z = tensor(a[1], "z"), *dr = tensor(a[2], "dr"), *dy = tensor(a[3], "dy"),
               *w_post = tensor(a[4], "w_post"), *gate = tensor(a[5], "gate"), *w_pre = tensor(a[7], "w_pre"),
               *dx = tensor(a[9], "dx"), *dz = tensor(a[10], "dz"), *ws = tensor(a[11], "ws");
  const Tensor* lead = r ? r : dr;
  need(lead != nullptr, "r or dr must be given");
  need(!w_pre || (r && dy), "w_pre: r and dy must be given");
  need(w_pre || (dr && !dy), "without w_pre: dr and no dy");
  const long long ldr = ROWS(r, nullptr), lddr = ROWS(dr, lead), lddy = ROWS(dy, lead), ldz = ROWS(z, lead);
  const long long M = lead->size(0), H = lead->size(1);
  at::ScalarType pt = at::ScalarType::Undefined;
  param(w_post, *lead, &pt, true, "w_post: expected a contiguous [H] tensor of the rows' dtype or float32");
  param(w_pre, *lead, &pt, true, "w_pre: expected a contiguous [H] tensor of the rows' dtype or float32");
  param(gate, *lead, &pt, false, "gate: expected the rows' dtype or float32");
  long long rs, cs;
  gate_strides(gate, M, H, &rs, &cs);
  need(w_pre || !dx || dx->is_same(*dr), "without w_pre the gradient of x is dr itself");
  const c10::cuda::CUDAGuard guard(lead->device());
  const at::ScalarType st = lead->scalar_type();
  if (pt == at::ScalarType::Undefined) pt = st;
  Tensor t_dx, t_dz, t_gate, t_post, t_pre, t_ws;
  const Tensor *dgate = nullptr, *dw_post = nullptr, *dw_pre = nullptr;
  if (z && !dz) dz = &(t_dz = empty({M, H}, *lead, st));
  if (w_pre && !dx) dx = &(t_dx = empty({M, H}, *lead, st));
  const long long lddx = w_pre ? ROWS(dx, lead) : 0, lddz = ROWS(dz, lead);
  Together grads;
  if (gate && gate->numel() > H) t_gate = empty(gate->sizes(), *lead, pt);
  else if (gate) grads.add(&t_gate, gate->sizes(), pt);
  if (w_post) grads.add(&t_post, {H}, pt);
  if (w_pre) grads.add(&t_pre, {H}, pt);
  grads.allocate(*lead);
  if (gate) dgate = &t_gate;
  if (w_post) dw_post = &t_post;
  if (w_pre) dw_pre = &t_pre;
  size_t bytes = 0;
  if (!ws) {
    check(detffn_join_workspace_size(M, H, &bytes), "detffn_join_workspace_size");
    ws = &(t_ws = empty({(long long)(bytes < 256 ? 256 : bytes)}, *lead, at::kByte));
  }
  need(ws->is_cuda() && ws->get_device() == lead->get_device() && ws->is_contiguous(), "ws: expected a contiguous CUDA buffer");
  check(detffn_join_backward(ptr(r), ldr, ptr(dr), lddr, ptr(dy), lddy, ptr(z), ldz, ptr(w_post), ptr(gate), rs, cs,
                             (float)number(a[6]), ptr(w_pre), (float)number(a[8]),
                             w_pre ? const_cast<void*>(ptr(dx)) : nullptr, lddx, const_cast<void*>(ptr(dz)), lddz,
                             const_cast<void*>(ptr(dgate)), const_cast<void*>(ptr(dw_post)),
                             const_cast<void*>(ptr(dw_pre)), M, H, type_of(st), type_of(pt),
                             const_cast<void*>(ptr(ws)), (size_t)ws->nbytes(), stream_of(lead->get_device())),
        "detffn_join_backward");
  return tuple({w_pre ? dx : dr, dz, dgate, dw_post, dw_pre});
  END_BODY
}

// A checkpoint's four tensors at a[0 .. 3], checked; [M, I] of its codes.
struct Ckpt {
  const Tensor *gq, *gs, *uq, *us;
  long long M, I;
  int device;
};
Ckpt checkpoint(PyObject* const* a) {
  Ckpt c;
  c.gq = tensor(a[0], "gate_codes");
  c.gs = tensor(a[1], "gate_scales");
  c.uq = tensor(a[2], "up_codes");
  c.us = tensor(a[3], "up_scales");
  need(c.gq && c.gs && c.uq && c.us && c.gq->dim() == 2, "checkpoint: expected codes [M, I] and scales [M, ceil(I / 64)]");
  c.M = c.gq->size(0);
  c.I = c.gq->size(1);
  c.device = c.gq->is_cuda() ? (int)c.gq->get_device() : -1;
  const char* what = "checkpoint: expected contiguous CUDA codes [M, I] (int8) and scales [M, ceil(I / 64)] (float32)";
  whole(*c.gq, c.device, at::kChar, {c.M, c.I}, what);
  whole(*c.uq, c.device, at::kChar, {c.M, c.I}, what);
  whole(*c.gs, c.device, at::kFloat, {c.M, (c.I + 63) / 64}, what);
  whole(*c.us, c.device, at::kFloat, {c.M, (c.I + 63) / 64}, what);
  return c;
}

// (gate, up, gate_codes, gate_scales, up_codes, up_scales) with the last four all None or none
PyObject* ckpt8_pack(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(6)
  const Tensor *gate = tensor(a[0], "gate"), *up = tensor(a[1], "up");
  need(gate && up && gate->is_cuda() && gate->dim() == 2 && type_of(gate->scalar_type()) >= 0,
       "gate: expected a CUDA tensor [M, I] in float32, float16 or bfloat16");
  const long long M = gate->size(0), I = gate->size(1);
  const int dev = (int)gate->get_device();
  WHOLE(*gate, dev, gate->scalar_type(), {M, I});
  WHOLE(*up, dev, gate->scalar_type(), {M, I});
  const c10::cuda::CUDAGuard guard(gate->device());
  Tensor gq, gs, uq, us;
  const Tensor *q0, *s0, *q1, *s1;
  if (a[2] != Py_None) {
    const Ckpt c = checkpoint(a + 2);
    need(c.M == M && c.I == I && c.device == dev, "ckpt: expected buffers of gate's shape on its device");
    q0 = c.gq, s0 = c.gs, q1 = c.uq, s1 = c.us;
  } else {
    const long long nb = (I + 63) / 64;
    Together all;
    all.add(&gq, {M, I}, at::kChar);
    all.add(&uq, {M, I}, at::kChar);
    all.add(&gs, {M, nb}, at::kFloat);
    all.add(&us, {M, nb}, at::kFloat);
    all.allocate(*gate);
    q0 = &gq, s0 = &gs, q1 = &uq, s1 = &us;
  }
  check(detffn_ckpt8_pack(gate->data_ptr(), up->data_ptr(), q0->data_ptr(), s0->data_ptr(), q1->data_ptr(),
                          s1->data_ptr(), M, I, type_of(gate->scalar_type()), stream_of(dev)),
        "detffn_ckpt8_pack");
  return tuple({q0, s0, q1, s1});
  END_BODY
}

// (gate_codes, gate_scales, up_codes, up_scales, gate, up, dtype code)
PyObject* ckpt8_unpack(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(7)
  const Ckpt c = checkpoint(a);
  const long long code = integer(a[6]);
  need(code >= DETFFN_F32 && code <= DETFFN_BF16, "dtype: expected float32, float16 or bfloat16");
  const at::ScalarType st = code == DETFFN_F32 ? at::kFloat : code == DETFFN_F16 ? at::kHalf : at::kBFloat16;
  const c10::cuda::CUDAGuard guard(c.gq->device());
  const Tensor *gate = tensor(a[4], "gate"), *up = tensor(a[5], "up");
  Tensor g, u;
  if (!gate) gate = &(g = empty({c.M, c.I}, *c.gq, st));
  if (!up) up = &(u = empty({c.M, c.I}, *c.gq, st));
  WHOLE(*gate, c.device, st, {c.M, c.I});
  WHOLE(*up, c.device, st, {c.M, c.I});
  check(detffn_ckpt8_unpack(c.gq->data_ptr(), c.gs->data_ptr(), c.uq->data_ptr(), c.us->data_ptr(), gate->data_ptr(),
                            up->data_ptr(), c.M, c.I, (int)code, stream_of(c.device)),
        "detffn_ckpt8_unpack");
  return tuple({gate, up});
  END_BODY
}

// (gate_codes, gate_scales, up_codes, up_scales, dh, dU, dG, h)
PyObject* ckpt8_silu_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(8)
  const Ckpt c = checkpoint(a);
  const Tensor *dh = tensor(a[4], "dh"), *dU = tensor(a[5], "dU"), *dG = tensor(a[6], "dG"), *h = tensor(a[7], "h");
  need(dh && type_of(dh->scalar_type()) >= 0, "dh: expected float32, float16 or bfloat16");
  const at::ScalarType st = dh->scalar_type();
  const c10::cuda::CUDAGuard guard(c.gq->device());
  Tensor u, g, v;
  if (!dU) dU = &(u = empty({c.M, c.I}, *c.gq, st));
  if (!dG) dG = &(g = empty({c.M, c.I}, *c.gq, st));
  if (!h) h = &(v = empty({c.M, c.I}, *c.gq, st));
  WHOLE(*dh, c.device, st, {c.M, c.I});
  WHOLE(*dU, c.device, st, {c.M, c.I});
  WHOLE(*dG, c.device, st, {c.M, c.I});
  WHOLE(*h, c.device, st, {c.M, c.I});
  check(detffn_ckpt8_silu_backward(dh->data_ptr(), c.gq->data_ptr(), c.gs->data_ptr(), c.uq->data_ptr(),
                                   c.us->data_ptr(), dU->data_ptr(), dG->data_ptr(), h->data_ptr(), c.M, c.I,
                                   type_of(st), stream_of(c.device)),
        "detffn_ckpt8_silu_backward");
  return tuple({dU, dG, h});
  END_BODY
}

// (handle, x, Wr, Wg, Wu, Wd, top_k, normalize, out, experts, weights, ws, path, spin_limit, flags)
PyObject* moe_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(15)
  const Tensor *x = tensor(a[1], "x"), *Wr = tensor(a[2], "Wr"), *Wg = tensor(a[3], "Wg"), *Wu = tensor(a[4], "Wu"),
               *Wd = tensor(a[5], "Wd"), *out = tensor(a[8], "out"), *experts = tensor(a[9], "experts"),
               *weights = tensor(a[10], "weights"), *ws = tensor(a[11], "ws");
  need(x && Wr && Wg && Wu && Wd && x->is_cuda() && x->dim() == 2 && Wg->dim() == 3 && type_of(x->scalar_type()) >= 0,
       "expected x [T, H], Wr [E, H], Wg and Wu [E, I, H], Wd [E, H, I] in float32, float16 or bfloat16");
  const long long T = x->size(0), H = x->size(1), E = Wg->size(0), I = Wg->size(1), k = integer(a[6]);
  const at::ScalarType st = x->scalar_type();
  const int dev = (int)x->get_device(), dt = type_of(st);
  WHOLE(*x, dev, st, {T, H});
  WHOLE(*Wr, dev, st, {E, H});
  WHOLE(*Wg, dev, st, {E, I, H});
  WHOLE(*Wu, dev, st, {E, I, H});
  WHOLE(*Wd, dev, st, {E, H, I});
  const c10::cuda::CUDAGuard guard(x->device());
  size_t bytes = 0;
  check(detffn_moe_workspace_size(T, E, k < 0 || k > 1 << 20 ? -1 : (int)k, H, I, dt, &bytes), "detffn_moe_workspace_size");
  Tensor t_out, t_experts, t_weights, t_ws;
  if (!out) out = &(t_out = empty({T, H}, *x, st));
  Together routing;
  if (!experts) routing.add(&t_experts, {T, k}, at::kInt);
  if (!weights) routing.add(&t_weights, {T, k}, at::kFloat);
  routing.allocate(*x);
  if (!experts) experts = &t_experts;
  if (!weights) weights = &t_weights;
  if (!ws) ws = &(t_ws = empty({(long long)(bytes < 256 ? 256 : bytes)}, *x, at::kByte));
  WHOLE(*out, dev, st, {T, H});
  WHOLE(*experts, dev, at::kInt, {T, k});
  WHOLE(*weights, dev, at::kFloat, {T, k});
  need(ws->is_cuda() && ws->get_device() == dev && ws->is_contiguous(), "ws: expected a contiguous CUDA buffer");
  detffn_options o{};
  o.leaf_width = 64;
  o.path = (int)integer(a[12]);
  o.shards = 1;
  o.spin_limit = integer(a[13]);
  o.flags = (int)integer(a[14]);
  const int normalize = PyObject_IsTrue(a[7]);
  if (normalize < 0) throw Refused();
  check(detffn_moe_forward(reinterpret_cast<detffn_handle>(integer(a[0])), x->data_ptr(), Wr->data_ptr(),
                           Wg->data_ptr(), Wu->data_ptr(), Wd->data_ptr(), out->data_ptr(),
                           static_cast<int*>(experts->data_ptr()), static_cast<float*>(weights->data_ptr()), T, E,
                           (int)k, normalize, H, I, dt, ws->data_ptr(), (size_t)ws->nbytes(), stream_of(dev), &o),
        "detffn_moe_forward");
  return tuple({out, experts, weights});
  END_BODY
}

PyObject* set_error(PyObject*, PyObject* e) {
  Py_XDECREF(g_error);
  Py_INCREF(e);
  g_error = e;
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(join_forward),  FAST(join_backward),       FAST(ckpt8_pack),
                         FAST(ckpt8_unpack),  FAST(ckpt8_silu_backward), FAST(moe_forward),
                         {"set_error", set_error, METH_O, nullptr},      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
