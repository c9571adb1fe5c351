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

detffn_options options(PyObject* path, PyObject* spin_limit, PyObject* flags) {
  detffn_options o{};
  o.leaf_width = 64;
  o.path = (int)integer(path);
  o.shards = 1;
  o.spin_limit = integer(spin_limit);
  o.flags = (int)integer(flags);
  return o;
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
  const detffn_options o = options(a[12], a[13], a[14]);
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

// What a grouped call's tensors share: x or dOut [R, ...], W [E, N, K], offsets.
struct Groups {
  long long R, E, K, N;
  int device, type;
  const int* offsets;
};
Groups groups(const Tensor* rows_of, const Tensor* W, const Tensor* offsets) {
  need(rows_of && W && offsets && rows_of->is_cuda() && rows_of->dim() == 2 && W->dim() == 3 &&
           type_of(rows_of->scalar_type()) >= 0,
       "expected x [R, K] and W [E, N, K] in float32, float16 or bfloat16 on a CUDA device, and offsets");
  Groups g;
  g.R = rows_of->size(0), g.E = W->size(0), g.N = W->size(1), g.K = W->size(2);
  g.device = (int)rows_of->get_device();
  g.type = type_of(rows_of->scalar_type());
  WHOLE(*W, g.device, rows_of->scalar_type(), {g.E, g.N, g.K});
  whole(*offsets, g.device, at::kInt, {g.E + 1}, "offsets: expected a contiguous int32 CUDA tensor [E + 1]");
  g.offsets = static_cast<const int*>(offsets->data_ptr());
  return g;
}
// Rows [R, width] of a grouped call.
long long group_rows(const Tensor* t, const Groups& g, long long width, const Tensor* like, const char* what) {
  need(t && t->dim() == 2 && t->size(0) == g.R && t->size(1) == width && t->scalar_type() == like->scalar_type() &&
           t->get_device() == like->get_device(),
       what);
  return rows(t, nullptr, what);
}
#define GROUP_ROWS(t, width, like) \
  group_rows(t, g, width, like, #t ": expected a 2-D CUDA tensor of contiguous rows with the call's shape, dtype and device")

const Tensor* group_scratch(const Groups& g, const Tensor* ws, const Tensor* like, Tensor* own) {
  size_t bytes = 0;
  check(detffn_grouped_workspace_size(g.R, g.E, g.K, g.N, g.type, &bytes), "detffn_grouped_workspace_size");
  if (!ws && bytes) ws = &(*own = empty({(long long)bytes}, *like, at::kByte));
  need(!ws || (ws->is_cuda() && ws->get_device() == g.device && ws->is_contiguous()), "ws: expected a contiguous CUDA buffer");
  return ws;
}

// (handle, x, W, offsets, out, ws, path, spin_limit, flags)
PyObject* grouped_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(9)
  const Tensor *x = tensor(a[1], "x"), *W = tensor(a[2], "W"), *offsets = tensor(a[3], "offsets"),
               *out = tensor(a[4], "out"), *ws = tensor(a[5], "ws");
  const Groups g = groups(x, W, offsets);
  const long long ldx = GROUP_ROWS(x, g.K, x);
  const c10::cuda::CUDAGuard guard(x->device());
  Tensor t_out, t_ws;
  if (!out) out = &(t_out = empty({g.R, g.N}, *x, x->scalar_type()));
  const long long ldo = GROUP_ROWS(out, g.N, x);
  ws = group_scratch(g, ws, x, &t_ws);
  const detffn_options o = options(a[6], a[7], a[8]);
  check(detffn_grouped_forward(reinterpret_cast<detffn_handle>(integer(a[0])), x->data_ptr(), ldx, W->data_ptr(),
                               g.offsets, out->data_ptr(), ldo, g.R, g.E, g.K, g.N, g.type, const_cast<void*>(ptr(ws)),
                               ws ? (size_t)ws->nbytes() : 0, stream_of(g.device), &o),
        "detffn_grouped_forward");
  return tuple({out});
  END_BODY
}

// (handle, x, W, offsets, dOut, dX, dW, need_dX, need_dW, ws, path, spin_limit, flags)
PyObject* grouped_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(13)
  const Tensor *x = tensor(a[1], "x"), *W = tensor(a[2], "W"), *offsets = tensor(a[3], "offsets"),
               *dOut = tensor(a[4], "dOut"), *dX = tensor(a[5], "dX"), *dW = tensor(a[6], "dW"), *ws = tensor(a[9], "ws");
  const bool want_x = PyObject_IsTrue(a[7]) == 1, want_w = PyObject_IsTrue(a[8]) == 1;
  need(want_x || want_w, "nothing to form: need_dX and need_dW are both false");
  need((want_x || !dX) && (want_w || !dW), "dX and dW go with need_dX and need_dW");
  const Groups g = groups(dOut, W, offsets);
  const long long lddo = GROUP_ROWS(dOut, g.N, dOut), ldx = want_w || x ? GROUP_ROWS(x, g.K, dOut) : 0;
  const c10::cuda::CUDAGuard guard(dOut->device());
  Tensor t_x, t_w, t_ws;
  if (want_x && !dX) dX = &(t_x = empty({g.R, g.K}, *dOut, dOut->scalar_type()));
  if (want_w && !dW) dW = &(t_w = empty({g.E, g.N, g.K}, *dOut, dOut->scalar_type()));
  const long long lddx = want_x ? GROUP_ROWS(dX, g.K, dOut) : 0;
  if (want_w) WHOLE(*dW, g.device, dOut->scalar_type(), {g.E, g.N, g.K});
  ws = group_scratch(g, ws, dOut, &t_ws);
  const detffn_options o = options(a[10], a[11], a[12]);
  check(detffn_grouped_backward(reinterpret_cast<detffn_handle>(integer(a[0])), ptr(x), ldx, W->data_ptr(), g.offsets,
                                dOut->data_ptr(), lddo, const_cast<void*>(ptr(dX)), lddx, const_cast<void*>(ptr(dW)), g.R,
                                g.E, g.K, g.N, g.type, const_cast<void*>(ptr(ws)), ws ? (size_t)ws->nbytes() : 0,
                                stream_of(g.device), &o),
        "detffn_grouped_backward");
  return tuple({dX, dW});
  END_BODY
}

at::ScalarType scalar_of(long long code) {
  need(code >= DETFFN_F32 && code <= DETFFN_BF16, "dtype: expected float32, float16 or bfloat16");
  return code == DETFFN_F32 ? at::kFloat : code == DETFFN_F16 ? at::kHalf : at::kBFloat16;
}
long long bounded(PyObject* o, const char* what) {
  const long long v = integer(o);
  need(v >= 1 && v <= 1 << 20, what);
  return v;
}

// A 4-bit matrix at a[0 .. 3]: codes, scales, K, group.
struct Bits4 {
  const Tensor *codes, *scales;
  long long N, K, group;
  int device, type;
};
Bits4 bits4(PyObject* const* a) {
  Bits4 m;
  m.codes = tensor(a[0], "codes");
  m.scales = tensor(a[1], "scales");
  m.K = bounded(a[2], "K: expected 1 to 2^20");
  m.group = bounded(a[3], "group: expected 32, 64 or 128");
  const char* what = "expected contiguous CUDA codes [N, 64 ceil(K / 128)] (uint8) and scales [N, ceil(K / group)] (float32, float16 or bfloat16)";
  need(m.codes && m.scales && m.codes->dim() == 2 && m.codes->is_cuda() && type_of(m.scales->scalar_type()) >= 0, what);
  m.N = m.codes->size(0);
  m.device = (int)m.codes->get_device();
  m.type = type_of(m.scales->scalar_type());
  whole(*m.codes, m.device, at::kByte, {m.N, (m.K + 127) / 128 * 64}, what);
  whole(*m.scales, m.device, m.scales->scalar_type(), {m.N, (m.K + m.group - 1) / m.group}, what);
  return m;
}

// (w, group, scale dtype code, codes, scales) with the last two both None or neither
PyObject* w4_pack(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(5)
  const Tensor *w = tensor(a[0], "w"), *codes = tensor(a[3], "codes"), *scales = tensor(a[4], "scales");
  need(w != nullptr, "w must be given");
  const long long ldw = ROWS(w, nullptr), N = w->size(0), K = w->size(1), group = bounded(a[1], "group: expected 32, 64 or 128");
  const at::ScalarType st = scalar_of(integer(a[2]));
  const int dev = (int)w->get_device();
  const c10::cuda::CUDAGuard guard(w->device());
  need(!codes == !scales, "codes and scales go together");
  Tensor c, s;
  if (!codes) {
    Together both;
    both.add(&c, {N, (K + 127) / 128 * 64}, at::kByte);
    both.add(&s, {N, (K + group - 1) / group}, st);
    both.allocate(*w);
    codes = &c, scales = &s;
  }
  WHOLE(*codes, dev, at::kByte, {N, (K + 127) / 128 * 64});
  WHOLE(*scales, dev, st, {N, (K + group - 1) / group});
  check(detffn_w4_pack(w->data_ptr(), ldw, codes->data_ptr(), scales->data_ptr(), N, K, (int)group, type_of(w->scalar_type()),
                       type_of(st), stream_of(dev)),
        "detffn_w4_pack");
  return tuple({codes, scales});
  END_BODY
}

// (codes, scales, K, group, dtype code, out)
PyObject* w4_unpack(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(6)
  const Bits4 m = bits4(a);
  const at::ScalarType st = scalar_of(integer(a[4]));
  const Tensor* out = tensor(a[5], "out");
  const c10::cuda::CUDAGuard guard(m.codes->device());
  Tensor t;
  if (!out) out = &(t = empty({m.N, m.K}, *m.codes, st));
  const long long ldo = ROWS(out, nullptr);
  need(out->size(0) == m.N && out->size(1) == m.K && out->scalar_type() == st && out->get_device() == m.device,
       "out: expected [N, K] of dtype on the device of the codes");
  check(detffn_w4_unpack(m.codes->data_ptr(), m.scales->data_ptr(), out->data_ptr(), ldo, m.N, m.K, (int)m.group, type_of(st),
                         m.type, stream_of(m.device)),
        "detffn_w4_unpack");
  return tuple({out});
  END_BODY
}

// (x, codes, scales, K, group, out, ws)
PyObject* w4_matvec(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(7)
  const Tensor *x = tensor(a[0], "x"), *out = tensor(a[5], "out"), *ws = tensor(a[6], "ws");
  need(x != nullptr, "x must be given");
  const Bits4 m = bits4(a + 1);
  const long long ldx = ROWS(x, nullptr), T = x->size(0);
  need(x->size(1) == m.K && x->get_device() == m.device, "x: expected [T, K] on the device of the codes");
  const c10::cuda::CUDAGuard guard(x->device());
  Tensor t;
  if (!out) out = &(t = empty({T, m.N}, *x, x->scalar_type()));
  const long long ldo = ROWS(out, nullptr);
  need(out->size(0) == T && out->size(1) == m.N && out->scalar_type() == x->scalar_type() && out->get_device() == m.device,
       "out: expected [T, N] of x's dtype on its device");
  const int dt = type_of(x->scalar_type());
  Tensor t_ws;
  if (!ws && (dt == DETFFN_F32 || (uintptr_t)x->data_ptr() % 16 || m.K % 8 || (T > 1 && ldx % 8))) {
    size_t bytes = 0;
    check(detffn_w4_matvec_workspace_size(T, m.K, dt, &bytes), "detffn_w4_matvec_workspace_size");
    ws = &(t_ws = empty({(long long)(bytes < 256 ? 256 : bytes)}, *x, at::kByte));
  }
  need(!ws || (ws->is_cuda() && ws->get_device() == m.device && ws->is_contiguous()), "ws: expected a contiguous CUDA buffer");
  check(detffn_w4_matvec(x->data_ptr(), ldx, m.codes->data_ptr(), m.scales->data_ptr(), out->data_ptr(), ldo, T, m.N, m.K,
                         (int)m.group, dt, m.type, const_cast<void*>(ptr(ws)), ws ? (size_t)ws->nbytes() : 0,
                         stream_of(m.device)),
        "detffn_w4_matvec");
  return tuple({out});
  END_BODY
}

// (x, gate's four, up's four, down's four, out, ws)
PyObject* w4_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(15)
  const Tensor *x = tensor(a[0], "x"), *out = tensor(a[13], "out"), *ws = tensor(a[14], "ws");
  need(x != nullptr, "x must be given");
  const Bits4 g = bits4(a + 1), u = bits4(a + 5), d = bits4(a + 9);
  const long long ldx = ROWS(x, nullptr), T = x->size(0), H = g.K, I = g.N;
  need(x->size(1) == H && x->get_device() == g.device, "x: expected [T, H] on the device of the codes");
  need(u.K == H && u.N == I && d.K == I && d.N == H && u.group == g.group && d.group == g.group && u.type == g.type &&
           d.type == g.type && u.device == g.device && d.device == g.device,
       "expected gate and up [I, H] and down [H, I] of one group, scale dtype and device");
  const c10::cuda::CUDAGuard guard(x->device());
  Tensor t, t_ws;
  if (!out) out = &(t = empty({T, H}, *x, x->scalar_type()));
  const long long ldo = ROWS(out, x);
  size_t bytes = 0;
  check(detffn_w4_workspace_size(T, H, I, type_of(x->scalar_type()), &bytes), "detffn_w4_workspace_size");
  if (!ws) ws = &(t_ws = empty({(long long)(bytes < 256 ? 256 : bytes)}, *x, at::kByte));
  need(ws->is_cuda() && ws->get_device() == g.device && ws->is_contiguous(), "ws: expected a contiguous CUDA buffer");
  check(detffn_w4_forward(x->data_ptr(), ldx, g.codes->data_ptr(), g.scales->data_ptr(), u.codes->data_ptr(),
                          u.scales->data_ptr(), d.codes->data_ptr(), d.scales->data_ptr(), out->data_ptr(), ldo, T, H, I,
                          (int)g.group, type_of(x->scalar_type()), g.type, ws->data_ptr(), (size_t)ws->nbytes(),
                          stream_of(g.device)),
        "detffn_w4_forward");
  return tuple({out});
  END_BODY
}

// The low 64 bits of an integer in [0, 2^64).
unsigned long long word64(PyObject* o, const char* what) {
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) {
    if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw Refused();
    PyErr_Clear();
    refuse(what);
  }
  return v;
}

// (x, p, seed (a number or a tensor), offset, residual, out, backward)
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  BODY(7)
  const Tensor *x = tensor(a[0], "x"), *residual = tensor(a[4], "residual"), *out = tensor(a[5], "out");
  need(x != nullptr, "x must be given");
  const long long ldx = ROWS(x, nullptr), ldr = ROWS(residual, x), M = x->size(0), H = x->size(1);
  const int dev = (int)x->get_device();
  const Tensor* state = THPVariable_Check(a[2]) ? tensor(a[2], "seed") : nullptr;
  if (state) whole(*state, dev, at::kLong, {2}, "seed: expected a number or a contiguous int64 CUDA tensor [2]");
  const unsigned long long seed = state ? 0 : word64(a[2], "seed: expected 0 to 2^64 - 1"),
                           offset = word64(a[3], "offset: expected 0 to 2^64 - 1");
  const c10::cuda::CUDAGuard guard(x->device());
  Tensor t;
  if (!out) out = &(t = empty({M, H}, *x, x->scalar_type()));
  const long long ldo = ROWS(out, x);
  const unsigned long long* words = static_cast<const unsigned long long*>(ptr(state));
  const int type = type_of(x->scalar_type());
  if (PyObject_IsTrue(a[6]) == 1)
    check(detffn_dropout_backward(x->data_ptr(), ldx, out->data_ptr(), ldo, number(a[1]), seed, offset, words, M, H, type,
                                  stream_of(dev)),
          "detffn_dropout_backward");
  else
    check(detffn_dropout_forward(x->data_ptr(), ldx, ptr(residual), ldr, out->data_ptr(), ldo, number(a[1]), seed, offset,
                                 words, M, H, type, stream_of(dev)),
          "detffn_dropout_forward");
  return tuple({out});
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
                         FAST(grouped_forward), FAST(grouped_backward),
                         FAST(w4_pack),         FAST(w4_unpack),      FAST(w4_matvec),
                         FAST(w4_forward),      FAST(dropout),
                         {"set_error", set_error, METH_O, nullptr},      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
