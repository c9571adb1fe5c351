"""ctypes binding of the operators around the FFN (argument marshalling only):
the residual join with its norms, 8-bit activation checkpoints, and the
mixture-of-experts layer for a few tokens.

Like ``detffn.py``: each function has the name of the C call it wraps, checks
tensor properties, passes pointers, sizes and a CUDA stream, and raises
``DetFFNError`` on a non-OK status.  A ``stream`` other than the current one
works on buffers of its own: what a call allocates for itself comes from that
stream's pool, and results it allocates are marked as used by the current
stream too.
"""
import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import detffn as _d
from .detffn import BF16, F16, F32, PATH_AUTO, _int, _ll, _vp

_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_f = ctypes.c_float
_sz = ctypes.c_size_t

_ARGS = {
    "detffn_join_forward": [_vp, _ll, _vp, _ll, _vp, _vp, _ll, _ll, _f, _vp, _f, _vp, _ll, _vp, _ll, _ll, _ll, _int,
                            _int, _vp],
    "detffn_join_workspace_size": [_ll, _ll, ctypes.POINTER(_sz)],
    "detffn_join_backward": [_vp, _ll, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _ll, _ll, _f, _vp, _f, _vp, _ll, _vp,
                             _ll, _vp, _vp, _vp, _ll, _ll, _int, _int, _vp, _sz, _vp],
    "detffn_ckpt8_pack": [_vp] * 6 + [_ll, _ll, _int, _vp],
    "detffn_ckpt8_unpack": [_vp] * 6 + [_ll, _ll, _int, _vp],
    "detffn_ckpt8_silu_backward": [_vp] * 8 + [_ll, _ll, _int, _vp],
    "detffn_moe_workspace_size": [_ll, _ll, _int, _ll, _ll, _int, ctypes.POINTER(_sz)],
    "detffn_moe_forward": [_vp] * 9 + [_ll, _ll, _int, _int, _ll, _ll, _int, _vp, _sz, _vp,
                                       ctypes.POINTER(_d.Options)],
}
_FN = {}


def _fn(name):
    f = _FN.get(name)
    if f is None:
        f = getattr(_d.lib(), name)
        f.argtypes = _ARGS[name]
        f.restype = ctypes.c_int
        _FN[name] = f
    return f


def _call(name, *args):
    status = (_FN.get(name) or _fn(name))(*args)
    if status != _d.OK:
        raise _d.DetFFNError(status, name)


class _On:
    """The device and stream of a call, and where what it allocates comes from."""

    __slots__ = ("dev", "raw", "stream", "switch")

    def __init__(self, dev, stream):
        self.dev = dev
        self.switch = dev.index != torch.cuda.current_device()
        self.stream = stream
        if stream is None:
            self.raw = torch.cuda.current_stream(dev).cuda_stream
        else:
            self.raw = stream.cuda_stream

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.dev)
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=self.dev)
        t.record_stream(torch.cuda.current_stream(self.dev))
        return t

    def device(self):
        return torch.cuda.device(self.dev) if self.switch else contextlib.nullcontext()


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _rows(t, name, shape=None, dtype=None, dev=None):
    """The row stride of a 2-D tensor of contiguous rows."""
    _need(t.dim() == 2 and t.is_cuda and t.dtype in _DTYPE and (t.stride(1) == 1 or t.shape[1] == 1),
          name + ": expected a 2-D CUDA tensor of contiguous rows in float32, float16 or bfloat16")
    _need((shape is None or t.shape == shape) and (dtype is None or t.dtype == dtype) and (dev is None or t.device == dev),
          name + ": shape, dtype and device must match the call's other rows")
    return t.stride(0)


def _params(dtype, H, dev, **given):
    """The one dtype of a call's parameter vectors."""
    pt = None
    for name, t in given.items():
        if t is None:
            continue
        _need(t.device == dev and (t.dtype == dtype or t.dtype == torch.float32),
              name + ": expected the rows' dtype or float32, on the same device")
        _need(pt is None or pt == t.dtype, "w_post, w_pre and gate must have one dtype")
        _need(name == "gate" or (t.shape == (H,) and t.is_contiguous()), name + ": expected a contiguous [H] tensor")
        pt = t.dtype
    return pt or dtype


def _gate_strides(gate, M, H):
    """(row, feature) element strides of a gate of shape [], [1], [H], [M, 1], [1, H] or [M, H]."""
    if gate is None:
        return 0, 0
    shape = tuple(gate.shape)
    shape = (1,) * (2 - len(shape)) + shape
    _need(len(shape) == 2 and shape[0] in (1, M) and shape[1] in (1, H), "gate: expected [], [1], [H], [M, 1] or [M, H]")
    rs = gate.stride(0) if shape[0] > 1 else 0
    cs = 1 if shape[1] > 1 else 0
    _need((rs > 0) == (shape[0] > 1) and (not cs or gate.stride(-1) == 1),
          "gate: an expanded gate is given in its own shape, with contiguous features")
    return rs, cs


def _ptr(t):
    return None if t is None else t.data_ptr()


def detffn_join_forward(x, z=None, w_post=None, gate=None, scale=1.0, w_pre=None, eps=1e-6, out=None, y=None,
                        stream=None):
    """The residual stream after a block, and the next block's normalised input:

        n = rmsnorm(z) * w_post (z itself without w_post)
        out = x + scale * gate * n;  y = rmsnorm(out) * w_pre

    Returns (out, y); y is None without w_pre, and out None without z (the
    norm before a block alone: y from x).  x, z [M, H] with any row stride;
    gate [], [1], [H], [M, 1] or [M, H]; w_post, w_pre [H].  out may be x."""
    ldx = _rows(x, "x")
    M, H = x.shape
    dt, dev = x.dtype, x.device
    ldz = 0 if z is None else _rows(z, "z", x.shape, dt, dev)
    pt = _params(dt, H, dev, w_post=w_post, w_pre=w_pre, gate=gate)
    rs, cs = _gate_strides(gate, M, H)
    on = _On(dev, stream)
    if z is not None and out is None:
        out = on.empty((M, H), dt)
    if w_pre is not None and y is None:
        y = on.empty((M, H), dt)
    ldo = 0 if out is None else _rows(out, "out", x.shape, dt, dev)
    ldy = 0 if y is None else _rows(y, "y", x.shape, dt, dev)
    with on.device():
        _call("detffn_join_forward", x.data_ptr(), ldx, _ptr(z), ldz, _ptr(w_post), _ptr(gate), rs, cs, scale,
              _ptr(w_pre), eps, _ptr(out), ldo, _ptr(y), ldy, M, H, _DTYPE[dt], _DTYPE[pt], on.raw)
    return out, y


class JoinGrads(NamedTuple):
    """Gradients of a residual join (None where the input was not given)."""
    dx: torch.Tensor
    dz: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]


def detffn_join_backward(r, z=None, dr=None, dy=None, w_post=None, gate=None, scale=1.0, w_pre=None, eps=1e-6,
                         dx=None, dz=None, ws=None, stream=None):
    """Gradients of detffn_join_forward from r, its out as stored (x where
    there was no z), the block output z, and the gradients dr of out and dy of
    y (one may be None: zero).  Without w_pre the residual's gradient dx is dr
    itself.  dx may be dr and dz may be z (in place)."""
    lead = r if r is not None else dr
    _need(lead is not None, "r or dr must be given")
    _need(w_pre is None or (r is not None and dy is not None), "w_pre: r and dy must be given")
    _need(w_pre is not None or (dy is None and dr is not None), "without w_pre: dr and no dy")
    _rows(lead, "r")
    M, H = lead.shape
    dt, dev = lead.dtype, lead.device
    ldr = 0 if r is None else r.stride(0)
    lddr = 0 if dr is None else _rows(dr, "dr", lead.shape, dt, dev)
    lddy = 0 if dy is None else _rows(dy, "dy", lead.shape, dt, dev)
    ldz = 0 if z is None else _rows(z, "z", lead.shape, dt, dev)
    pt = _params(dt, H, dev, w_post=w_post, w_pre=w_pre, gate=gate)
    rs, cs = _gate_strides(gate, M, H)
    on = _On(dev, stream)
    back = w_pre is not None
    if z is not None and dz is None:
        dz = on.empty((M, H), dt)
    if back and dx is None:
        dx = on.empty((M, H), dt)
    _need(back or dx is None or dx is dr, "without w_pre the gradient of x is dr itself")
    lddx = _rows(dx, "dx", lead.shape, dt, dev) if back else 0
    lddz = 0 if dz is None else _rows(dz, "dz", lead.shape, dt, dev)
    dgate = None if gate is None else on.empty(gate.shape, pt)
    dw_post = None if w_post is None else on.empty((H,), pt)
    dw_pre = None if w_pre is None else on.empty((H,), pt)
    if ws is None:
        ws = on.empty((detffn_join_workspace_size(M, H),), torch.uint8)
    with on.device():
        _call("detffn_join_backward", _ptr(r), ldr, _ptr(dr), lddr, _ptr(dy), lddy, _ptr(z), ldz, _ptr(w_post),
              _ptr(gate), rs, cs, scale, _ptr(w_pre), eps, _ptr(dx) if back else None, lddx, _ptr(dz), lddz,
              _ptr(dgate), _ptr(dw_post), _ptr(dw_pre), M, H, _DTYPE[dt], _DTYPE[pt], ws.data_ptr(), ws.numel(),
              on.raw)
    return JoinGrads(dx if back else dr, dz, dgate, dw_post, dw_pre)


def detffn_join_workspace_size(M, H):
    """Bytes of scratch detffn_join_backward needs."""
    n = _sz()
    _call("detffn_join_workspace_size", M, H, ctypes.byref(n))
    return max(n.value, 256)


class Ckpt8(NamedTuple):
    """Gate and up of a training forward in 8 bits: codes [M, I] (int8) and
    scales [M, ceil(I / 64)] (float32) of each."""
    gate_codes: torch.Tensor
    gate_scales: torch.Tensor
    up_codes: torch.Tensor
    up_scales: torch.Tensor


def _whole(t, name, dev, dtype=None, shape=None):
    _need(t.is_cuda and t.is_contiguous() and t.device == dev and (dtype is None or t.dtype == dtype) and
          (shape is None or t.shape == shape), name + ": expected a contiguous CUDA tensor of the call's shape and dtype")


def _ckpt(c):
    dev = c.gate_codes.device
    _need(c.gate_codes.dim() == 2, "checkpoint codes: expected [M, I]")
    M, I = c.gate_codes.shape
    s = (M, (I + 63) // 64)
    _whole(c.gate_codes, "gate_codes", dev, torch.int8)
    _whole(c.up_codes, "up_codes", dev, torch.int8, c.gate_codes.shape)
    _whole(c.gate_scales, "gate_scales", dev, torch.float32, s)
    _whole(c.up_scales, "up_scales", dev, torch.float32, s)
    return M, I, dev, [c.gate_codes.data_ptr(), c.gate_scales.data_ptr(), c.up_codes.data_ptr(), c.up_scales.data_ptr()]


def detffn_ckpt8_pack(gate, up, ckpt=None, stream=None):
    """gate and up [M, I] as an 8-bit checkpoint (``ckpt``: buffers to write)."""
    _need(gate.dim() == 2 and gate.dtype in _DTYPE, "gate: expected [M, I] in float32, float16 or bfloat16")
    dev = gate.device
    _whole(gate, "gate", dev)
    _whole(up, "up", dev, gate.dtype, gate.shape)
    M, I = gate.shape
    on = _On(dev, stream)
    if ckpt is None:
        s = (M, (I + 63) // 64)
        ckpt = Ckpt8(on.empty((M, I), torch.int8), on.empty(s, torch.float32), on.empty((M, I), torch.int8),
                     on.empty(s, torch.float32))
    cm, ci, cdev, ptrs = _ckpt(ckpt)
    _need((cm, ci, cdev) == (M, I, dev), "ckpt: expected buffers of gate's shape on its device")
    with on.device():
        _call("detffn_ckpt8_pack", gate.data_ptr(), up.data_ptr(), *ptrs, M, I, _DTYPE[gate.dtype], on.raw)
    return ckpt


def detffn_ckpt8_unpack(ckpt, gate=None, up=None, dtype=torch.bfloat16, stream=None):
    """(gate, up) [M, I] as the values a checkpoint stands for, in ``dtype``."""
    M, I, dev, ptrs = _ckpt(ckpt)
    _need(dtype in _DTYPE, "dtype: expected float32, float16 or bfloat16")
    on = _On(dev, stream)
    gate = on.empty((M, I), dtype) if gate is None else gate
    up = on.empty((M, I), dtype) if up is None else up
    _whole(gate, "gate", dev, dtype, ckpt.gate_codes.shape)
    _whole(up, "up", dev, dtype, ckpt.gate_codes.shape)
    with on.device():
        _call("detffn_ckpt8_unpack", *ptrs, gate.data_ptr(), up.data_ptr(), M, I, _DTYPE[dtype], on.raw)
    return gate, up


def detffn_ckpt8_silu_backward(dh, ckpt, dU=None, dG=None, h=None, stream=None):
    """The SiLU stage of the backward pass from a checkpoint: (dU, dG, h) in dh's dtype."""
    M, I, dev, ptrs = _ckpt(ckpt)
    _need(dh.dtype in _DTYPE, "dh: expected float32, float16 or bfloat16")
    _whole(dh, "dh", dev, None, ckpt.gate_codes.shape)
    on = _On(dev, stream)
    dU = on.empty((M, I), dh.dtype) if dU is None else dU
    dG = on.empty((M, I), dh.dtype) if dG is None else dG
    h = on.empty((M, I), dh.dtype) if h is None else h
    for name, t in (("dU", dU), ("dG", dG), ("h", h)):
        _whole(t, name, dev, dh.dtype, dh.shape)
    with on.device():
        _call("detffn_ckpt8_silu_backward", dh.data_ptr(), *ptrs, dU.data_ptr(), dG.data_ptr(), h.data_ptr(), M, I,
              _DTYPE[dh.dtype], on.raw)
    return dU, dG, h


_MOE_WS = {}


def detffn_moe_workspace_size(T, E, top_k, H, I, dtype=torch.bfloat16):
    """Bytes of scratch detffn_moe_forward needs."""
    key = (T, E, top_k, H, I, dtype)
    n = _MOE_WS.get(key)
    if n is None:
        v = _sz()
        _call("detffn_moe_workspace_size", T, E, top_k, H, I, _DTYPE[dtype], ctypes.byref(v))
        n = _MOE_WS[key] = max(v.value, 256)
    return n


def detffn_moe_forward(x, Wr, Wg, Wu, Wd, top_k, normalize=True, out=None, experts=None, weights=None, ws=None,
                       path=PATH_AUTO, stream=None, spin_limit=0, flags=0):
    """A mixture-of-experts layer for up to 64 tokens: x [T, H], router Wr
    [E, H], experts Wg, Wu [E, I, H] and Wd [E, H, I], top_k experts a token,
    their weights normalised over the chosen (or over all experts).  Returns
    (out [T, H], experts [T, top_k] int32, weights [T, top_k] float32)."""
    _need(x.dim() == 2 and Wr.dim() == 2 and Wg.dim() == 3 and x.dtype in _DTYPE, "expected x [T, H], Wr [E, H], Wg [E, I, H]")
    T, H = x.shape
    E, I = Wg.shape[0], Wg.shape[1]
    dt, dev = x.dtype, x.device
    _whole(x, "x", dev)
    _whole(Wr, "Wr", dev, dt, (E, H))
    _whole(Wg, "Wg", dev, dt, (E, I, H))
    _whole(Wu, "Wu", dev, dt, (E, I, H))
    _whole(Wd, "Wd", dev, dt, (E, H, I))
    on = _On(dev, stream)
    need = detffn_moe_workspace_size(T, E, top_k, H, I, dt)
    out = on.empty((T, H), dt) if out is None else out
    experts = on.empty((T, top_k), torch.int32) if experts is None else experts
    weights = on.empty((T, top_k), torch.float32) if weights is None else weights
    ws = on.empty((need,), torch.uint8) if ws is None else ws
    _whole(out, "out", dev, dt, (T, H))
    _whole(experts, "experts", dev, torch.int32, (T, top_k))
    _whole(weights, "weights", dev, torch.float32, (T, top_k))
    _call("detffn_moe_forward", _d.handle(dev), x.data_ptr(), Wr.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
          Wd.data_ptr(), out.data_ptr(), experts.data_ptr(), weights.data_ptr(), T, E, top_k, 1 if normalize else 0, H,
          I, _DTYPE[dt], ws.data_ptr(), ws.numel(), on.raw, _d._opts(path, 1, spin_limit, flags))
    return out, experts, weights
