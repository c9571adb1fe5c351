"""Binding of the operators around the FFN: the residual join with its norms,
8-bit activation checkpoints, and the mixture-of-experts layer for a few
tokens.

Each function has the name of the C call it wraps.  The checks of the tensors,
the allocation of results and scratch, and the call itself are in the native
half, ``csrc/bind.cpp``: these calls are made on a few kilobytes too, and take
there what they would cost in Python several times over.  Tensors that do not
fit raise ``ValueError``, a non-OK status ``DetFFNError``.

With a ``stream`` other than the current one, what a call allocates comes from
that stream's pool, and what it returns is marked as used by the current
stream too; the inputs' own streams are the caller's to order.
"""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import detffn as _d
from .detffn import BF16, F16, F32, PATH_AUTO

_CODE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_LIB = None


def _native():
    """The native half; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        _d.lib()
        from . import _native as n
        n.set_error(_d.DetFFNError)
        _LIB = n
    return _LIB


def _on(stream, f, *args):
    """f(*args) with `stream` as the current one."""
    now = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        got = f(*args)
    for t in got:
        if t is not None:
            t.record_stream(now)
    return got


def detffn_join_forward(x, z=None, w_post=None, gate=None, scale=1.0, w_pre=None, eps=1e-6, out=None, y=None,
                        stream=None):
    """The residual stream after a block, and the next block's normalised input:

        n = rmsnorm(z) * w_post (z itself without w_post)
        out = x + scale * gate * n;  y = rmsnorm(out) * w_pre

    Returns (out, y); y is None without w_pre, and out None without z (the
    norm before a block alone: y from x).  x, z [M, H] with any row stride;
    gate [], [1], [H], [M, 1] or [M, H]; w_post, w_pre [H].  out may be x."""
    f = (_LIB or _native()).join_forward
    if stream is None:
        return f(x, z, w_post, gate, scale, w_pre, eps, out, y)
    return _on(stream, f, x, z, w_post, gate, scale, w_pre, eps, out, y)


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
    y (dr may be None, zero, where dy is given; dy goes with w_pre).  Without
    w_pre the residual's gradient dx is dr itself.  dx may be dr and dz may be z (in place)."""
    f = (_LIB or _native()).join_backward
    if stream is None:
        return JoinGrads(*f(r, z, dr, dy, w_post, gate, scale, w_pre, eps, dx, dz, ws))
    return JoinGrads(*_on(stream, f, r, z, dr, dy, w_post, gate, scale, w_pre, eps, dx, dz, ws))


def detffn_join_workspace_size(M, H):
    """Bytes of scratch detffn_join_backward needs."""
    f = _d.lib().detffn_join_workspace_size
    f.argtypes = [_d._ll, _d._ll, ctypes.POINTER(ctypes.c_size_t)]
    n = ctypes.c_size_t()
    _d._check(f(M, H, ctypes.byref(n)), "detffn_join_workspace_size")
    return max(n.value, 256)


class Ckpt8(NamedTuple):
    """Gate and up of a training forward in 8 bits: codes [M, I] (int8) and
    scales [M, ceil(I / 64)] (float32) of each."""
    gate_codes: torch.Tensor
    gate_scales: torch.Tensor
    up_codes: torch.Tensor
    up_scales: torch.Tensor


def detffn_ckpt8_pack(gate, up, ckpt=None, stream=None):
    """gate and up [M, I] as an 8-bit checkpoint (``ckpt``: buffers to write)."""
    f = (_LIB or _native()).ckpt8_pack
    to = (None, None, None, None) if ckpt is None else ckpt
    if stream is None:
        return Ckpt8(*f(gate, up, *to))
    return Ckpt8(*_on(stream, f, gate, up, *to))


def detffn_ckpt8_unpack(ckpt, gate=None, up=None, dtype=torch.bfloat16, stream=None):
    """(gate, up) [M, I] as the values a checkpoint stands for, in ``dtype``."""
    f = (_LIB or _native()).ckpt8_unpack
    code = _CODE.get(dtype, -1)
    if stream is None:
        return f(*ckpt, gate, up, code)
    return _on(stream, f, *ckpt, gate, up, code)


def detffn_ckpt8_silu_backward(dh, ckpt, dU=None, dG=None, h=None, stream=None):
    """The SiLU stage of the backward pass from a checkpoint: (dU, dG, h) in dh's dtype."""
    f = (_LIB or _native()).ckpt8_silu_backward
    if stream is None:
        return f(*ckpt, dh, dU, dG, h)
    return _on(stream, f, *ckpt, dh, dU, dG, h)


def detffn_backward_ckpt8(x, Wg, Wu, Wd, ckpt, dOut, dX=None, dWg=None, dWu=None, dWd=None, ws=None, shards=1,
                          path=PATH_AUTO, stream=None, spin_limit=0, flags=0):
    """detffn_backward with gate and up from an 8-bit checkpoint; returns (dX, dWg, dWu, dWd)."""
    if stream is not None:
        return _on(stream, detffn_backward_ckpt8, x, Wg, Wu, Wd, ckpt, dOut, dX, dWg, dWu, dWd, ws, shards, path, None,
                   spin_limit, flags)
    _d._bf16(x, Wg, Wu, Wd, dOut, dX, dWg, dWu, dWd)
    if len(x.shape) != 2 or len(Wg.shape) != 2:
        raise ValueError("expected x [M, H] and Wg [I, H]")
    M, H = x.shape
    I = Wg.shape[0]
    # The C call sees addresses only, so every extent is checked here.
    for name, t, s in (("Wg", Wg, (I, H)), ("Wu", Wu, (I, H)), ("Wd", Wd, (H, I)), ("dOut", dOut, (M, H)),
                       ("dX", dX, (M, H)), ("dWg", dWg, (I, H)), ("dWu", dWu, (I, H)), ("dWd", dWd, (H, I))):
        if t is not None and (tuple(t.shape) != s or t.device != x.device):
            raise ValueError("%s: expected %s on the device of x" % (name, list(s)))
    for t, dt, n in zip(ckpt, (torch.int8, torch.float32) * 2, (I, (I + 63) // 64) * 2):
        if t.dtype != dt or tuple(t.shape) != (M, n) or not t.is_contiguous() or t.device != x.device:
            raise ValueError("checkpoint: expected contiguous CUDA codes [M, I] (int8) and scales [M, ceil(I / 64)] (float32)")
    if ws is not None and (ws.device != x.device or not ws.is_contiguous()):
        raise ValueError("ws: expected a contiguous buffer on the device of x")
    e = lambda t, *s: torch.empty(s, dtype=torch.bfloat16, device=x.device) if t is None else t  # noqa: E731
    dX, dWg, dWu, dWd = e(dX, M, H), e(dWg, I, H), e(dWu, I, H), e(dWd, H, I)
    if ws is None:
        ws = _d.workspace(_d.OP_BACKWARD, M, H, I, shards, path, x.device)
    f = _d.lib().detffn_backward_ckpt8
    f.argtypes = [_d._vp] * 14 + [_d._ll] * 3 + [_d._vp, ctypes.c_size_t, _d._vp, ctypes.POINTER(_d.Options)]
    p = [t.data_ptr() for t in (x, Wg, Wu, Wd, *ckpt, dOut, dX, dWg, dWu, dWd)]
    _d._check(f(_d.handle(x.device), *p, M, H, I, ws.data_ptr(), ws.numel() * ws.element_size(),
                torch.cuda.current_stream(x.device).cuda_stream, _d._opts(path, shards, spin_limit, flags)),
              "detffn_backward_ckpt8")
    return dX, dWg, dWu, dWd


def detffn_moe_workspace_size(T, E, top_k, H, I, dtype=torch.bfloat16):
    """Bytes of scratch detffn_moe_forward needs."""
    f = _d.lib().detffn_moe_workspace_size
    f.argtypes = [_d._ll, _d._ll, _d._int, _d._ll, _d._ll, _d._int, ctypes.POINTER(ctypes.c_size_t)]
    n = ctypes.c_size_t()
    _d._check(f(T, E, top_k, H, I, _CODE[dtype], ctypes.byref(n)), "detffn_moe_workspace_size")
    return max(n.value, 256)


def detffn_moe_forward(x, Wr, Wg, Wu, Wd, top_k, normalize=True, out=None, experts=None, weights=None, ws=None,
                       path=PATH_AUTO, stream=None, spin_limit=0, flags=0):
    """A mixture-of-experts layer for up to 64 tokens: x [T, H], router Wr
    [E, H], experts Wg, Wu [E, I, H] and Wd [E, H, I], top_k experts a token,
    their weights normalised over the chosen (or over all experts).  Returns
    (out [T, H], experts [T, top_k] int32, weights [T, top_k] float32)."""
    f = (_LIB or _native()).moe_forward
    handle = _d._HANDLES.get(x.get_device()) if x.is_cuda else 0
    if handle is None:
        handle = _d.handle(x.device)
    if stream is None:
        return f(handle, x, Wr, Wg, Wu, Wd, top_k, normalize, out, experts, weights, ws, path, spin_limit, flags)
    return _on(stream, f, handle, x, Wr, Wg, Wu, Wd, top_k, normalize, out, experts, weights, ws, path, spin_limit, flags)
