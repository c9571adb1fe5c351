"""Binding of the products grouped by expert, of the products with 4-bit weights
for a few tokens, and of dropout from a counter-based generator.

Each function has the name of the C call it wraps; the checks of the tensors, the
allocation of results and scratch, and the call itself are in the native half, as
in ``block.py``, whose remarks on errors and streams hold here too.
"""
import ctypes
from typing import NamedTuple

import torch

from . import block as _b
from . import detffn as _d
from .block import _CODE, _native, _on
from .detffn import PATH_AUTO


def _handle(t):
    h = _d._HANDLES.get(t.get_device()) if t.is_cuda else 0
    return _d.handle(t.device) if h is None else h


def detffn_grouped_workspace_size(R, E, K, N, dtype=torch.bfloat16):
    """Bytes of scratch the grouped products need."""
    f = _d.lib().detffn_grouped_workspace_size
    f.argtypes = [_d._ll] * 4 + [_d._int, ctypes.POINTER(ctypes.c_size_t)]
    n = ctypes.c_size_t()
    _d._check(f(R, E, K, N, _CODE[dtype], ctypes.byref(n)), "detffn_grouped_workspace_size")
    return n.value


def detffn_grouped_forward(x, W, offsets, out=None, ws=None, path=PATH_AUTO, stream=None, spin_limit=0, flags=0):
    """out[r] = W[e] x[r] for the rows offsets[e] <= r < offsets[e + 1] of each
    expert e: x [R, K] sorted by expert (any row stride), W [E, N, K], offsets
    int32 [E + 1] on the device, which no host waits for.  Returns out [R, N].
    Rows of no expert stay as they were in ``out`` (without it they hold
    whatever the memory held).  16-bit rows of a width that is a multiple of 8 run
    on the tensor cores only from 16-byte boundaries: a slice as wide[:, 1:] takes
    some thirty times as long where rows are many, a copy of it does not."""
    f = (_b._LIB or _native()).grouped_forward
    args = (_handle(x), x, W, offsets, out, ws, path, spin_limit, flags)
    return (f(*args) if stream is None else _on(stream, f, *args))[0]


def detffn_grouped_backward(x, W, offsets, dOut, dX=None, dW=None, need_dX=True, need_dW=True, ws=None, path=PATH_AUTO,
                            stream=None, spin_limit=0, flags=0):
    """Gradients of detffn_grouped_forward from dOut [R, N]: (dX [R, K], dW [E, N,
    K]), None for one that is not needed (x may be None without dW).  An expert
    without rows has a dW of zeros; rows of no expert stay as they were in dX.  One
    operand off the boundaries that detffn_grouped_forward names takes both gradients
    from the tensor cores."""
    f = (_b._LIB or _native()).grouped_backward
    args = (_handle(dOut), x, W, offsets, dOut, dX, dW, need_dX, need_dW, ws, path, spin_limit, flags)
    return f(*args) if stream is None else _on(stream, f, *args)


class W4(NamedTuple):
    """A matrix [N, K] in 4 bits: codes [N, 64 ceil(K / 128)] (uint8), scales [N,
    ceil(K / group)], and the K and group (32, 64 or 128) they are for.  The order
    of the codes is that of ``detffn_w4_pack`` in the header."""
    codes: torch.Tensor
    scales: torch.Tensor
    K: int
    group: int


def detffn_w4_pack(w, group=128, scale_dtype=None, w4=None, stream=None):
    """w [N, K] (any row stride) in 4 bits; scales in ``scale_dtype`` (w's own by
    default), or in the buffers of ``w4``."""
    f = (_b._LIB or _native()).w4_pack
    if w4 is not None and (w4.K != w.shape[-1] or w4.group != group):
        raise ValueError("w4: expected buffers of w's K and group")
    st = scale_dtype or (w4.scales.dtype if w4 is not None else w.dtype)
    args = (w, group, _CODE.get(st, -1), *(w4[:2] if w4 is not None else (None, None)))
    return W4(*(f(*args) if stream is None else _on(stream, f, *args)), w.shape[1], group)


def detffn_w4_unpack(w4, out=None, dtype=torch.bfloat16, stream=None):
    """The values [N, K] of a 4-bit matrix, FP32 products rounded to ``dtype`` (out's where it is given)."""
    f = (_b._LIB or _native()).w4_unpack
    args = (*w4, _CODE.get(dtype if out is None else out.dtype, -1), out)
    return (f(*args) if stream is None else _on(stream, f, *args))[0]


def detffn_w4_matvec_workspace_size(T, K, dtype=torch.bfloat16):
    """Bytes of scratch detffn_w4_matvec needs where x is FP32 or not on 16-byte boundaries."""
    f = _d.lib().detffn_w4_matvec_workspace_size
    f.argtypes = [_d._ll] * 2 + [_d._int, ctypes.POINTER(ctypes.c_size_t)]
    n = ctypes.c_size_t()
    _d._check(f(T, K, _CODE[dtype], ctypes.byref(n)), "detffn_w4_matvec_workspace_size")
    return max(n.value, 256)


def detffn_w4_matvec(x, w4, out=None, ws=None, stream=None):
    """x [T, K] times the transpose of a 4-bit matrix [N, K], for up to 64 tokens: [T, N]."""
    f = (_b._LIB or _native()).w4_matvec
    if stream is None:
        return f(x, *w4, out, ws)[0]
    return _on(stream, f, x, *w4, out, ws)[0]


def detffn_w4_workspace_size(T, H, I, dtype=torch.bfloat16):
    """Bytes of scratch detffn_w4_forward needs."""
    f = _d.lib().detffn_w4_workspace_size
    f.argtypes = [_d._ll] * 3 + [_d._int, ctypes.POINTER(ctypes.c_size_t)]
    n = ctypes.c_size_t()
    _d._check(f(T, H, I, _CODE[dtype], ctypes.byref(n)), "detffn_w4_workspace_size")
    return max(n.value, 256)


def detffn_w4_forward(x, Wg, Wu, Wd, out=None, ws=None, stream=None):
    """The gated FFN of up to 64 tokens x [T, H] from 4-bit matrices, Wg and Wu [I,
    H], Wd [H, I], of one group and scale dtype; returns out [T, H].  out may be x."""
    f = (_b._LIB or _native()).w4_forward
    args = (x, *Wg, *Wu, *Wd, out, ws)
    return (f(*args) if stream is None else _on(stream, f, *args))[0]


def detffn_dropout_forward(x, p, seed, offset=0, residual=None, out=None, stream=None):
    """residual + x / (1 - p) where an element is kept, residual (or 0) elsewhere: x
    [M, H] with any row stride.  The mask follows from (seed, offset) and an
    element's row and column alone, so nothing is stored for the backward pass; a
    program takes another offset for each call.  ``seed`` may be an int64 CUDA
    tensor (seed, base), read when the kernel runs, base added to offset: a
    captured step draws new masks when it is changed between replays.  out may be
    x or the residual."""
    f = (_b._LIB or _native()).dropout
    if stream is None:
        return f(x, p, seed, offset, residual, out, False)[0]
    return _on(stream, f, x, p, seed, offset, residual, out, False)[0]


def detffn_dropout_backward(dOut, p, seed, offset=0, dX=None, stream=None):
    """The gradient of x: dOut / (1 - p) where the forward's same p, seed and offset
    kept an element, 0 elsewhere (the residual's is dOut itself).  dX may be dOut."""
    f = (_b._LIB or _native()).dropout
    if stream is None:
        return f(dOut, p, seed, offset, None, dX, True)[0]
    return _on(stream, f, dOut, p, seed, offset, None, dX, True)[0]
