"""Host-side checks of the operators around the FFN (no GPU compute): their C
calls refuse bad arguments before anything is launched, and size their
workspaces.  The pointers below are made up and never read."""
import ctypes

import pytest
import torch

F32, F16, BF16 = 0, 1, 2
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = range(6)
A = [1 << 30, 2 << 30, 3 << 30, 4 << 30, 5 << 30, 6 << 30, 7 << 30, 8 << 30, 9 << 30, 10 << 30]


_vp, _ll, _int, _f, _sz = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
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
                                       _vp],
}


@pytest.fixture(scope="module")
def call():
    from gemm_deterministic_bf16_gb300 import build, detffn
    build.build()

    def go(name, *args):
        f = getattr(detffn.lib(), name)
        f.argtypes = _ARGS[name]
        return f(*args)
    return go


def fwd(call, **kw):
    a = dict(x=A[0], ldx=64, z=A[1], ldz=64, w_post=A[2], gate=A[3], rs=0, cs=1, scale=1.0, w_pre=A[4], eps=1e-6,
             out=A[5], ldo=64, y=A[6], ldy=64, M=4, H=64, dt=BF16, pt=F32)
    a.update(kw)
    return call("detffn_join_forward", *a.values(), None)


def test_join_forward_refusals(call):
    assert fwd(call, M=0) == OK                                   # nothing to do: nothing is launched
    assert fwd(call, M=0, x=None, z=None, w_post=None, gate=None, w_pre=None, out=None, y=None) == OK
    for bad in (dict(dt=3), dict(pt=-1), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(x=None), dict(out=None), dict(y=None), dict(w_pre=None), dict(z=None), dict(cs=2), dict(rs=-1),
                dict(z=None, w_post=None, gate=None), dict(z=None, w_post=None, gate=None, out=None, w_pre=None, y=None),
                dict(y=A[5]), dict(out=A[1]), dict(out=A[0] + 2), dict(out=A[2]), dict(y=A[0]), dict(y=A[3]),
                dict(out=A[0], ldo=72)):
        assert fwd(call, **bad) == INVALID, bad
    for bad in (dict(M=-1), dict(H=0), dict(H=32769), dict(ldx=63), dict(ldy=10), dict(rs=32, cs=1)):
        assert fwd(call, **bad) == SHAPE, bad
    for bad in (dict(x=A[0] + 1), dict(z=A[1] + 1), dict(w_pre=A[4] + 2), dict(gate=A[3] + 1), dict(out=A[5] + 1)):
        assert fwd(call, **bad) == ALIGN, bad
    assert fwd(call, dt=BF16, pt=F16) == UNSUPPORTED
    assert fwd(call, dt=F32, pt=BF16) == UNSUPPORTED


def test_interleaved_halves_are_told_from_overlaps(call):
    """out and y as the column halves of one buffer share no byte; the checks
    pass them, and the call stops at the next refusal (a misaligned gate)."""
    half = dict(out=A[5], ldo=128, y=A[5] + 128, ldy=128)
    assert fwd(call, gate=A[3] + 1, **half) == ALIGN
    assert fwd(call, out=A[5], ldo=128, y=A[5] + 126, ldy=128) == INVALID
    assert fwd(call, out=A[5] + 128, ldo=128, y=A[5] + 2, ldy=128) == INVALID


def bwd(call, **kw):
    a = dict(r=A[0], ldr=64, dr=A[1], lddr=64, dy=A[2], lddy=64, z=A[3], ldz=64, w_post=A[4], gate=A[5], rs=0, cs=1,
             scale=1.0, w_pre=A[6], eps=1e-6, dx=A[7], lddx=64, dz=A[8], lddz=64, dgate=A[9], dw_post=A[9] + 4096,
             dw_pre=A[9] + 8192, M=4, H=64, dt=BF16, pt=F32, ws=A[9] + 65536, n=1 << 20)
    a.update(kw)
    return call("detffn_join_backward", *a.values(), None)


def test_join_backward_refusals(call):
    for bad in (dict(dx=None), dict(r=None), dict(dy=None), dict(dw_pre=None), dict(dw_post=None), dict(dgate=None),
                dict(w_pre=None), dict(w_pre=None, dw_pre=None, dx=None), dict(z=None), dict(dz=None), dict(eps=-1.0),
                dict(dx=A[8]), dict(dz=A[0]), dict(dw_pre=A[9]), dict(dgate=A[4]), dict(dx=A[0]), dict(dw_post=A[9] + 65536)):
        assert bwd(call, **bad) == INVALID, bad
    assert bwd(call, H=0) == SHAPE and bwd(call, lddz=1) == SHAPE
    assert bwd(call, dx=A[7] + 1) == ALIGN and bwd(call, dw_pre=A[9] + 8194) == ALIGN
    for bad in (dict(ws=None), dict(ws=A[9] + 65540), dict(n=100)):
        assert bwd(call, **bad) == WORKSPACE, bad


def test_ckpt_refusals(call):
    a = [A[0], A[1], A[2], A[3], A[4], A[5], 4, 64, BF16, None]
    for name in ("detffn_ckpt8_pack", "detffn_ckpt8_unpack"):
        assert call(name, *a[:6], 0, 64, BF16, None) == OK
        assert call(name, *a[:6], 4, 64, 5, None) == INVALID
        assert call(name, *a[:6], -1, 64, BF16, None) == SHAPE
        assert call(name, *a[:6], 4, 0, BF16, None) == SHAPE
        for i in range(6):
            assert call(name, *(None if j == i else p for j, p in enumerate(a[:6])), 4, 64, BF16, None) == INVALID
    assert call("detffn_ckpt8_pack", A[0] + 1, *a[1:]) == ALIGN
    assert call("detffn_ckpt8_pack", *a[:3], A[3] + 2, *a[4:]) == ALIGN
    assert call("detffn_ckpt8_pack", A[0], A[1], A[0] + 8, *a[3:]) == INVALID
    b = [A[0], A[1], A[2], A[3], A[4], A[5], A[6], A[7], 4, 64, BF16, None]
    assert call("detffn_ckpt8_silu_backward", None, *b[1:]) == INVALID
    assert call("detffn_ckpt8_silu_backward", *b[:5], A[0], *b[6:]) == INVALID
    assert call("detffn_ckpt8_silu_backward", *b[:6], A[6] + 1, *b[7:]) == ALIGN


def test_workspace_sizes(call):
    n = ctypes.c_size_t()
    assert call("detffn_join_workspace_size", 16384, 4096, ctypes.byref(n)) == OK and n.value >= 152 * (3 * 4096 + 1) * 4
    big = n.value
    assert call("detffn_join_workspace_size", 1, 4096, ctypes.byref(n)) == OK and n.value < big
    assert call("detffn_join_workspace_size", 1, 40000, ctypes.byref(n)) == SHAPE
    assert call("detffn_join_workspace_size", 1, 64, None) == INVALID
    assert call("detffn_moe_workspace_size", 64, 128, 8, 4096, 1536, BF16, ctypes.byref(n)) == OK
    assert n.value >= 64 * 8 * 1536 * 2
    for T, E, k, H, I in ((65, 8, 2, 64, 64), (1, 0, 1, 64, 64), (1, 513, 1, 64, 64), (1, 8, 9, 64, 64),
                          (1, 32, 17, 64, 64), (1, 8, 0, 64, 64), (1, 8, 2, 0, 64), (1, 8, 2, 64, 1 << 17), (-1, 8, 2, 64, 64)):
        assert call("detffn_moe_workspace_size", T, E, k, H, I, BF16, ctypes.byref(n)) == SHAPE
    assert call("detffn_moe_workspace_size", 1, 8, 2, 64, 64, 4, ctypes.byref(n)) == INVALID


def test_moe_without_a_handle(call):
    assert call("detffn_moe_forward", None, *A[:8], 1, 8, 2, 1, 64, 64, BF16, A[8], 1 << 20, None, None) == INVALID


class _OnGpu:
    """What a contiguous CUDA tensor shows to the checks; it has no memory."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.bfloat16, device="cuda:0"):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)

    def is_contiguous(self):
        return True


@pytest.mark.parametrize("bad", [
    dict(Wu=_OnGpu((128, 256))), dict(Wu=_OnGpu((256, 192))), dict(Wd=_OnGpu((192, 256))), dict(Wd=_OnGpu((256, 128))),
    dict(dOut=_OnGpu((4, 256))), dict(dOut=_OnGpu((8, 192))), dict(dOut=_OnGpu((8 * 256,))), dict(dX=_OnGpu((4, 256))),
    dict(dWg=_OnGpu((128, 256))), dict(dWu=_OnGpu((192, 255))), dict(dWd=_OnGpu((192, 256))), dict(x=_OnGpu((2, 4, 256))),
    dict(x=_OnGpu((8 * 256,))), dict(Wg=_OnGpu((192,))), dict(Wg=_OnGpu((192, 128))), dict(Wu=_OnGpu((192, 256), device="cuda:1")),
    dict(dOut=_OnGpu((8, 256), device="cuda:1")), dict(dWd=_OnGpu((256, 192), device="cuda:1")),
    dict(ws=_OnGpu((1 << 30,), torch.uint8, "cuda:1")), dict(ws=_OnGpu((1 << 30,), torch.uint8, "cpu")),
    dict(gate_codes=_OnGpu((4, 192), torch.int8)), dict(up_scales=_OnGpu((8, 4), torch.float32)),
    dict(up_codes=_OnGpu((8, 192), torch.int8, "cuda:1"))])
def test_backward_ckpt8_checks_every_extent(monkeypatch, bad):
    """Tensors whose extents do not fit are refused before any address is taken."""
    from gemm_deterministic_bf16_gb300 import block, detffn

    def reached(*_):
        raise AssertionError("the call went past its checks")
    for name in ("lib", "handle", "workspace"):
        monkeypatch.setattr(detffn, name, reached)
    M, H, I = 8, 256, 192
    t = dict(x=_OnGpu((M, H)), Wg=_OnGpu((I, H)), Wu=_OnGpu((I, H)), Wd=_OnGpu((H, I)), dOut=_OnGpu((M, H)),
             dX=_OnGpu((M, H)), dWg=_OnGpu((I, H)), dWu=_OnGpu((I, H)), dWd=_OnGpu((H, I)), ws=None)
    c = dict(gate_codes=_OnGpu((M, I), torch.int8), gate_scales=_OnGpu((M, 3), torch.float32),
             up_codes=_OnGpu((M, I), torch.int8), up_scales=_OnGpu((M, 3), torch.float32))
    with pytest.raises(AssertionError):   # what fits gets there
        block.detffn_backward_ckpt8(ckpt=block.Ckpt8(**c), **t)
    (t if next(iter(bad)) in t else c).update(bad)
    with pytest.raises(ValueError):
        block.detffn_backward_ckpt8(ckpt=block.Ckpt8(**c), **t)
