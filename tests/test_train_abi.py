"""Host-side checks of the grouped products, the 4-bit products and dropout (no
GPU compute): their C calls refuse bad arguments before anything is launched.
The pointers below are made up and never read."""
import ctypes

import pytest

F32, F16, BF16 = 0, 1, 2
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = range(6)
A = [i << 30 for i in range(1, 12)]
_vp, _ll, _int, _sz, _u64 = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_size_t, ctypes.c_ulonglong
_ARGS = {
    "detffn_grouped_workspace_size": [_ll] * 4 + [_int, ctypes.POINTER(_sz)],
    "detffn_grouped_forward": [_vp, _vp, _ll, _vp, _vp, _vp, _ll, _ll, _ll, _ll, _ll, _int, _vp, _sz, _vp, _vp],
    "detffn_grouped_backward": [_vp, _vp, _ll, _vp, _vp, _vp, _ll, _vp, _ll, _vp, _ll, _ll, _ll, _ll, _int, _vp, _sz,
                                _vp, _vp],
    "detffn_w4_pack": [_vp, _ll, _vp, _vp, _ll, _ll, _int, _int, _int, _vp],
    "detffn_w4_unpack": [_vp, _vp, _vp, _ll, _ll, _ll, _int, _int, _int, _vp],
    "detffn_w4_matvec_workspace_size": [_ll, _ll, _int, ctypes.POINTER(_sz)],
    "detffn_w4_matvec": [_vp, _ll, _vp, _vp, _vp, _ll, _ll, _ll, _ll, _int, _int, _int, _vp, _sz, _vp],
    "detffn_w4_workspace_size": [_ll, _ll, _ll, _int, ctypes.POINTER(_sz)],
    "detffn_w4_forward": [_vp, _ll] + [_vp] * 7 + [_ll, _ll, _ll, _ll, _int, _int, _int, _vp, _sz, _vp],
    "detffn_dropout_forward": [_vp, _ll, _vp, _ll, _vp, _ll, ctypes.c_double, _u64, _u64, _vp, _ll, _ll, _int, _vp],
    "detffn_dropout_backward": [_vp, _ll, _vp, _ll, ctypes.c_double, _u64, _u64, _vp, _ll, _ll, _int, _vp],
}


@pytest.fixture(scope="module")
def call():
    from gemm_deterministic_bf16_gb300 import build, detffn
    build.build()

    def go(name, kw, **over):
        assert set(over) <= set(kw), over
        f = getattr(detffn.lib(), name)
        f.argtypes = _ARGS[name]
        return f(*dict(kw, **over).values())
    return go


# (A made-up handle: every refusal below comes before it is used.)
FWD = dict(h=A[10], x=A[0], ldx=64, W=A[1], off=A[2], out=A[3], ldo=32, R=16, E=2, K=64, N=32, dt=BF16, ws=A[5], n=1 << 29,
           stream=None, o=None)
BWD = dict(h=A[10], x=A[0], ldx=64, W=A[1], off=A[2], d=A[3], ldd=32, dX=A[4], lddx=64, dW=A[5], R=16, E=2, K=64, N=32,
           dt=BF16, ws=A[6], n=1 << 29, stream=None, o=None)


def test_grouped_refusals(call):
    for name, kw, out in (("detffn_grouped_forward", FWD, "out"), ("detffn_grouped_backward", BWD, "dX")):
        for bad in (dict(h=None), dict(dt=3), dict(off=None), {out: A[2]}):
            assert call(name, kw, **bad) == INVALID, (name, bad)
        for bad in (dict(R=-1), dict(R=1 << 31), dict(E=0), dict(E=1025), dict(K=0), dict(N=65537), dict(ldx=63)):
            assert call(name, kw, **bad) == SHAPE, (name, bad)
        for bad in (dict(x=A[0] + 1), dict(W=A[1] + 1), dict(off=A[2] + 2), {out: kw[out] + 1}):
            assert call(name, kw, **bad) == ALIGN, (name, bad)
    assert call("detffn_grouped_forward", FWD, R=0, x=None, out=None, off=None, W=None) == OK
    for bad in (dict(x=None), dict(W=None), dict(out=None), dict(out=A[0]), dict(out=A[1] + 4096 - 2)):
        assert call("detffn_grouped_forward", FWD, **bad) == INVALID, bad
    for bad in (dict(d=None), dict(dX=None, dW=None), dict(x=None), dict(W=None), dict(dX=A[3]), dict(dW=A[1]), dict(dX=A[5])):
        assert call("detffn_grouped_backward", BWD, **bad) == INVALID, bad
    n = _sz(7)
    assert call("detffn_grouped_workspace_size", dict(R=16, E=2, K=64, N=32, dt=BF16, n=ctypes.byref(n))) == OK and n.value == 0
    assert call("detffn_grouped_workspace_size", dict(R=16, E=2, K=63, N=32, dt=BF16, n=ctypes.byref(n))) == OK
    assert n.value >= (16 + 2 * 32) * 64 * 2
    for name, kw in (("detffn_grouped_forward", FWD), ("detffn_grouped_backward", BWD)):
        for bad in (dict(ws=None), dict(ws=kw["ws"] + 128), dict(n=n.value - 1)):
            assert call(name, kw, K=63, **bad) == WORKSPACE, bad
    assert call("detffn_grouped_workspace_size", dict(R=16, E=0, K=64, N=32, dt=BF16, n=ctypes.byref(n))) == SHAPE


PACK = dict(w=A[0], ldw=200, codes=A[1], scales=A[2], N=8, K=200, group=64, dt=BF16, st=F32, stream=None)
UNPACK = dict(codes=A[1], scales=A[2], w=A[0], ldw=200, N=8, K=200, group=64, dt=BF16, st=F32, stream=None)
MV = dict(x=A[0], ldx=200, codes=A[1], scales=A[2], out=A[3], ldo=8, T=4, N=8, K=200, group=64, dt=BF16, st=F32,
          ws=None, n=0, stream=None)
W4F = dict(x=A[0], ldx=200, gc=A[1], gs=A[2], uc=A[3], us=A[4], dc=A[5], ds=A[6], out=A[7], ldo=200, T=4, H=200, I=96,
           group=64, dt=BF16, st=F32, ws=A[8], n=1 << 20, stream=None)


def test_w4_refusals(call):
    for name, kw in (("detffn_w4_pack", PACK), ("detffn_w4_unpack", UNPACK), ("detffn_w4_matvec", MV)):
        for bad in (dict(dt=3), dict(st=-1), dict(codes=None), dict(scales=None)):
            assert call(name, kw, **bad) == INVALID, (name, bad)
        for bad in (dict(N=0), dict(K=0), dict(K=(1 << 20) + 1)):
            assert call(name, kw, **bad) == SHAPE, (name, bad)
        for bad in (dict(codes=A[1] + 8), dict(scales=A[2] + 2)):
            assert call(name, kw, **bad) == ALIGN, (name, bad)
        for g in (0, 16, 96, 256):
            assert call(name, kw, group=g) == UNSUPPORTED
    assert call("detffn_w4_pack", PACK, w=None) == INVALID and call("detffn_w4_pack", PACK, codes=A[0] + 16) == INVALID
    assert call("detffn_w4_pack", PACK, ldw=199) == SHAPE and call("detffn_w4_pack", PACK, w=A[0] + 1) == ALIGN
    assert call("detffn_w4_unpack", UNPACK, w=A[2] + 4) == INVALID
    for bad in (dict(T=65), dict(T=-1), dict(ldx=100), dict(ldo=7)):
        assert call("detffn_w4_matvec", MV, **bad) == SHAPE, bad
    assert call("detffn_w4_matvec", MV, T=0, x=None, out=None, codes=None, scales=None) == OK
    assert call("detffn_w4_matvec", MV, out=A[0] + 2) == INVALID and call("detffn_w4_matvec", MV, x=None) == INVALID
    for odd in (dict(x=A[0] + 2), dict(K=199), dict(ldx=201), dict(dt=F32)):   # rows that are laid out first need scratch
        assert call("detffn_w4_matvec", MV, **odd) == WORKSPACE, odd
        assert call("detffn_w4_matvec", MV, ws=A[5], n=1023, **odd) == WORKSPACE, odd
        assert call("detffn_w4_matvec", MV, ws=A[1], n=1 << 20, **odd) == INVALID, odd
    for bad in (dict(ws=None), dict(ws=A[8] + 128), dict(n=4 * 96 * 4 - 1)):
        assert call("detffn_w4_forward", W4F, **bad) == WORKSPACE, bad
    for bad in (dict(uc=None), dict(ds=None), dict(out=A[5]), dict(out=A[0] + 2), dict(ws=A[7]), dict(dt=9)):
        assert call("detffn_w4_forward", W4F, **bad) == INVALID, bad
    assert call("detffn_w4_forward", W4F, T=0, ws=None) == OK and call("detffn_w4_forward", W4F, I=0) == SHAPE
    n = _sz()
    assert call("detffn_w4_workspace_size", dict(T=4, H=200, I=96, dt=BF16, n=ctypes.byref(n))) == OK and n.value >= 4 * 96 * 4
    assert call("detffn_w4_workspace_size", dict(T=65, H=200, I=96, dt=BF16, n=ctypes.byref(n))) == SHAPE


DROP = dict(x=A[0], ldx=64, res=A[1], ldr=64, out=A[2], ldo=64, p=0.1, seed=1, offset=0, state=None, M=4, H=64, dt=BF16,
            stream=None)


def test_dropout_refusals(call):
    name = "detffn_dropout_forward"
    for bad in (dict(dt=3), dict(p=-0.5), dict(p=1.5), dict(p=float("nan")), dict(x=None), dict(out=None), dict(out=A[0] + 2),
                dict(out=A[1] + 128), dict(out=A[0], ldo=72), dict(state=A[2] + 8)):
        assert call(name, DROP, **bad) == INVALID, bad
    for bad in (dict(M=-1), dict(H=0), dict(ldx=63), dict(ldr=1), dict(ldo=2)):
        assert call(name, DROP, **bad) == SHAPE, bad
    for bad in (dict(x=A[0] + 1), dict(res=A[1] + 1), dict(out=A[2] + 1), dict(state=A[3] + 4)):
        assert call(name, DROP, **bad) == ALIGN, bad
    assert call(name, DROP, M=0, x=None, out=None) == OK
    back = dict(d=A[0], ldd=64, dX=A[1], lddx=64, p=0.1, seed=1, offset=0, state=None, M=4, H=64, dt=BF16, stream=None)
    assert call("detffn_dropout_backward", back, dX=A[0] + 2) == INVALID
    assert call("detffn_dropout_backward", back, M=0) == OK
