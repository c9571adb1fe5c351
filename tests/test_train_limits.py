"""Ends of what the grouped products accept (no GPU compute): their C calls refuse
what their kernels cannot count, before anything is launched.  The pointers below
are made up and never read."""
import ctypes

import pytest

from tests.test_train_abi import _ARGS, BWD, FWD, OK, SHAPE, WORKSPACE, _sz


@pytest.fixture(scope="module")
def lib():
    from gemm_deterministic_bf16_gb300 import build, detffn
    build.build()
    for name, args in _ARGS.items():
        getattr(detffn.lib(), name).argtypes = args
    return detffn.lib()


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_rows_of_a_grouped_call(lib, dtype):
    """Rows are counted, and cut into tiles of up to 256, in 32-bit integers: R + 255 has to be one."""
    n, most = _sz(), (1 << 31) - 256
    assert lib.detffn_grouped_workspace_size(most, 1, 8, 8, dtype, ctypes.byref(n)) == OK
    for R in (most + 1, (1 << 31) - 1):
        assert lib.detffn_grouped_workspace_size(R, 1, 8, 8, dtype, ctypes.byref(n)) == SHAPE
        for f, kw in ((lib.detffn_grouped_forward, FWD), (lib.detffn_grouped_backward, BWD)):
            assert f(*dict(kw, R=R, E=1, K=9, N=8, dt=dtype, ws=None, n=0).values()) == SHAPE
    if dtype:   # (the largest is refused for its missing scratch alone)
        kw = dict(FWD, R=most, E=1, K=9, ldx=9, N=8, ldo=8, dt=dtype, ws=None, n=0)
        assert lib.detffn_grouped_forward(*kw.values()) == WORKSPACE
