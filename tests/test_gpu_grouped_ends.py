"""The products grouped by expert at the ends of what they accept: waits that run
out at any point."""
import pytest
import torch

from tests.test_gpu_grouped import G, TENSOR, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["forward", "dX", "dW"])
@pytest.mark.parametrize("sizes,K,N", [([100, 60], 256, 264), ([1, 0, 700], 1032, 520)], ids=str)
def test_waits_of_few_tries(G, sizes, K, N, what):
    """With limits that ordinary waits may well reach, at any point of a call, every call ends; the
    status says whether one ran out, and calls that did not are whole."""
    x, W, d, off, _ = make(sizes, K, N, torch.bfloat16)

    def go(**kw):
        if what == "forward":
            return G.detffn_grouped_forward(x, W, off, path=TENSOR, **kw)
        return next(t for t in G.detffn_grouped_backward(x, W, off, d, need_dX=what == "dX", need_dW=what == "dW", path=TENSOR,
                                                         **kw) if t is not None)
    want = go()
    for limit in (1, 1, 2, 3, 5, 8, 16, 64):
        got = go(spin_limit=limit)
        torch.cuda.synchronize()
        status = G.detffn_get_status()
        assert status in (0, 7)
        assert status == 7 or torch.equal(got, want)
        assert torch.equal(go(), want)
    assert G.detffn_get_status() == 0
