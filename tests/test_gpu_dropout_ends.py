"""Dropout with p = 1 and p = 0 where rows are far apart or many."""
import pytest
import torch

from tests.test_gpu_dropout import G  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p", [1.0, 0.0])
@pytest.mark.parametrize("dtype,step", [(torch.bfloat16, (1 << 30) + 8), (torch.float32, (1 << 29) + 4), (torch.bfloat16, (1 << 30) - 8)])
def test_rows_far_apart(G, dtype, step, p):
    """Rows 2 GiB and more apart, as any stride is accepted."""
    M, H = 3, 40
    far = torch.zeros((M - 1) * step + H, dtype=dtype, device="cuda").as_strided((M, H), (step, 1))
    x, r = (torch.randn((M, H), device="cuda").to(dtype) for _ in range(2))
    zero = torch.zeros_like(x)
    kept = x if p == 0 else zero
    for residual in (None, r):
        far.fill_(7.0)
        out = G.detffn_dropout_forward(x, p, 3, residual=residual, out=far)
        assert torch.equal(out, kept if residual is None else (kept.float() + r.float()).to(dtype))
    far.copy_(r)
    assert torch.equal(G.detffn_dropout_forward(x, p, 3, residual=far), (kept.float() + r.float()).to(dtype))


@pytest.mark.parametrize("p", [1.0, 0.0])
def test_many_short_rows(G, p):
    M, H = (1 << 22) + 3, 5
    wide = torch.full((M, H + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    r = torch.randn((M, H), device="cuda").bfloat16()
    x = torch.randn((M, H), device="cuda").bfloat16()
    kept = x if p == 0 else torch.zeros_like(x)
    assert torch.equal(G.detffn_dropout_forward(x, p, 3, out=wide[:, :H]), kept)
    assert torch.equal(G.detffn_dropout_forward(x, p, 3, residual=r, out=wide[:, :H]), (kept.float() + r.float()).bfloat16())
    assert bool((wide[:, H:] == 7.0).all())
