"""The grouped products, dropout and the 4-bit products used together with the
joins and the checkpoints: the example's training and serving steps against
64-bit references."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def G():
    import gemm_deterministic_bf16_gb300 as G
    from gemm_deterministic_bf16_gb300 import build
    build.build()
    assert G.detffn_get_status() == 0
    return G


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("experts_block", os.path.join(ROOT, "examples", "experts_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm64(v, w, eps=1e-6):
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt() * w


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("M,H,I,E,k,drop", [(200, 128, 192, 6, 2, 0.25), (65, 72, 40, 5, 3, 0.0)])
def test_training_step(G, example, M, H, I, E, k, drop):
    """Against autograd in 64 bits with the step's own choices of experts and its
    mask.  A value kept in 8 bits is off by 0.6 % of the values' spread; each BF16
    stage adds below 0.4 % (half a step is 0.39 %, its root mean square a third
    less), and a gradient passes eight of them: 3 % of each gradient's norm bounds
    the root of their squares with room.  The router's gradient is a small
    difference of sums that carry those errors: twice that."""
    p = example.parameters(H, I, E)
    for n in ("Wg", "Wu", "Wd"):
        p[n] = p[n] * 4
    p["Wr"] = p["Wr"] * 40                        # far-apart logits
    torch.manual_seed(M)
    x = torch.randn((M, H), device="cuda").bfloat16()
    dr, dy = (torch.randn_like(x) * 0.1 for _ in range(2))
    (r, y), grads = example.train_step(p, x, dr, dy, k, drop, seed=7, step=3, scale=0.8)
    _, a16 = G.detffn_join_forward(x, w_pre=p["w_in"])
    ids = example.route(a16, p["Wr"], k)[1]
    mask = G.detffn_dropout_forward(torch.ones((M, H), device="cuda"), drop, 7, 3).double()
    assert abs(float(mask.mean()) - 1.0) < 0.05
    leaf = {n: t.double().requires_grad_(True) for n, t in dict(p, x=x).items()}
    q = leaf
    a = norm64(q["x"], q["w_in"])
    w = torch.softmax((a @ q["Wr"].T).gather(1, ids), -1)
    f = torch.zeros_like(a)
    for e in range(E):
        g = a @ q["Wg"][e].T
        f = f + (w * (ids == e)).sum(-1, keepdim=True) * ((g * torch.sigmoid(g) * (a @ q["Wu"][e].T)) @ q["Wd"][e].T)
    r64 = q["x"] + 0.8 * q["g"] * norm64(f * mask, q["w_out"])
    y64 = norm64(r64, q["w_next"])
    names = list(leaf)
    want = dict(zip(names, torch.autograd.grad((r64 * dr.double()).sum() + (y64 * dy.double()).sum(), [leaf[n] for n in names])))
    assert rel(r, r64.detach()) < 0.01 and rel(y, y64.detach()) < 0.01
    for n in names:
        assert rel(grads[n], want[n]) < (0.06 if n == "Wr" else 0.03), (n, rel(grads[n], want[n]))
    again = example.train_step(p, x, dr, dy, k, drop, seed=7, step=3, scale=0.8)
    assert torch.equal(again[0][0], r) and all(torch.equal(again[1][n], grads[n]) for n in ("x", "Wg", "Wu", "Wd", "g"))
    assert G.detffn_get_status() == 0


@pytest.mark.parametrize("T", [1, 7, 33])
def test_serving_step_in_4_bits(G, example, T):
    """Against the packed matrices' own values: three BF16 stages, 2 % of the norm."""
    H, I = 256, 640
    p = example.in_4_bits(example.parameters(H, I), 64)
    torch.manual_seed(T)
    x = torch.randn((T, H), device="cuda").bfloat16()
    r, y = example.serve_step(p, x, 0.8)
    Wg, Wu, Wd = (G.detffn_w4_unpack(p[n], dtype=torch.float32).double() for n in ("Wg", "Wu", "Wd"))
    q = {n: p[n].double() for n in ("w_in", "w_out", "w_next", "g")}
    a = norm64(x.double(), q["w_in"])
    g = a @ Wg.T
    f = (g * torch.sigmoid(g) * (a @ Wu.T)) @ Wd.T
    r64 = x.double() + 0.8 * q["g"] * norm64(f, q["w_out"])
    assert rel(r, r64) < 0.02 and rel(y, norm64(r64, q["w_next"])) < 0.02
