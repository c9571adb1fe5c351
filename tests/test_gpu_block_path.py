"""The operators around the FFN used together: the backward pass from an 8-bit
checkpoint against its own contractions bit for bit, and the example's training
and serving steps against 64-bit references."""
import importlib.util
import os

import pytest
import torch

from gemm_deterministic_bf16_gb300.inputs import ffn_inputs
from tests.gpu_util import dev

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
    spec = importlib.util.spec_from_file_location("ffn_block", os.path.join(ROOT, "examples", "ffn_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("M,H,I,k", [(8, 256, 768, 1), (32, 256, 1024, 2), (256, 512, 1536, 1), (128, 256, 1024, 4)])
def test_backward_from_a_checkpoint_is_its_contractions(G, M, H, I, k, path):
    """The call is the tree contractions of detffn_backward around
    detffn_ckpt8_silu_backward: the same bits as calling them one by one."""
    t = {n: dev(v) for n, v in ffn_inputs(M, H, I, seed=M + k).items()}
    x, Wg, Wu, Wd, dOut = (t[n] for n in ("x", "Wg", "Wu", "Wd", "dOut"))
    gate, up = (torch.empty((M, I), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    G.detffn_forward(x, Wg, Wu, Wd, gate_save=gate, up_save=up, path=path)
    c = G.detffn_ckpt8_pack(gate, up)
    got = G.detffn_backward_ckpt8(x, Wg, Wu, Wd, c, dOut, shards=k, path=path)
    gemm = lambda a, b: G.detffn_tree_gemm(a, b, path=path)  # noqa: E731
    dU, dG, h = G.detffn_ckpt8_silu_backward(gemm(dOut, Wd.t()), c)
    dX = (gemm(dG, Wg.t()).float() + gemm(dU, Wu.t()).float()).bfloat16()
    at = (lambda v: v.t()) if M > 32 or path == 1 else (lambda v: v.t().contiguous())
    for a, b in zip(got, (dX, gemm(at(dG), at(x)), gemm(at(dU), at(x)), gemm(at(dOut), at(h)))):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = G.detffn_backward_ckpt8(x, Wg, Wu, Wd, c, dOut, shards=k, path=path, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert G.detffn_get_status() == 0


def test_backward_from_a_checkpoint_refuses(G):
    t = {n: dev(v) for n, v in ffn_inputs(8, 256, 768, seed=1).items()}
    g = torch.zeros((8, 768), dtype=torch.bfloat16, device="cuda")
    c = G.detffn_ckpt8_pack(g, g)
    args = (t["x"], t["Wg"], t["Wu"], t["Wd"])
    with pytest.raises(ValueError):
        G.detffn_backward_ckpt8(*args, c._replace(gate_codes=c.gate_codes[:4].contiguous()), t["dOut"])
    with pytest.raises(ValueError):
        G.detffn_backward_ckpt8(*args, c._replace(up_scales=c.up_scales.double()), t["dOut"])
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_backward_ckpt8(*args, c, t["dOut"], dX=t["x"])
    assert e.value.status == 1
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_backward_ckpt8(*args, c, t["dOut"], ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5


def norm64(v, w, eps=1e-6):
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt() * w


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_training_step(G, example):
    """Against autograd in 64 bits.  A stored 8-bit value is off by at most
    max / 254 of its block, 0.6 % of the values' spread (root mean square, the
    largest of 64 normal values being about 2.7 times the spread); each BF16
    stage and tree adds below 0.5 %, and a gradient passes six of them: 3 % of
    each gradient's norm bounds the sum of squares with room."""
    M, H, I = 128, 256, 768
    p = example.parameters(H, I)
    torch.manual_seed(4)
    x = torch.randn((M, H), device="cuda").bfloat16()
    dr, dy = (torch.randn_like(x) * 0.1 for _ in range(2))
    (r, y), grads = example.train_step(p, x, dr, dy, 0.8)
    leaf = {n: t.double().requires_grad_(True) for n, t in dict(p, x=x).items()}
    q = leaf
    a = norm64(q["x"], q["w_in"])
    g = a @ q["Wg"].T
    f = (g * torch.sigmoid(g) * (a @ q["Wu"].T)) @ q["Wd"].T
    r64 = q["x"] + 0.8 * q["g"] * norm64(f, q["w_out"])
    y64 = norm64(r64, q["w_next"])
    names = list(leaf)
    want = dict(zip(names, torch.autograd.grad((r64 * dr.double()).sum() + (y64 * dy.double()).sum(),
                                               [leaf[n] for n in names])))
    assert rel(r, r64.detach()) < 0.01 and rel(y, y64.detach()) < 0.01
    for n in names:
        assert rel(grads[n], want[n]) < 0.03, (n, rel(grads[n], want[n]))


@pytest.mark.parametrize("T", [1, 5, 64])
def test_serving_step(G, example, T):
    """BF16 stages as above, each below 0.5 %: 2 % of the norm."""
    H, I, E, k = 256, 192, 8, 2
    p = example.parameters(H, I, E)
    p["Wr"] = p["Wr"] * 40                        # far-apart logits: the BF16 norm cannot change a choice
    torch.manual_seed(T)
    x = torch.randn((T, H), device="cuda").bfloat16()
    r, y = example.serve_step(p, x, k, 0.8)
    q = {n: t.double() for n, t in p.items()}
    _, a = G.detffn_join_forward(x, w_pre=p["w_in"])
    a = a.double()
    w, ids = torch.softmax(a @ q["Wr"].T, -1).topk(k, -1)
    w = w / w.sum(-1, keepdim=True)
    f = torch.zeros_like(a)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            g = q["Wg"][e] @ a[t]
            f[t] += w[t, j] * (q["Wd"][e] @ (g * torch.sigmoid(g) * (q["Wu"][e] @ a[t])))
    r64 = x.double() + 0.8 * q["g"] * norm64(f, q["w_out"])
    assert rel(r, r64) < 0.02 and rel(y, norm64(r64, q["w_next"])) < 0.02
