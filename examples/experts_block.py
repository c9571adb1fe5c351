"""A block with experts in the FFN's place, trained on many tokens, and a dense
one served in 4 bits.

Training sorts the tokens' choices by expert on the device (no size reaches the
host), multiplies each expert's rows with its own matrices, keeps gate and up in
8 bits, and drops elements of the block's output by a mask that is formed again
in the backward pass:

    a = rmsnorm(x) * w_in
    f = sum over the chosen experts of  w * FFN_e(a)
    r = x + scale * g * rmsnorm(dropout(f)) * w_out,   y = rmsnorm(r) * w_next

    python examples/experts_block.py [--tokens 4096] [--width 1024] [--hidden 512]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import gemm_deterministic_bf16_gb300 as G  # noqa: E402
from ffn_block import _time, parameters  # noqa: E402


def route(a, Wr, top_k):
    """Weights [M, k] of each token's experts, the order that sorts its choices by
    expert, its inverse, and each expert's range of the sorted rows."""
    logits = a.float() @ Wr.float().T
    top, ids = logits.topk(top_k, -1)
    w = torch.softmax(top, -1)
    order = torch.argsort(ids.flatten(), stable=True)
    inverse = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=a.device))
    counts = torch.zeros(Wr.shape[0], dtype=torch.int64, device=a.device).scatter_add_(0, ids.flatten(), torch.ones_like(order))
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    return w, ids, order, inverse, offsets


def train_step(p, x, dr, dy, top_k, drop=0.1, seed=0, step=0, scale=1.0, eps=1e-6):
    """Forward and backward: (r, y) and the gradients of x and of every parameter."""
    M, H = x.shape
    _, a = G.detffn_join_forward(x, w_pre=p["w_in"], eps=eps)
    w, ids, order, inverse, offsets = route(a, p["Wr"], top_k)
    token = order // top_k
    rows = a[token]
    gate = G.detffn_grouped_forward(rows, p["Wg"], offsets)
    up = G.detffn_grouped_forward(rows, p["Wu"], offsets)
    saved = G.detffn_ckpt8_pack(gate, up)
    h = (torch.nn.functional.silu(gate.float()) * up.float()).bfloat16()
    del gate, up
    pairs = G.detffn_grouped_forward(h, p["Wd"], offsets)
    f = (pairs[inverse].view(M, top_k, H).float() * w[..., None]).sum(1).bfloat16()
    f = G.detffn_dropout_forward(f, drop, seed, step)
    r, y = G.detffn_join_forward(x, f, p["w_out"], p["g"], scale, p["w_next"], eps)

    d = G.detffn_join_backward(r, f, dr, dy, p["w_out"], p["g"], scale, p["w_next"], eps)
    df = G.detffn_dropout_backward(d.dz, drop, seed, step)
    dpairs = (df[token].float() * w.flatten()[order][:, None]).bfloat16()
    dw = (pairs[inverse].view(M, top_k, H).float() * df[:, None].float()).sum(-1)
    dh, dWd = G.detffn_grouped_backward(h, p["Wd"], offsets, dpairs)
    dU, dG, _ = G.detffn_ckpt8_silu_backward(dh, saved)
    da_g, dWg = G.detffn_grouped_backward(rows, p["Wg"], offsets, dG)
    da_u, dWu = G.detffn_grouped_backward(rows, p["Wu"], offsets, dU)
    da = (da_g.float() + da_u.float())[inverse].view(M, top_k, H).sum(1)
    dlogits = torch.zeros((M, p["Wr"].shape[0]), device=x.device).scatter_(1, ids, w * (dw - (w * dw).sum(-1, keepdim=True)))
    da = (da + dlogits @ p["Wr"].float()).bfloat16()
    first = G.detffn_join_backward(x, dr=d.dx, dy=da, w_pre=p["w_in"], eps=eps)
    return (r, y), dict(x=first.dx, w_in=first.dw_pre, w_out=d.dw_post, w_next=d.dw_pre, g=d.dgate, Wr=dlogits.T @ a.float(),
                        Wg=dWg, Wu=dWu, Wd=dWd)


def in_4_bits(p, group=128):
    """A dense FFN's matrices in 4 bits."""
    return dict(p, **{n: G.detffn_w4_pack(p[n], group) for n in ("Wg", "Wu", "Wd")})


def serve_step(p, x, scale=1.0, eps=1e-6):
    """A few tokens through a dense block whose matrices are in 4 bits: (r, y)."""
    _, a = G.detffn_join_forward(x, w_pre=p["w_in"], eps=eps)
    f = G.detffn_w4_forward(a, p["Wg"], p["Wu"], p["Wd"])
    return G.detffn_join_forward(x, f, p["w_out"], p["g"], scale, p["w_next"], eps)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    a = ap.parse_args()
    from gemm_deterministic_bf16_gb300 import build
    build.build()
    p = parameters(a.width, a.hidden, a.experts)
    x = torch.randn((a.tokens, a.width), device="cuda").bfloat16()
    dr, dy = (torch.randn_like(x) * 1e-2 for _ in range(2))
    us = _time(lambda: train_step(p, x, dr, dy, a.top_k))
    (r, _), grads = train_step(p, x, dr, dy, a.top_k)
    print("training step, %d tokens, %d of %d experts: %.0f us; |r| %.3f, |dx| %.3g, |dWd| %.3g" % (
        a.tokens, a.top_k, a.experts, us, float(r.float().norm()), float(grads["x"].float().norm()),
        float(grads["Wd"].float().norm())))
    p = in_4_bits(parameters(a.width, 4 * a.width))
    for tokens in (1, 16):
        x = torch.randn((tokens, a.width), device="cuda").bfloat16()
        print("serving step in 4 bits, %d tokens: %.0f us" % (tokens, _time(lambda: serve_step(p, x))))


if __name__ == "__main__":
    main()
