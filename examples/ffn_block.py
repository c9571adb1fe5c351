"""One FFN block of a network, trained and served with the library.

Training keeps gate and up of the forward in 8 bits and joins the norms, the
gate and the residual scale around the FFN in one pass each way:

    a    = rmsnorm(x) * w_in                      (the norm before the block)
    f    = FFN(a)                                  (gate and up kept in 8 bits)
    r    = x + scale * g * rmsnorm(f) * w_out      (norm after, gate, residual)
    y    = rmsnorm(r) * w_next                     (the next block's norm, same pass)

Serving runs a few tokens through the same joins with a mixture of experts in
the FFN's place.  (The layer keeps FP32 sums where the FFN follows its tree, so
one expert served is a rounding apart from the same FFN trained.)

    python examples/ffn_block.py [--tokens 512] [--width 1024] [--hidden 4096]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_deterministic_bf16_gb300 as G  # noqa: E402


def parameters(H, I, experts=0, seed=0):
    """Random weights: a dense FFN, or `experts` of them with a router."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, std=0.02, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).bfloat16()

    e = (experts,) if experts else ()
    p = dict(w_in=n(H, std=0.1, mean=1.0), w_out=n(H, std=0.1, mean=1.0), w_next=n(H, std=0.1, mean=1.0),
             g=n(H, std=0.1, mean=0.5), Wg=n(*e, I, H), Wu=n(*e, I, H), Wd=n(*e, H, I))
    if experts:
        p["Wr"] = n(experts, H)
    return p


def train_step(p, x, dr, dy, scale=1.0, eps=1e-6):
    """Forward and backward: (r, y) and the gradients of x and of every parameter."""
    M, H = x.shape
    I = p["Wg"].shape[0]
    _, a = G.detffn_join_forward(x, w_pre=p["w_in"], eps=eps)
    gate = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
    up = torch.empty_like(gate)
    f = G.detffn_forward(a, p["Wg"], p["Wu"], p["Wd"], gate_save=gate, up_save=up)
    saved = G.detffn_ckpt8_pack(gate, up)
    del gate, up                                  # what stays until the backward pass is `saved`
    r, y = G.detffn_join_forward(x, f, p["w_out"], p["g"], scale, p["w_next"], eps)

    d = G.detffn_join_backward(r, f, dr, dy, p["w_out"], p["g"], scale, p["w_next"], eps)
    da, dWg, dWu, dWd = G.detffn_backward_ckpt8(a, p["Wg"], p["Wu"], p["Wd"], saved, d.dz)
    first = G.detffn_join_backward(x, dr=d.dx, dy=da, w_pre=p["w_in"], eps=eps)
    return (r, y), dict(x=first.dx, w_in=first.dw_pre, w_out=d.dw_post, w_next=d.dw_pre, g=d.dgate, Wg=dWg, Wu=dWu,
                        Wd=dWd)


def serve_step(p, x, top_k, scale=1.0, eps=1e-6):
    """A few tokens through the block with a mixture of experts: (r, y)."""
    _, a = G.detffn_join_forward(x, w_pre=p["w_in"], eps=eps)
    f, _, _ = G.detffn_moe_forward(a, p["Wr"], p["Wg"], p["Wu"], p["Wd"], top_k)
    return G.detffn_join_forward(x, f, p["w_out"], p["g"], scale, p["w_next"], eps)


def _time(step, n=20):
    for _ in range(3):
        step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        step()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n * 1e6


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    a = ap.parse_args()
    from gemm_deterministic_bf16_gb300 import build
    build.build()
    p = parameters(a.width, a.hidden)
    x = torch.randn((a.tokens, a.width), device="cuda").bfloat16()
    dr, dy = (torch.randn_like(x) * 1e-2 for _ in range(2))
    us = _time(lambda: train_step(p, x, dr, dy))
    (r, _), grads = train_step(p, x, dr, dy)
    print("training step, %d tokens: %.0f us; |r| %.3f, |dx| %.3g, |dWd| %.3g" % (
        a.tokens, us, float(r.float().norm()), float(grads["x"].float().norm()), float(grads["Wd"].float().norm())))
    p = parameters(a.width, a.hidden // 4, a.experts)
    for tokens in (1, 16):
        x = torch.randn((tokens, a.width), device="cuda").bfloat16()
        us = _time(lambda: serve_step(p, x, a.top_k))
        print("serving step, %d tokens, %d of %d experts: %.0f us" % (tokens, a.top_k, a.experts, us))


if __name__ == "__main__":
    main()
