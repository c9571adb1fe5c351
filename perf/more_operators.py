"""Measured cases of the operators that train and serve an FFN with experts and
in few bits: products grouped by expert (forward and backward), products with
4-bit weights for a few tokens (one matrix, and the gated FFN from three), and
dropout from a counter-based generator whose mask is never stored.

``run(state)`` makes one pass.  With ``own`` false it evaluates the operator in
plain torch operations, in 32 bits, rounded once at the end; with ``own`` true
it calls the library.  ``exact(case, seed)`` evaluates the definition in 64
bits, written apart from both.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
RUN = 128          # codes of a row that are laid out together
W4_TOKENS = 32     # tokens of the largest measured 4-bit call
MAX_ROWS = 16384


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _grouped(name, back, R, E, K, N, dtype):
    c = {"op": "grouped_backward" if back else "grouped_forward", "R": R, "E": E, "K": K, "N": N, "dtype": dtype}
    return dict(c, name=name) if name else c


def _w4(name, T, K, N, group, dtype, scales):
    c = {"op": "w4_matvec", "T": T, "K": K, "N": N, "group": group, "dtype": dtype, "scales": scales}
    return dict(c, name=name) if name else c


def _w4_ffn(name, T, H, I, group, dtype, scales):
    c = {"op": "w4_forward", "T": T, "H": H, "I": I, "group": group, "dtype": dtype, "scales": scales}
    return dict(c, name=name) if name else c


def _dropout(name, back, M, H, p, dtype, residual=False):
    c = {"op": "dropout_backward" if back else "dropout_forward", "M": M, "H": H, "p": p, "dtype": dtype,
         "residual": residual and not back}
    return dict(c, name=name) if name else c


def listed():
    return [
        # A serving batch of 33 tokens, three choices each, over many small experts: bound by the weights.
        _grouped("grouped_fwd_serving", False, 99, 64, 2048, 768, "bf16"),
        # A prompt's tokens, two choices each, through the gate projection of 16 experts.
        _grouped("grouped_fwd_prompt", False, 16384, 16, 4096, 1536, "bf16"),
        # A width that no vector divides, in 32 bits.
        _grouped("grouped_fwd_odd_f32", False, 777, 5, 1031, 515, "f32"),
        # Fine-tuning on a short ragged batch: the down projection's two gradients.
        _grouped("grouped_bwd_ragged", True, 1499, 16, 1416, 4096, "f16"),
        # A training batch: both gradients of a gate projection.
        _grouped("grouped_bwd_batch", True, 16384, 16, 4096, 1536, "bf16"),
        # One decoded token through one square projection: latency counts.
        _w4("w4_matvec_token", 1, 4096, 4096, 128, "bf16", "bf16"),
        # Three tokens, rows that end inside a group, 32-bit activations.
        _w4("w4_matvec_odd_f32", 3, 1416, 5003, 32, "f32", "f32"),
        # A decode batch through an output projection over a vocabulary.
        _w4("w4_matvec_vocab", 8, 4096, 131072, 64, "f16", "f16"),
        # One decoded token through the FFN of the decode benchmark.
        _w4_ffn("w4_ffn_token", 1, 4096, 12288, 128, "bf16", "bf16"),
        # The largest decode batch through the same FFN.
        _w4_ffn("w4_ffn_batch", W4_TOKENS, 4096, 12288, 128, "bf16", "bf16"),
        # Dropout after the FFN with the residual, one short sequence.
        _dropout("dropout_fwd_short", False, 32, 4096, 0.1, "bf16", True),
        # The gradient of a training batch: the same mask formed again.
        _dropout("dropout_bwd_batch", True, MAX_ROWS, 4096, 0.1, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, odd):
    n = _log(rng, lo, hi)
    return n if rng.random() < odd else max(64, n // 8 * 8)


def draw(rng):
    kind = rng.choice(("grouped_forward", "grouped_forward", "grouped_backward", "grouped_backward", "w4_matvec",
                       "w4_matvec", "w4_forward", "dropout_forward", "dropout_backward"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    scales = rng.choice((dtype, "f32"))
    if kind.startswith("grouped"):
        K, N = _width(rng, 64, 8192, 0.25), _width(rng, 64, 8192, 0.25)
        full = 16 * 4096 * 1536
        E = max(1, min(_log(rng, 1, 64), full // (K * N)))
        # 32-bit products run an order of magnitude below 16-bit ones; a drawn case costs no more than a listed one.
        R = max(1, min(_log(rng, 1, MAX_ROWS), MAX_ROWS * 4096 * 1536 // (K * N * (16 if dtype == "f32" else 1))))
        return _grouped(None, kind == "grouped_backward", R, E, K, N, dtype)
    if kind.startswith("w4"):
        T, group = _log(rng, 1, W4_TOKENS), rng.choice((32, 64, 128))
        if kind == "w4_matvec":
            return _w4(None, min(T, 8), _width(rng, 256, 16384, 0.25), _log(rng, 64, 32768), group, dtype, scales)
        return _w4_ffn(None, T, _width(rng, 256, 4096, 0.25), _width(rng, 256, 12288, 0.25), group, dtype, scales)
    M, H = _log(rng, 1, MAX_ROWS), _width(rng, 64, 8192, 0.4)
    M = max(1, min(M, MAX_ROWS * 4096 // (H * (SIZE[dtype] // 2) * 2)))
    return _dropout(None, kind == "dropout_backward", M, H, rng.choice((0.05, 0.1, 0.25, 0.5, round(rng.random() * 0.9, 3))),
                    dtype, rng.random() < 0.5)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _shares(E):
    """Expected share of the rows of each expert: uneven, as routers are."""
    w = [1.0 + 3.0 * ((7 * e) % E) / E for e in range(E)]
    return [v / sum(w) for v in w]


def _sizes(case, seed):
    rng = random.Random(seed * 1000003 + case["R"] * 64 + case["E"])
    n = [0] * case["E"]
    for e in rng.choices(range(case["E"]), weights=_shares(case["E"]), k=case["R"]):
        n[e] += 1
    return n


def _order(device):
    """Code of a run stored at each of its 128 nibble places: chunk t, word g, nibble p hold code 32 g + 8 t + 2 (p mod 4) + p / 4."""
    i = torch.arange(RUN, device=device)
    t, g, p = i // 32, i // 8 % 4, i % 8
    return 32 * g + 8 * t + 2 * (p % 4) + p // 4


def _pack(w, group, dtype):
    """Codes [N, 64 ceil(K / 128)] (uint8) and scales [N, ceil(K / group)] of w [N, K]."""
    N, K = w.shape
    pad = -K % RUN
    w = torch.nn.functional.pad(w, (0, pad))
    b = w.view(N, -1, group)
    scale = (b.abs().amax(-1) / 7.0).to(dtype)
    q = torch.where(scale[..., None] > 0, b / scale.float()[..., None], 0.0).round().clamp(-7, 7)
    q = (q.view(N, -1, RUN) + 8.0).to(torch.uint8)[:, :, _order(w.device)].reshape(N, -1, 2)
    return (q[..., 0] | (q[..., 1] << 4)).contiguous(), scale[:, :(K + group - 1) // group].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op.startswith("grouped"):
        R, E, K, N = (case[n] for n in ("R", "E", "K", "N"))
        s["sizes"] = _sizes(case, seed)
        ends = [0]
        for n in s["sizes"]:
            ends.append(ends[-1] + n)
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["x"] = normal((R, K), dt)
        w = torch.empty((E, N, K), dtype=dt, device="cuda")
        for e in range(E):        # no 32-bit copy of all the weights at once
            w[e] = normal((N, K), dt, 0.02)
        s["W"] = w
        if op == "grouped_backward":
            s["dOut"] = normal((R, N), dt, 1e-1)
    elif op.startswith("w4"):
        group, st = case["group"], DTYPES[case["scales"]]

        def matrix(N, K):
            parts = [_pack(normal((min(16384, N - n), K), torch.float32, 0.02), group, st) for n in range(0, N, 16384)]
            return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])

        if op == "w4_matvec":
            s["W"] = matrix(case["N"], case["K"])
            s["x"] = normal((case["T"], case["K"]), dt)
        else:
            s["Wg"], s["Wu"] = matrix(case["I"], case["H"]), matrix(case["I"], case["H"])
            s["Wd"] = matrix(case["H"], case["I"])
            s["x"] = normal((case["T"], case["H"]), dt)
    else:
        M, H = case["M"], case["H"]
        s["seed"] = random.Random(seed).getrandbits(63)
        s["offset"] = 1 + seed % 1000
        s["x"] = normal((M, H), dt)
        s["residual"] = normal((M, H), dt) if case["residual"] else None
    return s


# --------------------------------------------------------------------------
# Plain forms (32 bits, rounded once)
# --------------------------------------------------------------------------
def _ranges(sizes):
    a = 0
    for e, n in enumerate(sizes):
        yield e, a, a + n
        a += n


def _plain_grouped_forward(s):
    x, W = s["x"], s["W"]
    out = torch.empty((x.shape[0], W.shape[1]), dtype=x.dtype, device=x.device)
    for e, a, b in _ranges(s["sizes"]):
        if b > a:
            out[a:b] = x[a:b].float() @ W[e].float().T
    return {"out": out}


def _plain_grouped_backward(s):
    x, W, d = s["x"], s["W"], s["dOut"]
    dX, dW = torch.empty_like(x), torch.empty_like(W)
    for e, a, b in _ranges(s["sizes"]):
        de = d[a:b].float()
        if b > a:
            dX[a:b] = de @ W[e].float()
        dW[e] = de.T @ x[a:b].float()
    return {"dX": dX, "dW": dW}


def _values(W, K, group):
    """The 32-bit values [N, K] of codes and scales."""
    codes, scales = W
    N = codes.shape[0]
    q = torch.stack((codes & 15, codes >> 4), -1).view(N, -1, RUN)
    place = torch.empty(RUN, dtype=torch.int64, device=codes.device)
    place[_order(codes.device)] = torch.arange(RUN, device=codes.device)
    q = q[:, :, place].reshape(N, -1)[:, :K].float() - 8.0
    pad = -K % group
    q = torch.nn.functional.pad(q, (0, pad)).view(N, -1, group) * scales.float()[..., None]
    return q.view(N, -1)[:, :K]


def _plain_w4_matvec(s):
    c, x = s["case"], s["x"]
    return {"out": (x.float() @ _values(s["W"], c["K"], c["group"]).T).to(x.dtype)}


def _plain_w4_forward(s):
    c, x = s["case"], s["x"].float()
    g, u = (x @ _values(s[n], c["H"], c["group"]).T for n in ("Wg", "Wu"))
    h = g / (1.0 + torch.exp(-g)) * u
    return {"out": (h @ _values(s["Wd"], c["I"], c["group"]).T).to(s["x"].dtype)}


def _mulhilo(a, m):
    """High and low 32 bits of a * m, for a (int64 tensor) and m below 2^32."""
    lo = a * (m & 0xFFFF)                    # below 2^48
    hi = a * (m >> 16) + (lo >> 16)          # below 2^49
    return hi >> 16, ((hi & 0xFFFF) << 16) | (lo & 0xFFFF)


def _keep(M, H, p, seed, offset, device):
    """The mask [M, H]: Philox4x32-10 words of counter (column / 4, row, offset) under the key seed, kept from p 2^32 on."""
    c0 = torch.arange((H + 3) // 4, device=device).expand(M, -1)
    c1 = torch.arange(M, device=device)[:, None].expand(-1, c0.shape[1])
    c2, c3 = torch.full_like(c0, offset & 0xFFFFFFFF), torch.full_like(c0, (offset >> 32) & 0xFFFFFFFF)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack((c0, c1, c2, c3), -1).view(M, -1)[:, :H] >= int(p * 4294967296.0)


def _plain_dropout(s):
    c, x = s["case"], s["x"]
    keep = _keep(c["M"], c["H"], c["p"], s["seed"], s["offset"], x.device)
    v = torch.where(keep, x.float() * (1.0 / (1.0 - c["p"])), 0.0)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(x.dtype)


_PLAIN = {"grouped_forward": _plain_grouped_forward, "grouped_backward": _plain_grouped_backward,
          "w4_matvec": _plain_w4_matvec, "w4_forward": _plain_w4_forward,
          "dropout_forward": lambda s: {"out": _plain_dropout(s)}, "dropout_backward": lambda s: {"dX": _plain_dropout(s)}}


# --------------------------------------------------------------------------
# The library's operators
# --------------------------------------------------------------------------
def _own_grouped_forward(s):
    import gemm_deterministic_bf16_gb300 as G
    return {"out": G.detffn_grouped_forward(s["x"], s["W"], s["offsets"])}


def _own_grouped_backward(s):
    import gemm_deterministic_bf16_gb300 as G
    dX, dW = G.detffn_grouped_backward(s["x"], s["W"], s["offsets"], s["dOut"])
    return {"dX": dX, "dW": dW}


def _own_w4_matvec(s):
    import gemm_deterministic_bf16_gb300 as G
    c = s["case"]
    return {"out": G.detffn_w4_matvec(s["x"], G.W4(*s["W"], c["K"], c["group"]))}


def _own_w4_forward(s):
    import gemm_deterministic_bf16_gb300 as G
    c = s["case"]
    Wg, Wu = (G.W4(*s[n], c["H"], c["group"]) for n in ("Wg", "Wu"))
    return {"out": G.detffn_w4_forward(s["x"], Wg, Wu, G.W4(*s["Wd"], c["I"], c["group"]))}


def _own_dropout_forward(s):
    import gemm_deterministic_bf16_gb300 as G
    return {"out": G.detffn_dropout_forward(s["x"], s["case"]["p"], s["seed"], s["offset"], residual=s["residual"])}


def _own_dropout_backward(s):
    import gemm_deterministic_bf16_gb300 as G
    return {"dX": G.detffn_dropout_backward(s["x"], s["case"]["p"], s["seed"], s["offset"])}


_OWN = {"grouped_forward": _own_grouped_forward, "grouped_backward": _own_grouped_backward,
        "w4_matvec": _own_w4_matvec, "w4_forward": _own_w4_forward, "dropout_forward": _own_dropout_forward,
        "dropout_backward": _own_dropout_backward}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def _w4_bytes(N, K, case):
    return N * ((K + 1) // 2 + SIZE[case["scales"]] * ((K + case["group"] - 1) // case["group"]))


def work(case):
    op, n = case["op"], SIZE[case["dtype"]]
    if op.startswith("grouped"):
        R, E, K, N = (case[m] for m in ("R", "E", "K", "N"))
        # Experts that R independent choices are expected to hit.
        hit = sum(1.0 - (1.0 - p) ** R for p in _shares(E))
        if op == "grouped_forward":
            return {"bytes": n * (R * (K + N) + hit * N * K), "flops": 2.0 * R * N * K}
        return {"bytes": n * (R * (2 * K + N) + (hit + E) * N * K), "flops": 4.0 * R * N * K}
    if op == "w4_matvec":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": _w4_bytes(N, K, case) + n * T * (K + N), "flops": 2.0 * T * N * K}
    if op == "w4_forward":
        T, H, I = case["T"], case["H"], case["I"]
        return {"bytes": 2 * _w4_bytes(I, H, case) + _w4_bytes(H, I, case) + 2 * n * T * H, "flops": 6.0 * T * H * I}
    return {"bytes": n * case["M"] * case["H"] * (3 if case["residual"] else 2), "flops": 2 * case["M"] * case["H"]}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def _expert_of_rows(s):
    return torch.repeat_interleave(torch.arange(len(s["sizes"])), torch.tensor(s["sizes"])).cuda()


def _exact_grouped_forward(s):
    x, of = s["x"].double(), _expert_of_rows(s)
    out = torch.zeros((x.shape[0], s["W"].shape[1]), dtype=torch.float64, device=x.device)
    for e in range(s["W"].shape[0]):
        r = torch.nonzero(of == e).flatten()
        out[r] = torch.einsum("rk,nk->rn", x[r], s["W"][e].double())
    return {"out": out}


def _exact_grouped_backward(s):
    x, d, of = s["x"].double(), s["dOut"].double(), _expert_of_rows(s)
    dX, dW = torch.zeros_like(x), torch.zeros(s["W"].shape, dtype=torch.float64, device=x.device)
    for e in range(s["W"].shape[0]):
        r = torch.nonzero(of == e).flatten()
        dX[r] = torch.einsum("rn,nk->rk", d[r], s["W"][e].double())
        dW[e] = torch.einsum("rn,rk->nk", d[r], x[r])
    return {"dX": dX, "dW": dW}


def _read64(W, K, group):
    """Rows of 64-bit values, each code picked by its place."""
    codes, scales = W
    k = torch.arange(K, device=codes.device)
    g, t, j = k % RUN // 32, k % 32 // 8, k % 8
    nibble = j // 2 + 4 * (j % 2)
    byte = k // RUN * 64 + t * 16 + g * 4 + nibble // 2
    q = (codes[:, byte].to(torch.int16) >> (4 * (nibble % 2)).to(torch.int16)) % 16
    return (q.double() - 8.0) * scales.double()[:, k // group]


def _product64(x, W, K, group):
    out = []
    for n in range(0, W[0].shape[0], 8192):
        out.append(torch.einsum("tk,nk->tn", x, _read64((W[0][n:n + 8192], W[1][n:n + 8192]), K, group)))
    return torch.cat(out, 1)


def _exact_w4_matvec(s):
    c = s["case"]
    return {"out": _product64(s["x"].double(), s["W"], c["K"], c["group"])}


def _exact_w4_forward(s):
    c, x = s["case"], s["x"].double()
    g, u = _product64(x, s["Wg"], c["H"], c["group"]), _product64(x, s["Wu"], c["H"], c["group"])
    return {"out": _product64(g * torch.sigmoid(g) * u, s["Wd"], c["I"], c["group"])}


def _exact_dropout(s):
    c = s["case"]
    M, blocks, mask = c["M"], (c["H"] + 3) // 4, np.uint64(0xFFFFFFFF)
    ctr = [np.tile(np.arange(blocks, dtype=np.uint64), M), np.repeat(np.arange(M, dtype=np.uint64), blocks),
           np.full(M * blocks, s["offset"] & 0xFFFFFFFF, np.uint64), np.full(M * blocks, s["offset"] >> 32, np.uint64)]
    for i in range(10):
        key = [np.uint64(((s["seed"] >> (32 * j)) + i * w) & 0xFFFFFFFF) for j, w in ((0, 0x9E3779B9), (1, 0xBB67AE85))]
        a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(b >> np.uint64(32)) ^ ctr[1] ^ key[0], b & mask, (a >> np.uint64(32)) ^ ctr[3] ^ key[1], a & mask]
    keep = np.stack(ctr, 1).reshape(M, -1)[:, :c["H"]] >= math.floor(c["p"] * 2.0 ** 32)
    v = s["x"].double() * torch.from_numpy(keep).to(s["x"].device) / (1.0 - c["p"])
    return v if s["residual"] is None else v + s["residual"].double()


_EXACT = {"grouped_forward": _exact_grouped_forward, "grouped_backward": _exact_grouped_backward,
          "w4_matvec": _exact_w4_matvec, "w4_forward": _exact_w4_forward,
          "dropout_forward": lambda s: {"out": _exact_dropout(s)}, "dropout_backward": lambda s: {"dX": _exact_dropout(s)}}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
