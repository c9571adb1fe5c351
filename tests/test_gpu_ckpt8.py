"""8-bit activation checkpoints: codes, scales and values bit for bit against
the same FP32 arithmetic on the host, and the SiLU backward stage against its
formulas in 64 bits.

Tolerance of the stage: sigma is formed from exp at a relative error of at
most (|g| + 4) 2^-23 (the rounded exponent and a 2-ulp exp2), one addition and
one reciprocal (2 ulp); with mag the product of the absolute values of the
factors, |error| <= u |value| + (|g| + 8) 2^-22 mag, u the output's unit
roundoff."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11), "f32": (torch.float32, 2.0 ** -24)}


@pytest.fixture(scope="module")
def G():
    import gemm_deterministic_bf16_gb300 as G
    from gemm_deterministic_bf16_gb300 import build
    build.build()
    return G


def pack_host(v):
    """Codes and scales of a float32 array [M, I], in float32 arithmetic."""
    M, I = v.shape
    nb = -(-I // 64)
    b = np.zeros((M, nb * 64), np.float32)
    b[:, :I] = v
    b = b.reshape(M, nb, 64)
    with np.errstate(all="ignore"):
        top = np.abs(b).max(-1)
        scale = np.minimum(top * np.float32(1.0 / 127.0), np.float32(float.fromhex("0x1.02040600p+121")))
        scale = np.where(np.isfinite(b).all(-1), scale, np.float32(np.nan)).astype(np.float32)
        q = np.where(scale[..., None] > 0, np.rint(b / scale[..., None]), 0)
    q = np.clip(np.nan_to_num(q), -127, 127).astype(np.int8)
    return q.reshape(M, -1)[:, :I], scale


SIZES = [(1, 1), (1, 64), (3, 63), (2, 65), (5, 1000), (32, 12288), (7, 5003), (300, 256), (1, 100000)]


def data(M, I, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((M, I), generator=g) * 1.5).to(DT[dt][0]).cuda()


def same(a, b):
    return np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,I", SIZES)
def test_pack_and_unpack(G, dt, M, I):
    gate, up = data(M, I, dt, M + I), data(M, I, dt, M + I + 1)
    c = G.detffn_ckpt8_pack(gate, up)
    for v, q, s in ((gate, c.gate_codes, c.gate_scales), (up, c.up_codes, c.up_scales)):
        rq, rs = pack_host(v.float().cpu().numpy())
        assert same(s.cpu().numpy(), rs) and same(q.cpu().numpy(), rq)
    for to in DT:
        got = G.detffn_ckpt8_unpack(c, dtype=DT[to][0])
        for v, q, s in zip(got, (c.gate_codes, c.up_codes), (c.gate_scales, c.up_scales)):
            ref = (q.float() * s.repeat_interleave(64, 1)[:, :I]).cpu().to(DT[to][0])
            assert torch.equal(v.cpu(), ref)


def test_round_trip_error(G):
    """A stored value is within half a code of the original: max|v| / 254 of its block."""
    v = data(64, 1024, "f32", 9)
    got, _ = G.detffn_ckpt8_unpack(G.detffn_ckpt8_pack(v, v), dtype=torch.float32)
    top = v.view(64, 16, 64).abs().amax(-1, keepdim=True).expand(-1, -1, 64).reshape(64, 1024)
    assert bool(((got - v).abs() <= top / 254 * (1 + 1e-5)).all())


@pytest.mark.parametrize("dt", list(DT))
def test_special_blocks(G, dt):
    """Blocks of zeros, one nonzero, ties between codes, subnormals, the type's
    largest values, an infinity, a NaN."""
    M, I = 8, 130
    v = torch.zeros((M, I))
    v[1, 70] = -3.0
    v[2, :64] = torch.arange(64) * 2.0 - 63.0
    v[2, 0] = 127.0                                   # scale 1: the odd halves are exact ties below
    v[2, 1:64] = torch.arange(63) / 2.0
    v[3] = torch.finfo(DT[dt][0]).max
    v[4] = torch.finfo(DT[dt][0]).tiny / 2
    v[5, 3] = float("inf")
    v[6, 65] = float("nan")
    v[7, 129] = -float("inf")
    v = v.to(DT[dt][0]).cuda()
    c = G.detffn_ckpt8_pack(v, v)
    q, s = pack_host(v.float().cpu().numpy())
    assert same(c.gate_codes.cpu().numpy(), q) and same(c.gate_scales.cpu().numpy(), s)
    assert same(c.up_codes.cpu().numpy(), q) and same(c.up_scales.cpu().numpy(), s)
    got, _ = G.detffn_ckpt8_unpack(c, dtype=DT[dt][0])
    assert not got[0].any() and bool(got[3].isfinite().all())
    assert bool(got[5, :64].isnan().all()) and bool(got[5, 64:].isfinite().all())
    assert bool(got[6, 64:128].isnan().all()) and bool(got[7, 128:].isnan().all()) and not got[7, :128].any()


def stage64(dh, g, u):
    sig = 1 / (1 + np.exp(-g))
    return {"dU": (dh * g * sig, np.abs(dh * g * sig)),
            "dG": (dh * u * sig * (1 + g * (1 - sig)), np.abs(dh * u) * sig * (1 + np.abs(g) * (1 - sig))),
            "h": (g * sig * u, np.abs(g * sig * u))}


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,I", SIZES)
def test_silu_backward(G, dt, M, I):
    c = G.detffn_ckpt8_pack(4 * data(M, I, "f32", 5), data(M, I, "f32", 6))
    dh = data(M, I, dt, 7)
    got = dict(zip(("dU", "dG", "h"), G.detffn_ckpt8_silu_backward(dh, c)))
    g, u = (t.cpu().double().numpy() for t in G.detffn_ckpt8_unpack(c, dtype=torch.float32))
    tiny = 2.0 ** -25 if dt == "f16" else 1e-37
    with np.errstate(over="ignore"):
        ref = stage64(dh.cpu().double().numpy(), g, u)
    for n, (v, mag) in ref.items():
        err = np.abs(got[n].cpu().double().numpy() - v)
        bound = DT[dt][1] * np.abs(v) + (np.abs(g) + 8) * 2.0 ** -22 * mag + tiny
        assert (err <= bound).all(), (n, float((err / bound).max()))


def test_silu_backward_of_extreme_gates(G):
    """Gates far out on both sides and at zero: no NaN from exp's overflow."""
    g = torch.tensor([[-3e38, -1e4, -200.0, -100.0, -88.0, 0.0, 88.0, 100.0, 1e4, 3e38]]).t().repeat(1, 64).cuda()
    c = G.detffn_ckpt8_pack(g, torch.ones_like(g))
    dU, dG, h = G.detffn_ckpt8_silu_backward(torch.ones_like(g), c)
    assert bool(dU[:3].abs().lt(1e-30).all()) and bool(dG[:3].abs().lt(1e-30).all())
    assert torch.allclose(h[6:, 0], g[6:, 0], rtol=1e-5) and torch.allclose(dG[6:, 0], torch.ones(4, device="cuda"))
    assert float(dG[5, 0]) == 0.5 and float(dU[5, 0]) == 0.0
    assert bool(torch.isfinite(torch.cat([dU, dG, h])).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_offset_views_equal_aligned(G, dt):
    """Buffers that start off the 16-byte grid give the same bits."""
    M, I = 9, 256
    gate, up, dh = (data(M, I, dt, k) for k in (1, 2, 3))
    off = lambda t: torch.cat([torch.zeros(1, dtype=t.dtype, device="cuda"), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    c = G.detffn_ckpt8_pack(gate, up)
    o = G.detffn_ckpt8_pack(off(gate), off(up), G.Ckpt8(*(off(t) for t in c)))
    assert all(torch.equal(a, b) for a, b in zip(c, o))
    for a, b in zip(G.detffn_ckpt8_unpack(c, dtype=DT[dt][0]), G.detffn_ckpt8_unpack(o, off(gate), off(up), DT[dt][0])):
        assert torch.equal(a, b)
    for a, b in zip(G.detffn_ckpt8_silu_backward(dh, c), G.detffn_ckpt8_silu_backward(off(dh), o)):
        assert torch.equal(a, b)


def test_empty_and_streams(G):
    e = torch.empty((0, 100), dtype=torch.bfloat16, device="cuda")
    c = G.detffn_ckpt8_pack(e, e)
    assert c.gate_scales.shape == (0, 2) and G.detffn_ckpt8_unpack(c)[0].shape == (0, 100)
    assert G.detffn_ckpt8_silu_backward(e, c)[2].shape == (0, 100)
    gate, up = data(64, 1000, "bf16", 1), data(64, 1000, "bf16", 2)
    a = G.detffn_ckpt8_silu_backward(gate, G.detffn_ckpt8_pack(gate, up))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        b = G.detffn_ckpt8_silu_backward(gate, G.detffn_ckpt8_pack(gate, up, stream=side), stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals(G):
    v = data(4, 128, "bf16", 1)
    c = G.detffn_ckpt8_pack(v, v)
    with pytest.raises(ValueError):
        G.detffn_ckpt8_pack(v, v.float())
    with pytest.raises(ValueError):
        G.detffn_ckpt8_pack(v[:, :64], v[:, :64])                    # not contiguous
    with pytest.raises(ValueError):
        G.detffn_ckpt8_pack(v.view(-1), v.view(-1))
    with pytest.raises(ValueError):
        G.detffn_ckpt8_unpack(c, dtype=torch.float64)
    with pytest.raises(ValueError):
        G.detffn_ckpt8_silu_backward(v[:2].contiguous(), c)
    with pytest.raises(ValueError):
        G.detffn_ckpt8_silu_backward(v, c._replace(gate_scales=c.gate_scales[:, :1].contiguous()))
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_ckpt8_silu_backward(v, c, dU=v)
    assert e.value.status == 1
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_ckpt8_pack(v, v, c._replace(up_codes=c.gate_codes))
    assert e.value.status == 1


@pytest.mark.parametrize("M,I", [(64, 1024), (7, 5003)])
def test_silu_backward_in_fp32_for_any_gate(G, M, I):
    """FP32: with e = 2^-24, exp is off by at most 2 ulp (4 e), 1 + exp and its
    reciprocal by e each, so sigma by 6 e and 1 - sigma by 11 e; a product or a sum
    adds e.  The longest chain, dG's, ends below 24 e, whatever the gate."""
    g = torch.Generator().manual_seed(I)
    gate = ((torch.rand((M, I), generator=g) * 2 - 1) * 86).cuda()
    gate[:, :64] = -88.0
    c = G.detffn_ckpt8_pack(gate, data(M, I, "f32", 6))
    dh = data(M, I, "f32", 7)
    got = dict(zip(("dU", "dG", "h"), G.detffn_ckpt8_silu_backward(dh, c)))
    gd, u = (t.cpu().double().numpy() for t in G.detffn_ckpt8_unpack(c, dtype=torch.float32))
    for n, (v, mag) in stage64(dh.cpu().double().numpy(), gd, u).items():
        err = np.abs(got[n].cpu().double().numpy() - v)
        assert (err <= 24 * 2.0 ** -24 * mag + 1e-42).all(), (n, float((err / (24 * 2.0 ** -24 * mag)).max()))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_silu_backward_of_gates_at_the_end_of_the_range(G, dt):
    """exp(88) is a number, though more than 2^126: its reciprocal times a large
    factor is an ordinary number."""
    g = torch.tensor([-80.0, -86.0, -87.5, -88.0]).repeat_interleave(64).expand(3, 256).contiguous().cuda()
    c = G.detffn_ckpt8_pack(g, torch.full_like(g, 2.0 ** 120))
    dh = torch.full_like(g, 2.0 ** 118).to(DT[dt][0])
    dU, dG, h = G.detffn_ckpt8_silu_backward(dh, c)
    gd, u = (t.cpu().double().numpy() for t in G.detffn_ckpt8_unpack(c, dtype=torch.float32))
    ref = stage64(np.full_like(gd, 2.0 ** 118), gd, u)
    for got, n in ((dU, "dU"), (h, "h")):   # (dG's factors alone leave the range)
        v, mag = ref[n]
        err = np.abs(got.cpu().double().numpy() - v)
        assert (err <= DT[dt][1] * np.abs(v) + (np.abs(gd) + 8) * 2.0 ** -22 * mag).all(), n
