"""The residual join (norms before and after a block, gate, residual scale)
against its formulas in 64 bits: outputs, every gradient, central differences,
all gate shapes, types, widths, strides and in-place use.

Tolerances.  u is the unit roundoff of the stored type, e = 2^-24 that of
FP32.  A sum of squares over a row is formed by chains of at most 64 additions
in a thread, 5 in a warp and 16 over warps, each term with one rounding: its
relative error is at most 86 e, its inverse root's half that plus 2 ulp
(rsqrt) -- below 48 e.  Each output then takes a handful of products and sums
of terms whose absolute values sum to `mag`: |error| <= u |value| + 64 e mag
for outputs without further sums, and + 150 e mag where two sums over the row
enter.  Sums over tokens add the M / 152 rows of a thread, up to 16 groups, 10
sets and 16 threads: for the M here below ceil(M / 304) + 46 additions."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11), "f32": (torch.float32, 2.0 ** -24)}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38}   # half the spacing of subnormals
E = 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    import gemm_deterministic_bf16_gb300 as G
    from gemm_deterministic_bf16_gb300 import build
    build.build()
    return G


def gate_shape(kind, M, H):
    return {"scalar": (1,), "feature": (H,), "token": (M, 1), "full": (M, H)}[kind]


def inputs(M, H, dt, pt, gate, seed, post=True, pre=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda s, d, std=1.0, mean=0.0: (torch.randn(s, generator=g) * std + mean).to(DT[d][0]).cuda()  # noqa: E731
    return dict(x=n((M, H), dt), z=n((M, H), dt, 0.7), dr=n((M, H), dt, 0.5), dy=n((M, H), dt, 0.5) if pre else None,
                w_post=n((H,), pt, 0.2, 1.0) if post else None, w_pre=n((H,), pt, 0.2, 1.0) if pre else None,
                gate=None if gate == "none" else n(gate_shape(gate, M, H), pt, 0.5, 0.5))


def d(t):
    return None if t is None else t.detach().cpu().double()


def norm64(v, w, eps):
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt() * w


def close(got, ref, mag, dt, c):
    got, ref, mag = d(got), ref.double(), mag.double()
    u = DT[dt][1]
    bound = u * ref.abs() + c * E * mag + TINY[dt]
    bad = ~((got - ref).abs() <= bound)
    assert not bool(bad.any()), "worst %.3g of the bound" % float(((got - ref).abs() / bound).max())


def forward64(x, z, w_post, gate, scale, w_pre, eps):
    x, z, w_post, gate, w_pre = (d(t) for t in (x, z, w_post, gate, w_pre))
    if z is None:
        r, mag = x, x.abs()
    else:
        n = z if w_post is None else norm64(z, w_post, eps)
        t = scale * (n if gate is None else n * gate)
        r, mag = x + t, x.abs() + t.abs()
    return r, mag, None if w_pre is None else norm64(r, w_pre, eps)


CASES = [(1, 1, "f32", "f32", "none"), (1, 4096, "bf16", "bf16", "feature"), (5, 33, "f16", "f16", "token"),
         (3, 255, "bf16", "f32", "full"), (7, 256, "bf16", "bf16", "scalar"), (2, 8193, "f16", "f32", "feature"),
         (4, 16384, "bf16", "f32", "full"), (2, 32768, "f32", "f32", "feature"), (305, 1031, "f32", "f32", "token"),
         (700, 512, "bf16", "bf16", "feature"), (33, 4104, "f16", "f16", "full"), (640, 40, "f32", "f32", "scalar")]


@pytest.mark.parametrize("M,H,dt,pt,gate", CASES)
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_forward(G, M, H, dt, pt, gate, post, pre):
    s = inputs(M, H, dt, pt, gate, M + H, post, pre)
    out, y = G.detffn_join_forward(s["x"], s["z"], s["w_post"], s["gate"], 0.75, s["w_pre"], 1e-5)
    r, mag, yr = forward64(s["x"], s["z"], s["w_post"], s["gate"], 0.75, s["w_pre"], 1e-5)
    close(out, r, mag, dt, 64)
    assert (y is None) == (not pre)
    if pre:
        rms = (r.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        close(y, yr, mag / rms * d(s["w_pre"]).abs() + yr.abs(), dt, 150)


def test_norm_alone_equals_join_without_block(G):
    s = inputs(9, 777, "bf16", "f32", "none", 3)
    out, y = G.detffn_join_forward(s["x"], w_pre=s["w_pre"])
    assert out is None
    close(y, norm64(d(s["x"]), d(s["w_pre"]), 1e-6), norm64(d(s["x"]), d(s["w_pre"]), 1e-6).abs(), "bf16", 150)


def backward64(s, r, scale, eps, with_dr=True):
    """Gradients in 64 bits and, for each, the sum of the absolute values of its terms."""
    z, w_post, gate, w_pre, dr, dy = (d(s[n]) for n in ("z", "w_post", "gate", "w_pre", "dr", "dy"))
    r = d(r)
    H = r.shape[1]
    dx = dr if with_dr else torch.zeros_like(r)
    mag = dx.abs()
    got = {}
    if w_pre is not None:
        a = 1 / (r.square().mean(-1, keepdim=True) + eps).sqrt()
        k = (dy * w_pre * r).sum(-1, keepdim=True)
        ka = (dy * w_pre * r).abs().sum(-1, keepdim=True)
        dx = dx + a * dy * w_pre - r * a ** 3 / H * k
        mag = mag + (a * dy * w_pre).abs() + (r * a ** 3 / H).abs() * ka
        got["dw_pre"] = ((dy * r * a).sum(0), (dy * r * a).abs().sum(0))
    got["dx"] = (dx, mag)
    b = 1 / (z.square().mean(-1, keepdim=True) + eps).sqrt() if w_post is not None else torch.ones_like(z[:, :1])
    w = w_post if w_post is not None else torch.ones(H, dtype=z.dtype)
    n = z * b * w
    dn, dm = scale * dx, abs(scale) * mag
    if gate is not None:
        full = gate.expand_as(z) if gate.dim() == 2 else gate.reshape(1, -1).expand_as(z)
        tg, tm = dn * n, dm * n.abs()
        sh = tuple(gate.shape)
        red = [i for i in range(2) if ((1,) * (2 - len(sh)) + sh)[i] == 1 and z.shape[i] > 1]
        got["dgate"] = tuple((v.sum(red, keepdim=True) if red else v).reshape(sh) for v in (tg, tm))
        dn, dm = dn * full, dm * full.abs()
    if w_post is not None:
        got["dw_post"] = ((dn * z * b).sum(0), (dm * (z * b).abs()).sum(0))
        e, em = (dn * w * z).sum(-1, keepdim=True), (dm * (w * z).abs()).sum(-1, keepdim=True)
        got["dz"] = (b * dn * w - z * b ** 3 / H * e, b * dm * w.abs() + (z * b ** 3 / H).abs() * em)
    else:
        got["dz"] = (dn, dm)
    return got


@pytest.mark.parametrize("M,H,dt,pt,gate", CASES)
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_backward(G, M, H, dt, pt, gate, post, pre):
    s = inputs(M, H, dt, pt, gate, 2 * M + H, post, pre)
    r = s["x"]
    got = G.detffn_join_backward(r, s["z"], s["dr"], s["dy"], s["w_post"], s["gate"], 0.75, s["w_pre"], 1e-5)
    ref = backward64(s, r, 0.75, 1e-5)
    sums = -(-M // 304) + 46
    for name, (v, mag) in ref.items():
        t = getattr(got, name)
        over_tokens = name in ("dw_pre", "dw_post") or (name == "dgate" and gate in ("scalar", "feature"))
        close(t, v, mag, pt if name in ("dw_pre", "dw_post", "dgate") else dt, 300 + (sums if over_tokens else 0) +
              (86 if gate in ("scalar", "token") else 0))
        assert t.shape == v.shape
    for name in ("dw_pre", "dw_post", "dgate"):
        assert (getattr(got, name) is None) == (name not in ref)


# Many rows to every group of threads, so that rings turn several times: whole
# vectors, other rows, and rows that several thread blocks share.  (The chains of
# the column sums: rows of a thread, groups of a block, 152 blocks or fewer; the
# bound of test_backward holds them all.)
@pytest.mark.parametrize("gate", ["none", "feature", "scalar", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("M,H,dt", [(10949, 264, "bf16"), (10949, 261, "f16"), (4001, 264, "f32"), (687, 4104, "bf16"),
                                    (1301, 2560, "f16"), (900, 5120, "bf16"), (450, 9216, "bf16"), (300, 12296, "f16"),
                                    (310, 9001, "f16")])
def test_many_rows(G, M, H, dt, gate, post, pre):
    test_forward(G, M, H, dt, dt, gate, post, pre)
    test_backward(G, M, H, dt, dt, gate, post, pre)


def test_backward_without_dr(G):
    s = inputs(6, 300, "f32", "f32", "feature", 5)
    got = G.detffn_join_backward(s["x"], s["z"], None, s["dy"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    for name, (v, mag) in backward64(s, s["x"], 1.0, 1e-6, with_dr=False).items():
        close(getattr(got, name), v, mag, "f32", 400)


def test_backward_of_the_norm_alone(G):
    s = inputs(6, 300, "f32", "f32", "none", 6)
    got = G.detffn_join_backward(s["x"], dr=s["dr"], dy=s["dy"], w_pre=s["w_pre"])
    s["w_post"] = None
    ref = backward64(s, s["x"], 1.0, 1e-6)
    assert got.dz is None and got.dw_post is None and got.dgate is None
    for name in ("dx", "dw_pre"):
        close(getattr(got, name), *ref[name], "f32", 400)


@pytest.mark.parametrize("gate", ["none", "scalar", "feature", "token", "full"])
def test_gradients_against_differences(G, gate):
    """Central differences of a random projection of the FP32 forward.  The
    step 2^-6 along a unit-variance direction leaves a third-order error below
    2^-10 of the derivative's scale; FP32 rounding of the projections (about
    1e-6 of their size) over the step adds 1e-4."""
    M, H = 4, 96
    s = inputs(M, H, "f32", "f32", gate, 11)
    f = lambda v: G.detffn_join_forward(v["x"], v["z"], v["w_post"], v["gate"], 0.6, v["w_pre"], 1e-3)  # noqa: E731
    out, _ = f(s)
    got = G.detffn_join_backward(out, s["z"], s["dr"], s["dy"], s["w_post"], s["gate"], 0.6, s["w_pre"], 1e-3)
    proj = lambda v: float((v[0].double() * s["dr"].double()).sum() + (v[1].double() * s["dy"].double()).sum())  # noqa: E731
    grad = {"x": got.dx, "z": got.dz, "w_post": got.dw_post, "w_pre": got.dw_pre, "gate": got.dgate}
    for name, gr in grad.items():
        if gr is None:
            continue
        torch.manual_seed(1)
        v = torch.randn_like(s[name])
        h = 2.0 ** -6
        up, dn = dict(s), dict(s)
        up[name], dn[name] = s[name] + h * v, s[name] - h * v
        num = (proj(f(up)) - proj(f(dn))) / (2 * h)
        ana = float((gr.double() * v.double()).sum())
        scale = float((gr.double() * v.double()).square().sum().sqrt()) + 1.0
        assert abs(num - ana) <= 4e-3 * scale, (name, num, ana)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,pad,shift", [(256, 8, 0), (256, 3, 0), (250, 6, 1), (4096, 8, 8)])
def test_row_strides_and_offsets_equal_contiguous(G, dt, H, pad, shift):
    M = 11
    s = inputs(M, H, dt, dt, "full", 21)
    ref = G.detffn_join_forward(s["x"], s["z"], s["w_post"], s["gate"], 1.5, s["w_pre"])
    refb = G.detffn_join_backward(s["x"], s["z"], s["dr"], s["dy"], s["w_post"], s["gate"], 1.5, s["w_pre"])

    def wide(t):
        b = torch.full((M, H + pad + shift), 3.0, dtype=t.dtype, device="cuda")
        v = b[:, shift:shift + H]
        v.copy_(t)
        return b, v

    v = {n: (t if t is None or t.dim() == 1 else wide(t)[1]) for n, t in s.items()}
    ob, out = wide(torch.zeros_like(s["x"]))
    yb, y = wide(torch.zeros_like(s["x"]))
    G.detffn_join_forward(v["x"], v["z"], v["w_post"], v["gate"], 1.5, v["w_pre"], out=out, y=y)
    got = G.detffn_join_backward(v["x"], v["z"], v["dr"], v["dy"], v["w_post"], v["gate"], 1.5, v["w_pre"])
    u = DT[dt][1] if dt != "f32" else 2.0 ** -20
    for a, b in [(out, ref[0]), (y, ref[1])] + [(getattr(got, n), getattr(refb, n)) for n in got._fields]:
        assert torch.allclose(a.double(), b.double(), rtol=2 * u, atol=2e-5 if dt == "f32" else 2e-2)
    for b in (ob, yb):   # nothing outside the rows was written
        assert bool((b[:, :shift] == 3).all()) and bool((b[:, shift + H:] == 3).all())


@pytest.mark.parametrize("H", [256, 257])
def test_in_place(G, H):
    s = inputs(6, H, "bf16", "bf16", "feature", 31)
    ref = G.detffn_join_forward(s["x"], s["z"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    refb = G.detffn_join_backward(s["x"], s["z"], s["dr"], s["dy"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    x = s["x"].clone()
    out, y = G.detffn_join_forward(x, s["z"], s["w_post"], s["gate"], 1.0, s["w_pre"], out=x)
    assert out is x and torch.equal(out, ref[0]) and torch.equal(y, ref[1])
    dr, z = s["dr"].clone(), s["z"].clone()
    got = G.detffn_join_backward(s["x"], z, dr, s["dy"], s["w_post"], s["gate"], 1.0, s["w_pre"], dx=dr, dz=z)
    assert all(torch.equal(getattr(got, n), getattr(refb, n)) for n in got._fields)


def test_empty(G):
    s = inputs(0, 64, "bf16", "f32", "feature", 1)
    out, y = G.detffn_join_forward(s["x"], s["z"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    assert out.shape == y.shape == (0, 64)
    got = G.detffn_join_backward(s["x"], s["z"], s["dr"], s["dy"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    assert got.dx.shape == (0, 64) and not got.dw_pre.any() and not got.dw_post.any() and not got.dgate.any()


def test_rows_that_are_not_finite_stay_in_their_row(G):
    s = inputs(8, 520, "bf16", "f32", "token", 41)
    ref = G.detffn_join_forward(s["x"], s["z"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    refb = G.detffn_join_backward(s["x"], s["z"], s["dr"], s["dy"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    z, x = s["z"].clone(), s["x"].clone()
    z[2, 5], x[4, 7], z[6] = float("nan"), float("inf"), 0.0
    out, y = G.detffn_join_forward(x, z, s["w_post"], s["gate"], 1.0, s["w_pre"])
    got = G.detffn_join_backward(x, z, s["dr"], s["dy"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    ok = [0, 1, 3, 5, 7]
    assert bool(out[2].isnan().all()) and bool(y[2].isnan().all()) and bool(y[4, 7].isnan())
    assert torch.equal(out[6], x[6])                     # a row of zeros: eps keeps the norm finite
    for a, b in ((out, ref[0]), (y, ref[1]), (got.dx, refb.dx), (got.dz, refb.dz), (got.dgate, refb.dgate)):
        assert torch.equal(a[ok], b[ok])


def test_repeats_and_other_streams(G):
    s = inputs(1000, 1024, "bf16", "f32", "feature", 51)
    args = (s["z"], s["dr"], s["dy"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    a = G.detffn_join_backward(s["x"], *args)
    f = G.detffn_join_forward(s["x"], s["z"], s["w_post"], s["gate"], 1.0, s["w_pre"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        b = G.detffn_join_backward(s["x"], *args, stream=side)
        g = G.detffn_join_forward(s["x"], s["z"], s["w_post"], s["gate"], 1.0, s["w_pre"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(a, b)) and all(torch.equal(p, q) for p, q in zip(f, g))


def test_refusals(G):
    s = inputs(4, 64, "bf16", "f32", "feature", 61)
    x, z = s["x"], s["z"]
    with pytest.raises(ValueError):
        G.detffn_join_forward(x.t(), z)                                      # rows not contiguous
    with pytest.raises(ValueError):
        G.detffn_join_forward(x, z.float())                                  # another dtype
    with pytest.raises(ValueError):
        G.detffn_join_forward(x, z, gate=s["gate"].half())                   # parameters in a third dtype
    with pytest.raises(ValueError):
        G.detffn_join_forward(x, z, gate=s["gate"][:32])                     # no such shape
    with pytest.raises(ValueError):
        G.detffn_join_forward(x, z, gate=s["gate"].expand(4, 64))            # expanded over tokens
    with pytest.raises(ValueError):
        G.detffn_join_forward(x.cpu(), z.cpu())
    with pytest.raises(ValueError):
        G.detffn_join_backward(x, z, s["dr"], s["dy"])                       # dy without w_pre
    for bad in (dict(out=z), dict(y=x, w_pre=s["w_pre"]), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(G.DetFFNError) as e:
            G.detffn_join_forward(x, z, **bad)
        assert e.value.status == 1
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_join_forward(x)                                             # neither z nor w_pre
    assert e.value.status == 1
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_join_forward(torch.zeros(1, 32769, device="cuda"), torch.zeros(1, 32769, device="cuda"))
    assert e.value.status == 2
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_join_backward(x, z, s["dr"], s["dy"], s["w_post"], s["gate"], 1.0, s["w_pre"],
                               ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    assert np.isfinite(float(G.detffn_join_forward(x, z)[0].float().sum()))  # still works


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("M,H", [(6, 256), (5, 1031), (3, 8192)])
@pytest.mark.parametrize("size,eps", [(1e17, 1e-6), (1e15, 1e-6), (1e13, 1e-6), (1e-6, 0.0), (1e-13, 0.0), (1e-16, 0.0),
                                      (1e-15, 1e-30)])
def test_rows_far_from_one(G, size, eps, M, H, post, pre, dt):
    """Rows whose cube leaves FP32's range while their squares' sum stays in it.
    dy goes along r and dr's part along z, so that the projections taken off are
    as large as what they are taken from; the bounds are those of the other tests."""
    s = inputs(M, H, dt, "f32", "feature", M + H, post, pre)
    s["x"], s["z"] = (s["x"].float() * size).to(DT[dt][0]), (s["z"].float() * size).to(DT[dt][0])
    unit = lambda t: t.float() / size  # noqa: E731
    if pre:
        s["dy"] = (s["dy"].float() * 0.1 + unit(s["x"])).to(DT[dt][0])
        s["dr"] = (s["dr"].float() / size * 0.1 + unit(s["z"]) / size).to(DT[dt][0])
    out, y = G.detffn_join_forward(s["x"], s["z"], s["w_post"], s["gate"], 0.75, s["w_pre"], eps)
    r, mag, yr = forward64(s["x"], s["z"], s["w_post"], s["gate"], 0.75, s["w_pre"], eps)
    close(out, r, mag, dt, 64)
    if pre:
        rms = (r.square().mean(-1, keepdim=True) + eps).sqrt()
        close(y, yr, mag / rms * d(s["w_pre"]).abs() + yr.abs(), dt, 150)
    got = G.detffn_join_backward(s["x"], s["z"], s["dr"], s["dy"], s["w_post"], s["gate"], 0.75, s["w_pre"], eps)
    for name, (v, m) in backward64(s, s["x"], 0.75, eps).items():
        close(getattr(got, name), v, m, "f32" if name in ("dw_pre", "dw_post", "dgate") else dt, 350)


@pytest.mark.parametrize("gate", ["none", "feature", "scalar", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("M,H,dt,pt", [(4096, 4096, "bf16", "bf16"), (2048, 1024, "bf16", "f32"), (9000, 256, "f16", "f16"),
                                       (1200, 2056, "f32", "f32"), (700, 8192, "bf16", "bf16"), (900, 1031, "bf16", "f32"),
                                       (200, 12288, "f16", "f16")])
def test_a_row_does_not_depend_on_the_others(G, M, H, dt, pt, gate, post, pre):
    """A row's out, y, dx and dz have the same bits in a call of one row, of a few and
    of all (a decoded token's and a prompt's): so has dgate where it is a row's own."""
    s = inputs(M, H, dt, pt, gate, 3 * M + H, post, pre)
    row = lambda t, a, b: t if t is None or t.shape[0] != M or t.dim() < 2 else t[a:b]  # noqa: E731
    f = lambda v: G.detffn_join_forward(v["x"], v["z"], v["w_post"], v["gate"], 0.75, v["w_pre"])  # noqa: E731
    full = f(s)
    for a, b in ((0, 1), (M - 1, M), (3, 7), (0, M // 2 + 1), (M // 3, M)):
        part = f({n: row(t, a, b) for n, t in s.items()})
        assert all(p is None or torch.equal(p, w[a:b]) for p, w in zip(part, full)), (a, b)
    g = lambda v: G.detffn_join_backward(v["x"], v["z"], v["dr"], v["dy"], v["w_post"], v["gate"], 0.75, v["w_pre"])  # noqa: E731
    full = g(s)
    for a, b in ((0, 2), (M - 5, M), (M // 3, M)):   # (a token's gate of one row is a shared one)
        part = g({n: row(t, a, b) for n, t in s.items()})
        for n in ("dx", "dz") + (("dgate",) if gate in ("token", "full") else ()):
            assert torch.equal(getattr(part, n), getattr(full, n)[a:b]), (n, a, b)


# Many rows to every cluster of four and of eight thread blocks, forward and
# backward: the exchanged sums take turns in two halves and the rings turn.
@pytest.mark.parametrize("gate", ["none", "feature", "scalar", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("M,H,dt", [(200, 20480, "bf16"), (200, 32761, "f16"), (133, 32768, "f32"), (301, 16392, "bf16")])
def test_many_rows_over_clusters(G, M, H, dt, gate, post, pre):
    test_forward(G, M, H, dt, dt, gate, post, pre)
    test_backward(G, M, H, dt, dt, gate, post, pre)
