"""The mixture-of-experts layer for a few tokens against its definition in 64
bits.

Tolerance, element by element: with e = 2^-24, u the unit roundoff of the
stored type and sums of absolute values, a gate or up value is off by at most
H e S_x (S_x = |x| |W|^T; the tensor cores' partial sums are covered by the
factor 2 below), h by that through |SiLU'| <= 1.1 and up, plus 2^-16 |h| (at
least 16 significant bits are kept of it; FP16's second term is exact to 2^-25),
and out by the weighted sum of those plus u |out|."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11), "f32": (torch.float32, 2.0 ** -24)}
E24 = 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    import gemm_deterministic_bf16_gb300 as G
    from gemm_deterministic_bf16_gb300 import build
    build.build()
    assert G.detffn_get_status() == 0
    return G


def inputs(T, E, H, I, dt, seed, k=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(DT[dt][0])  # noqa: E731
    s = dict(x=n((T, H)), Wr=n((E, H), 0.5 / H ** 0.5), Wg=n((E, I, H), 1 / H ** 0.5), Wu=n((E, I, H), 1 / H ** 0.5),
             Wd=n((E, H, I), 1 / I ** 0.5))
    for _ in range(50):   # no token whose choice hangs on the last bits of an FP32 sum
        top = (s["x"].double() @ s["Wr"].double().T).topk(min(k + 1, E), -1).values
        near = (top[:, :-1] - top[:, 1:] < 2e-5).any(-1)
        if not bool(near.any()):
            break
        s["x"] = torch.where(near[:, None], n((T, H)), s["x"])
    return s


def route64(x, Wr, k, normalize):
    p = torch.softmax(x.double() @ Wr.double().T, -1)
    top, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    w, ids = top[:, :k], ids[:, :k]
    return (w / w.sum(-1, keepdim=True) if normalize else w), ids


def moe64(s, ids, w, dt):
    """out and the bound of its error, given the routing."""
    x = s["x"].double()
    out, bound = torch.zeros_like(x), torch.zeros_like(x)
    H, I = s["Wg"].shape[2], s["Wg"].shape[1]
    u = DT[dt][1]
    for e in ids.unique().tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        wg, wu, wd = (s[n][e].double() for n in ("Wg", "Wu", "Wd"))
        g, up = x[t] @ wg.T, x[t] @ wu.T
        eg, eu = 2 * H * E24 * (x[t].abs() @ wg.abs().T), 2 * H * E24 * (x[t].abs() @ wu.abs().T)
        a = g * torch.sigmoid(g)
        h = a * up
        eh = 1.1 * eg * up.abs() + (a.abs() + 1.1 * eg) * eu + (2.0 ** -16 + 16 * E24) * h.abs() + 2.0 ** -25
        wt = w[t, j, None]
        out[t] += wt * (h @ wd.T)
        bound[t] += wt * (eh @ wd.abs().T + (2 * I + 40) * E24 * (h.abs() @ wd.abs().T))
    return out, bound * (1 + u) + u * out.abs() + 1e-30


def check(G, s, k, normalize, dt, **kw):
    out, ids, w = G.detffn_moe_forward(s["x"], s["Wr"], s["Wg"], s["Wu"], s["Wd"], k, normalize=normalize, **kw)
    assert G.detffn_get_status() == 0
    wr, idr = route64(s["x"], s["Wr"], k, normalize)
    assert torch.equal(ids.long(), idr)
    assert bool(((w.double() - wr).abs() <= 2e-5 * wr + 1e-30).all())
    ref, bound = moe64(s, idr, wr, dt)
    bad = ~((out.double() - ref).abs() <= bound + 2e-5 * ref.abs())
    assert not bool(bad.any()), float(((out.double() - ref).abs() / bound).max())
    return out


# Tokens, experts, top_k, H, I: one token to the most, one expert to many,
# widths inside and across tiles, odd widths (the general kernels).
CASES = [(1, 1, 1, 64, 64), (1, 8, 2, 256, 128), (1, 128, 8, 512, 192), (3, 4, 4, 136, 72), (16, 32, 4, 512, 256),
         (17, 16, 3, 264, 200), (64, 8, 2, 256, 384), (64, 64, 6, 512, 128), (33, 512, 16, 128, 64), (5, 7, 5, 1032, 1416),
         (64, 1, 1, 320, 72), (2, 3, 2, 8, 8), (1, 2, 1, 4096, 768), (40, 5, 2, 2048, 1024)]


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,k,H,I", CASES)
def test_layer(G, T, E, k, H, I, dt, normalize):
    check(G, inputs(T, E, H, I, dt, T + E + H, k), k, normalize, dt)


@pytest.mark.parametrize("T,E,k,H,I", [(12, 8, 8, 2048, 1416), (48, 3, 2, 2056, 4104), (9, 5, 5, 2048, 2000)])
def test_units_that_fill_a_second_round_in_part(G, T, E, k, H, I):
    check(G, inputs(T, E, H, I, "bf16", T + H, k), k, True, "bf16")


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("T,E,k", [(20, 4, 3), (64, 3, 2), (40, 16, 2)])
def test_tokens_that_are_not_finite_stay_alone(G, T, E, k, path):
    """All tokens share tiles with one of NaN, one of infinities and one that overflows h."""
    s = inputs(T, E, 256, 192, "bf16", 3 * T, k)
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"], k)
    want = G.detffn_moe_forward(s["x"], *rest, path=path)
    x = s["x"].clone()
    x[3], x[7], x[11] = float("nan"), float("inf"), 3e38
    got = G.detffn_moe_forward(x, *rest, path=path)
    assert G.detffn_get_status() == 0
    keep = [t for t in range(T) if t not in (3, 7, 11)]
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, want))
    assert bool(got[0][3].isnan().all())


@pytest.mark.parametrize("T,E,k,H,I", [(1, 2, 1, 1, 1), (3, 5, 2, 33, 17), (9, 4, 3, 255, 129), (64, 6, 2, 100, 36)])
@pytest.mark.parametrize("dt", list(DT))
def test_odd_widths(G, T, E, k, H, I, dt):
    check(G, inputs(T, E, H, I, dt, 7 * T + H, k), k, True, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_the_general_kernels_by_option(G, dt):
    check(G, inputs(9, 8, 256, 192, dt, 3, 2), 2, True, dt, path=G.PATH_EXACT)


def test_ties_go_to_the_lowest_index(G):
    """Small whole numbers: every logit is exact, and many are equal."""
    T, E, k, H, I = 32, 48, 8, 64, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    s = inputs(T, E, H, I, "bf16", 5)
    s["x"] = torch.randint(-1, 2, (T, H), generator=g, device="cuda").bfloat16()
    s["Wr"] = torch.randint(-1, 2, (E, H), generator=g, device="cuda").bfloat16()
    s["Wr"][E // 2:] = s["Wr"][:E // 2]
    s["x"][3] = 0                                     # all logits equal
    out, ids, w = G.detffn_moe_forward(s["x"], s["Wr"], s["Wg"], s["Wu"], s["Wd"], k)
    logits = (s["x"].double() @ s["Wr"].double().T)
    ref = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), ref)
    assert ids[3].tolist() == list(range(k)) and torch.equal(w[3], torch.full((k,), 1.0 / k, device="cuda"))


def test_every_token_to_one_expert(G):
    T, E, H, I = 64, 16, 256, 256
    s = inputs(T, E, H, I, "bf16", 8)
    s["Wr"].zero_()
    s["Wr"][11] = s["x"].float().mean(0).bfloat16()
    s["x"] = (s["x"] * 0.1 + s["Wr"][11] * 8)
    out = check(G, s, 1, True, "bf16")
    assert bool(out.any())


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("T,E,k,H,I", [(64, 32, 4, 512, 320), (23, 8, 2, 1024, 192)])
def test_a_token_does_not_depend_on_the_others(G, T, E, k, H, I, path):
    s = inputs(T, E, H, I, "bf16", 13, k)
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"], k)
    full = G.detffn_moe_forward(s["x"], *rest, path=path)
    again = G.detffn_moe_forward(s["x"], *rest, path=path)
    assert all(torch.equal(a, b) for a, b in zip(full, again))
    for rows in ([0], [T - 1], list(range(3, 12)), list(range(T))[::-1]):
        part = G.detffn_moe_forward(s["x"][rows].contiguous(), *rest, path=path)
        assert all(torch.equal(a[rows], b) for a, b in zip(full, part)), rows


def test_a_token_that_is_not_finite_stays_alone(G):
    s = inputs(12, 8, 256, 128, "bf16", 17, 2)
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"], 2)
    ref = G.detffn_moe_forward(s["x"], *rest)
    x = s["x"].clone()
    x[4, 9], x[7, 0] = float("nan"), float("inf")
    out, ids, w = G.detffn_moe_forward(x, *rest)
    ok = [i for i in range(12) if i not in (4, 7)]
    assert all(torch.equal(a[ok], b[ok]) for a, b in zip((out, ids, w), ref))
    assert bool(out[4].isnan().all()) and bool(out[7].isnan().all()) and bool(w[4].isnan().all())
    assert bool((ids >= 0).all()) and bool((ids < 8).all())


def test_empty_streams_and_workspace(G):
    s = inputs(6, 8, 256, 192, "bf16", 19, 2)
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"], 2)
    assert G.detffn_moe_forward(s["x"][:0], *rest)[0].shape == (0, 256)
    ref = G.detffn_moe_forward(s["x"], *rest)
    ws = torch.full((G.detffn_moe_workspace_size(6, 8, 2, 256, 192),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):   # a workspace full of old values, used again and again
        assert all(torch.equal(a, b) for a, b in zip(ref, G.detffn_moe_forward(s["x"], *rest, ws=ws)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        got = G.detffn_moe_forward(s["x"], *rest, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_a_workspace_of_either_16_bit_type_serves_both(G):
    size = lambda dt: G.detffn_moe_workspace_size(6, 8, 2, 256, 192, dtype=dt)  # noqa: E731
    assert size(torch.float16) == size(torch.bfloat16)
    s = inputs(6, 8, 256, 192, "f16", 19, 2)
    ws = torch.empty(G.detffn_moe_workspace_size(6, 8, 2, 256, 192), dtype=torch.uint8, device="cuda")
    check(G, s, 2, True, "f16", ws=ws)


def test_stalled_wait_times_out_and_recovers(G):
    """The test-only stall flag withholds the copies, so the bounded waits run
    out: the call returns, the status says so, a call before it is read leaves
    out untouched, and after that the bits are those of a normal call."""
    s = inputs(9, 8, 512, 256, "bf16", 29, 2)
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"], 2)
    ref = G.detffn_moe_forward(s["x"], *rest, path=G.PATH_TENSOR)[0]
    assert G.detffn_get_status() == 0
    out = torch.full_like(ref, 7.0)
    G.detffn_moe_forward(s["x"], *rest, out=out, path=G.PATH_TENSOR, spin_limit=2048, flags=G.FLAG_TEST_STALL)
    torch.cuda.synchronize()
    again = torch.full_like(ref, 7.0)
    G.detffn_moe_forward(s["x"], *rest, out=again, path=G.PATH_TENSOR)
    torch.cuda.synchronize()
    assert bool((again == 7.0).all())
    assert G.detffn_get_status() == 7 and G.detffn_get_status() == 0
    assert torch.equal(G.detffn_moe_forward(s["x"], *rest, path=G.PATH_TENSOR)[0], ref)
    assert G.detffn_get_status() == 0


def test_refusals(G):
    s = inputs(6, 8, 256, 192, "bf16", 23, 2)
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"])
    big = torch.zeros((65, 256), dtype=torch.bfloat16, device="cuda")
    for x, k in ((big, 2), (s["x"], 9), (s["x"], 0), (s["x"], 17)):
        with pytest.raises(G.DetFFNError) as e:
            G.detffn_moe_forward(x, *rest, k)
        assert e.value.status == 2
    with pytest.raises(ValueError):
        G.detffn_moe_forward(s["x"].float(), *rest, 2)
    with pytest.raises(ValueError):
        G.detffn_moe_forward(s["x"], s["Wr"][:4].contiguous(), *rest[1:], 2)
    with pytest.raises(ValueError):
        G.detffn_moe_forward(s["x"], s["Wr"], s["Wg"].transpose(1, 2), s["Wu"], s["Wd"], 2)
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_moe_forward(s["x"], *rest, 2, out=s["x"])
    assert e.value.status == 1
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_moe_forward(s["x"], *rest, 2, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    odd = inputs(2, 4, 33, 17, "bf16", 3)
    with pytest.raises(G.DetFFNError) as e:          # the tensor kernels take widths that are multiples of 8
        G.detffn_moe_forward(odd["x"], odd["Wr"], odd["Wg"], odd["Wu"], odd["Wd"], 1, path=G.PATH_TENSOR)
    assert e.value.status == 4
    for bad in (dict(flags=2), dict(path=5), dict(spin_limit=-1)):
        with pytest.raises(G.DetFFNError) as e:
            G.detffn_moe_forward(s["x"], *rest, 2, **bad)
        assert e.value.status == 1


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,k,H,I", [(7, 16, 2, 2048, 1416), (64, 32, 4, 512, 320), (1, 8, 8, 1024, 768)])
def test_h_of_other_thread_blocks_is_seen(G, T, E, k, H, I, dt):
    """Down units load rows of h that other thread blocks have just written.  The
    workspace is filled with NaN before each call, so a load that came too early
    would show."""
    s = inputs(T, E, H, I, dt, T + 31, k)
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"], k)
    want = check(G, s, k, True, dt)
    ws = torch.empty(G.detffn_moe_workspace_size(T, E, k, H, I, DT[dt][0]), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        ws.fill_(255)
        assert torch.equal(G.detffn_moe_forward(s["x"], *rest, ws=ws)[0], want)
    assert G.detffn_get_status() == 0


def moe64_wide(s, ids, w, u):
    """As moe64, with the bound of h as the header states it: 2^-16 of a value, or of
    2^-13 where that is more."""
    x = s["x"].double()
    out, bound = torch.zeros_like(x), torch.zeros_like(x)
    H, I = s["Wg"].shape[2], s["Wg"].shape[1]
    for e in ids.unique().tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        wg, wu, wd = (s[n][e].double() for n in ("Wg", "Wu", "Wd"))
        g, up = x[t] @ wg.T, x[t] @ wu.T
        eg, eu = 2 * H * E24 * (x[t].abs() @ wg.abs().T), 2 * H * E24 * (x[t].abs() @ wu.abs().T)
        a = g * torch.sigmoid(g)
        h = a * up
        top = h.abs().amax(-1, keepdim=True)
        low = torch.where(top >= 2.0 ** -13 * (1 - 1e-3), 2.0 ** -13, 0.0)
        eh = 1.1 * eg * up.abs() + (a.abs() + 1.1 * eg) * eu + (2.0 ** -16 + 16 * E24) * torch.maximum(h.abs(), low)
        wt = w[t, j, None]
        out[t] += wt * (h @ wd.T)
        bound[t] += wt * (eh @ wd.abs().T + (2 * I + 40) * E24 * (h.abs() @ wd.abs().T))
    return out, bound * (1 + u) + u * out.abs() + 2.0 ** -25


# The size of h and the standard deviation of Wd.
@pytest.mark.parametrize("size,wd", [(1e5, 2e-3), (2e6, 1e-4), (3e7, 1e-5), (1e9, 3e-7), (1e-4, 30.0), (1e-5, 300.0), (1e-7, 1e4)])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 128), (9, 8, 3, 264, 200), (64, 6, 2, 512, 320), (3, 2, 1, 2056, 1000)])
@pytest.mark.parametrize("path", [1, 2])
def test_fp16_hidden_values_far_from_one(G, size, wd, T, E, k, H, I, path):
    """h beyond FP16's largest number, and so small that FP16's steps are coarse,
    where the output itself is an ordinary number."""
    s = inputs(T, E, H, I, "f16", T + H, k)
    f = size ** 0.5
    s["Wg"], s["Wu"] = ((s[n].float() * f).half() for n in ("Wg", "Wu"))
    if size < 1:
        # SiLU(g) is g / 2 there
        s["Wg"] = (s["Wg"].float() * 2).half()
    s["Wd"] = (s["Wd"].float() * (I ** 0.5 * wd)).half()
    out, ids, w = G.detffn_moe_forward(s["x"], s["Wr"], s["Wg"], s["Wu"], s["Wd"], k, path=path)
    assert G.detffn_get_status() == 0
    wr, idr = route64(s["x"], s["Wr"], k, True)
    assert torch.equal(ids.long(), idr)
    ref, bound = moe64_wide(s, idr, wr, DT["f16"][1])
    assert float(ref.abs().max()) < 65504 and bool(out.isfinite().all())
    bad = ~((out.double() - ref).abs() <= bound + 2e-5 * ref.abs())
    assert not bool(bad.any()), float(((out.double() - ref).abs() / bound).max())


def test_fp16_tokens_of_any_size_stay_alone(G):
    """Tokens whose h the tensor cores' two terms hold, and others, in one call."""
    T, E, H, I, k = 24, 4, 512, 328, 2
    s = inputs(T, E, H, I, "f16", 77, k)
    s["Wd"] = (s["Wd"].float() * 1e-3).half()
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"], k)
    want = G.detffn_moe_forward(s["x"], *rest)
    x = s["x"].clone()
    x[2], x[3], x[9], x[10], x[17] = x[2] * 3000, x[3] * 1e-4, 0.0, float("inf"), float("nan")
    got = G.detffn_moe_forward(x, *rest)
    keep = [t for t in range(T) if t not in (2, 3, 9, 10, 17)]
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, want))
    for t in (2, 3, 9, 10, 17):   # and each is what it is alone
        assert torch.equal(G.detffn_moe_forward(x[t:t + 1].contiguous(), *rest)[0][0].nan_to_num(7.0), got[0][t].nan_to_num(7.0))
    assert bool(got[0][2].isfinite().all()) and not bool(got[0][9].any()) and bool(got[0][17].isnan().all())


@pytest.mark.parametrize("path", [1, 2])
def test_bf16_hidden_values_beyond_its_largest(G, path):
    """h = 2^128 (1 - 2^-10) is an FP32 number that rounds to BF16's infinity."""
    x = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, :2] = 1
    Wg, Wu = (torch.zeros((1, 64, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Wg[0, :, 0], Wg[0, :, 1], Wu[0, :, 0] = 2.0 ** 64, -2.0 ** 54, 2.0 ** 64
    Wd = torch.zeros((1, 64, 64), dtype=torch.bfloat16, device="cuda")
    Wd[0, :, 5] = 2.0 ** -120
    out = G.detffn_moe_forward(x, torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda"), Wg, Wu, Wd, 1, path=path)[0]
    assert torch.equal(out.float(), torch.full_like(out, 256.0, dtype=torch.float32))



@pytest.mark.parametrize("path,name,launches", [(2, "moe_tensor", 2), (1, "moe_general", 5)])
def test_profiling_records_the_layer(G, path, name, launches):
    T, E, k, H, I = 3, 8, 2, 256, 192
    s = inputs(T, E, H, I, "bf16", 41, k)
    rest = (s["Wr"], s["Wg"], s["Wu"], s["Wd"], k)
    want = G.detffn_moe_forward(s["x"], *rest, path=path)
    G.detffn_profiling(True)
    got = [G.detffn_moe_forward(s["x"], *rest, path=path) for _ in range(4)]
    ops = G.detffn_profile_read()
    G.detffn_profiling(False)
    assert list(ops) == [name] and ops[name]["launches"] == 4 * launches and ops[name]["ms"] > 0
    assert ops[name]["bytes"] == 4 * 2 * (2 * T * H + E * H + T * k * 3 * H * I)
    assert ops[name]["flops"] == 4 * (2 * T * E * H + 6 * T * k * H * I)
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    G.detffn_moe_forward(s["x"], *rest, path=path)
    assert not G.detffn_profile_read()


@pytest.mark.parametrize("path", [1, 2])
def test_gates_at_the_end_of_the_range(G, path):
    """SiLU(-88) is -88 exp(-88), and exp(88) is a number, though more than 2^126;
    exp(90) is not one, and SiLU(-90) is.  One feature's h to each output."""
    H = I = 64
    g = torch.tensor([-80.0, -86.0, -87.5, -88.0, -88.5, -89.0, -89.5, -90.0]).repeat(8)
    x, Wr = torch.zeros((1, H)), torch.zeros((1, H))
    Wg, Wu = torch.zeros((1, I, H)), torch.zeros((1, I, H))
    x[0, 0] = 1
    Wg[0, :, 0], Wu[0, :, 0] = g, 2.0 ** 120
    t = [v.bfloat16().cuda() for v in (x, Wr, Wg, Wu, torch.eye(I)[None])]
    out = G.detffn_moe_forward(*t, 1, path=path)[0][0].cpu().double()
    h = g.double() * torch.sigmoid(g.double()) * 2.0 ** 120
    # (exp(-90) is subnormal in FP32, in steps of 2^-19 of it at the most)
    assert bool(((out - h).abs() <= (2.0 ** -8 + 2.0 ** -15) * h.abs()).all()), (out / h)
