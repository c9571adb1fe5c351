"""4-bit weights: the layout against its formula, packing against its rule, the
products against 64-bit ones.

Tolerance of a product: with n the steps from a code to the result, each off by
at most 2^-23 (a group's sum, at most 128 products in any order that may cut off,
the scale, the sum of the groups, the warps' and terms' sums), the error is at
most n 2^-23 of the sum of the magnitudes, n = 128 + 1 + K / 32 + 16; then half a
step of the stored type."""
import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ALL = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def G():
    import gemm_deterministic_bf16_gb300 as G
    from gemm_deterministic_bf16_gb300 import build
    build.build()
    return G


def place(K):
    """Byte and nibble of each code of a row."""
    k = torch.arange(K)
    g, t, j = k % 128 // 32, k % 32 // 8, k % 8
    p = j // 2 + 4 * (j % 2)
    return k // 128 * 64 + 4 * (4 * t + g) + p // 2, p % 2


def codes_of(w4):
    byte, nib = place(w4.K)
    c = w4.codes.cpu()[:, byte].long()
    return torch.where(nib == 1, c >> 4, c & 15)


def values64(w4):
    k = torch.arange(w4.K)
    return ((codes_of(w4) - 8).double() * w4.scales.cpu().double()[:, k // w4.group]).cuda()


def matrix(G, N, K, group, st, seed=0):
    """Codes of all sixteen values and scales over a wide range."""
    g = torch.Generator(device="cuda").manual_seed(seed + N + K)
    codes = torch.randint(0, 256, (N, (K + 127) // 128 * 64), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.randn((N, (K + group - 1) // group), generator=g, device="cuda") * 0.01).to(st)
    return G.W4(codes, scales, K, group)


def check(got, x, v, dtype, K):
    want, size = x.double() @ v.T, x.double().abs() @ v.abs().T
    tol = (145 + K / 32) * 2.0 ** -23 * size + HALF[dtype] * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -25 * (dtype == torch.float16)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float((got.double() - want).abs().max()))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(1, 16, 128), (1, 1, 1), (2, 33, 257), (3, 100, 1416), (8, 64, 4096), (9, 40, 640),
                                   (17, 130, 384), (33, 48, 129), (64, 31, 1000), (5, 7, 31)])
def test_matvec(G, T, N, K, group, dtype):
    for st in {dtype, torch.float32, torch.bfloat16}:
        w = matrix(G, N, K, group, st)
        x = torch.randn((T, K), generator=torch.Generator(device="cuda").manual_seed(K), device="cuda").to(dtype)
        check(G.detffn_w4_matvec(x, w), x, values64(w), dtype, K)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("N,K", [(64, 4096), (40, 515)])
def test_matvec_strides_and_single_tokens(G, N, K, dtype):
    w = matrix(G, N, K, 64, dtype)
    wide = torch.randn((20, K + 9), device="cuda").to(dtype)
    x = wide[:, 1:K + 1]
    to = torch.full((20, N + 5), float("nan"), dtype=dtype, device="cuda")
    out = G.detffn_w4_matvec(x, w, out=to[:, 2:N + 2])
    check(out, x, values64(w), dtype, K)
    assert bool(to[:, :2].isnan().all()) and bool(to[:, N + 2:].isnan().all())
    dense = G.detffn_w4_matvec(x.contiguous(), w)
    assert torch.equal(dense, out)
    for t in (0, 7, 19):   # a token alone has the bits it has among others
        assert torch.equal(G.detffn_w4_matvec(x[t:t + 1].contiguous(), w), dense[t:t + 1])


@pytest.mark.parametrize("dtype", ALL)
def test_values_that_are_not_finite(G, dtype):
    w = matrix(G, 24, 300, 32, torch.float32)
    x = torch.randn((4, 300), device="cuda").to(dtype)
    x[1, 5] = float("nan")
    x[2, 299] = float("inf")
    out = G.detffn_w4_matvec(x, w)
    assert bool(out[1].isnan().all()) and not bool(out[2].isfinite().any()) and bool(out[0].isfinite().all())
    c = codes_of(w)[:, 299].cuda() - 8
    s = c * w.scales[:, -1].sign()
    want = torch.where(s == 0, float("nan"), s.sign() * float("inf"))
    assert torch.equal(out[2].float().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
    # FP32's largest and smallest values keep their digits.
    if dtype == torch.float32:
        x = torch.zeros((2, 300), device="cuda")
        x[0, 0], x[1, 0] = 3.4e38, 1e-30
        one = G.W4(torch.full_like(w.codes, 0x99), torch.ones_like(w.scales), 300, 32)
        assert torch.equal(G.detffn_w4_matvec(x, one), x[:, :1].expand(2, 24))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(5, 128), (3, 1000), (33, 257), (1, 1)])
def test_pack_and_unpack(G, N, K, group, dtype):
    g = torch.Generator(device="cuda").manual_seed(N * K)
    wide = torch.randn((N, K + 3), generator=g, device="cuda").to(dtype)
    w = wide[:, 1:K + 1]
    w[0, :K // 2] = 0
    for st in {dtype, torch.float32}:
        w4 = G.detffn_w4_pack(w, group, st)
        pad = -K % group
        b = torch.nn.functional.pad(w.float(), (0, pad)).view(N, -1, group)
        top = b.abs().amax(-1)
        scale = (top / torch.full_like(top, 7.0)).to(st)   # (a division by a Python number multiplies by 1 / 7)
        q = torch.where(scale[..., None] > 0, b / scale.float()[..., None], 0.0).round().clamp(-7, 7).view(N, -1)[:, :K]
        assert torch.equal(w4.scales, scale) and torch.equal(codes_of(w4), (q + 8).long().cpu())
        for to in ALL:
            v = G.detffn_w4_unpack(w4, dtype=to)
            assert torch.equal(v, values64(w4).float().to(to))   # (a 4-bit number times a scale of 24 bits: FP32 rounds once)
        again = G.detffn_w4_pack(w, group, w4=w4)
        assert again.codes.data_ptr() == w4.codes.data_ptr() and torch.equal(codes_of(again), (q + 8).long().cpu())


def test_pack_of_what_has_no_scale(G):
    w = torch.ones((4, 256), device="cuda")
    w[0, 3], w[1, 130], w[2] = float("inf"), float("nan"), 1e-46
    w[3] = 3e38
    p = G.detffn_w4_pack(w, 128, torch.float32)
    assert bool(p.scales[0, 0].isnan()) and bool(p.scales[1, 1].isnan()) and p.scales[2].tolist() == [0, 0]
    v = G.detffn_w4_unpack(p, dtype=torch.float32)
    assert bool(v[0, :128].isnan().all()) and bool((v[0, 128:] == 1).all()) and not bool(v[2].any())
    assert bool(G.detffn_w4_pack(w, 128, torch.float16).scales[3].isnan().all())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("T,H,I,group", [(1, 256, 512, 128), (1, 100, 77, 32), (4, 384, 1000, 64), (16, 128, 768, 128),
                                         (33, 129, 260, 64), (64, 64, 64, 32)])
def test_ffn(G, T, H, I, group, dtype):
    """The hidden activation h is off by the two products' errors, passed on
    through the third: each of its relative steps counts once more on sum |h| |w|.
    SiLU adds 8 steps of 2^-23; h's terms (16 bits, cut off) 2^-15 of it for a
    16-bit result."""
    Wg, Wu, Wd = matrix(G, I, H, group, dtype), matrix(G, I, H, group, dtype, 1), matrix(G, H, I, group, dtype, 2)
    x = torch.randn((T, H), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").to(dtype)
    x64, g64, u64, d64 = x.double(), values64(Wg), values64(Wu), values64(Wd)
    g, u = x64 @ g64.T, x64 @ u64.T
    h = g * torch.sigmoid(g) * u
    eps = (145 + H / 32) * 2.0 ** -23
    dg, du = eps * (x64.abs() @ g64.abs().T), eps * (x64.abs() @ u64.abs().T)
    dh = 1.1 * dg * u.abs() + g.abs() * du + 1.1 * dg * du + 8 * 2.0 ** -23 * h.abs()   # |SiLU'| <= 1.1, |SiLU(g)| <= |g|
    dh = dh + (0.0 if dtype == torch.float32 else 2.0 ** -15) * (h.abs() + dh)
    want = h @ d64.T
    tol = (dh + (145 + I / 32) * 2.0 ** -23 * (h.abs() + dh)) @ d64.abs().T + HALF[dtype] * want.abs() * (1 + 2.0 ** -8) + \
        2.0 ** -25 * (dtype == torch.float16)
    out = G.detffn_w4_forward(x, Wg, Wu, Wd)
    assert bool(((out.double() - want).abs() <= tol).all())
    for t in {0, T - 1}:
        assert torch.equal(G.detffn_w4_forward(x[t:t + 1].contiguous(), Wg, Wu, Wd), out[t:t + 1])
    assert torch.equal(G.detffn_w4_forward(x, Wg, Wu, Wd, out=x), out)   # in place


def test_streams_and_graphs(G):
    Wg, Wu, Wd = matrix(G, 512, 256, 128, torch.bfloat16), matrix(G, 512, 256, 128, torch.bfloat16, 1), matrix(G, 256, 512, 128, torch.bfloat16, 2)
    x = torch.randn((3, 256), device="cuda").bfloat16()
    want = G.detffn_w4_forward(x, Wg, Wu, Wd)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = G.detffn_w4_forward(x, Wg, Wu, Wd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = G.detffn_w4_forward(x, Wg, Wu, Wd)
        z = G.detffn_w4_matvec(y, Wg)
    x.mul_(2)
    graph.replay()
    assert torch.equal(y, G.detffn_w4_forward(x, Wg, Wu, Wd)) and torch.equal(z, G.detffn_w4_matvec(y, Wg))


def test_no_tokens(G):
    w = matrix(G, 16, 64, 32, torch.bfloat16)
    assert G.detffn_w4_matvec(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w).shape == (0, 16)


def test_refusals(G):
    w = matrix(G, 16, 64, 32, torch.bfloat16)
    x = torch.randn((2, 64), device="cuda").bfloat16()
    for bad in ((x[:, :63], w), (x.double(), w), (x.cpu(), w), (x, w._replace(K=200)), (x, w._replace(group=64)),
                (x, w._replace(codes=w.codes.char())), (x, w._replace(scales=w.scales.double()))):
        with pytest.raises(ValueError):
            G.detffn_w4_matvec(*bad)
    with pytest.raises(ValueError):
        G.detffn_w4_forward(x, w, w, w)
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_w4_matvec(torch.zeros((65, 64), device="cuda").bfloat16(), w)
    assert e.value.status == 2
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_w4_pack(x, 16)
    assert e.value.status == 4
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_w4_matvec(x, w._replace(codes=torch.zeros(16 * 64 + 8, dtype=torch.uint8, device="cuda")[8:].view(16, 64)))
    assert e.value.status == 3


def test_addresses_beyond_32_bits(G):
    """Codes of more than 2^32 bytes: the first and the last rows' products."""
    N, K = 1 << 20, 8320
    w = G.W4(torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda"), torch.zeros((N, K // 128), dtype=torch.bfloat16, device="cuda"), K, 128)
    part = matrix(G, 64, K, 128, torch.bfloat16)
    for at in (slice(0, 64), slice(N - 64, N)):
        w.codes[at] = part.codes
        w.scales[at] = part.scales
    x = torch.randn((3, K), device="cuda").bfloat16()
    out = G.detffn_w4_matvec(x, w)
    want = G.detffn_w4_matvec(x, part)
    assert torch.equal(out[:, :64], want) and torch.equal(out[:, N - 64:], want) and not bool(out[:, 64:N - 64].any())
    check(want, x, values64(part), torch.bfloat16, K)
    v = torch.empty((64, K), dtype=torch.float32, device="cuda")
    last = w._replace(codes=w.codes[N - 64:], scales=w.scales[N - 64:])
    assert torch.equal(G.detffn_w4_unpack(last, out=v), values64(part).float())


@pytest.mark.parametrize("dtype", ALL)
def test_long_rows(G, dtype):
    for T in (1, 9):
        w = matrix(G, 24, 100003, 128, torch.float32)
        x = torch.randn((T, 100003), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").to(dtype)
        check(G.detffn_w4_matvec(x, w), x, values64(w), dtype, 100003)


def test_two_streams_at_once(G):
    ws = [matrix(G, 512, 256, 128, torch.bfloat16, i) for i in range(2)] + [matrix(G, 256, 512, 128, torch.bfloat16, 2)]
    xs = [torch.randn((t, 256), device="cuda").bfloat16() for t in (1, 20)]
    want = [G.detffn_w4_forward(x, *ws) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [(n % 2, G.detffn_w4_forward(xs[n % 2], *ws, stream=streams[n // 2 % 2])) for n in range(16)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)
