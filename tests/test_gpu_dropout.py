"""Dropout against the generator evaluated in Python integers, element by element.

Tolerance: one FP32 product with 1 / (1 - p) rounded to FP32, and a sum: three
roundings of 2^-24 of |x| / (1 - p) and |residual|, then half a step of the type."""
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


def philox(c, k):
    c, k = list(c), list(k)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def test_generator_known_answers():
    """The published vectors of Philox4x32-10."""
    assert philox((0,) * 4, (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert philox((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def mask(M, H, p, seed, offset):
    limit = int(p * 4294967296.0)
    split = lambda v: (v & 0xFFFFFFFF, v >> 32)  # noqa: E731
    rows = []
    for m in range(M):
        w = []
        for c in range((H + 3) // 4):
            w += philox((c, m, *split(offset)), split(seed))
        rows.append([v >= limit for v in w[:H]])
    return torch.tensor(rows, device="cuda").view(M, H)


def check(got, x, res, keep, p):
    x64 = torch.where(keep, x.double(), 0.0) / (1 - p) if p < 1 else torch.zeros_like(x.double())
    r64 = res.double() if res is not None else torch.zeros_like(x64)
    want = x64 + r64
    tol = 3 * 2.0 ** -24 * (x64.abs() + r64.abs()) + HALF[x.dtype] * want.abs() * (1 + 2.0 ** -8) + \
        (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    assert bool(((got.double() - want).abs() <= tol).all())
    if res is None:
        assert not bool(got[~keep].any())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("M,H", [(1, 1), (1, 8), (3, 64), (7, 13), (5, 1031), (33, 40), (2, 4096)])
def test_forward_and_backward(G, M, H, dtype):
    x, r = (torch.randn((M, H), device="cuda").to(dtype) for _ in range(2))
    for p, seed, offset in ((0.1, 1, 0), (0.5, (1 << 64) - 1, 1 << 40), (0.999, 12345678901234567, 7)):
        keep = mask(M, H, p, seed, offset)
        check(G.detffn_dropout_forward(x, p, seed, offset), x, None, keep, p)
        check(G.detffn_dropout_forward(x, p, seed, offset, residual=r), x, r, keep, p)
        check(G.detffn_dropout_backward(x, p, seed, offset), x, None, keep, p)


@pytest.mark.parametrize("dtype", ALL)
def test_ends_of_p(G, dtype):
    x, r = (torch.randn((9, 72), device="cuda").to(dtype) for _ in range(2))
    assert torch.equal(G.detffn_dropout_forward(x, 0.0, 3), x)
    bad = x.clone()
    bad[2] = float("nan")
    bad[3] = float("inf")
    assert not bool(G.detffn_dropout_forward(bad, 1.0, 3).any())
    assert torch.equal(G.detffn_dropout_forward(bad, 1.0, 3, residual=r), r)
    out, keep = G.detffn_dropout_forward(bad, 0.5, 3), mask(9, 72, 0.5, 3, 0)
    assert not bool(out[~keep].any()) and not bool(out[2:4][keep[2:4]].isfinite().any())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("H,pad,at", [(64, 8, 8), (64, 3, 1), (37, 5, 2), (200, 0, 0)])
def test_strides_and_in_place(G, H, pad, at, dtype):
    """The mask does not depend on strides, alignment or the number of rows; out may be x or the residual."""
    wide, rwide = (torch.randn((11, H + pad), device="cuda").to(dtype) for _ in range(2))
    x, r = wide[:, at:at + H], rwide[:, at:at + H]
    want = G.detffn_dropout_forward(x.contiguous(), 0.3, 5, 6, residual=r.contiguous())
    to = torch.full((11, H + 4), float("nan"), dtype=dtype, device="cuda")
    assert torch.equal(G.detffn_dropout_forward(x, 0.3, 5, 6, residual=r, out=to[:, 1:H + 1]), want)
    assert bool(to[:, 0].isnan().all()) and bool(to[:, H + 1:].isnan().all())
    assert torch.equal(G.detffn_dropout_forward(x[:4].contiguous(), 0.3, 5, 6, residual=r[:4].contiguous()), want[:4])
    a, b = wide.clone(), rwide.clone()
    assert torch.equal(G.detffn_dropout_forward(a[:, at:at + H], 0.3, 5, 6, residual=r, out=a[:, at:at + H]), want)
    assert torch.equal(G.detffn_dropout_forward(x, 0.3, 5, 6, residual=b[:, at:at + H], out=b[:, at:at + H]), want)
    for m, old in ((a, wide), (b, rwide)):
        assert torch.equal(m[:, :at], old[:, :at]) and torch.equal(m[:, at + H:], old[:, at + H:])


def test_many_rows(G):
    """More units than a grid's threads: words of far rows and columns, the share kept, and the gradient's mask."""
    M, H, p, seed = 3001, 1032, 0.25, 99
    x = torch.ones((M, H), device="cuda")
    out = G.detffn_dropout_forward(x, p, seed, 4)
    for m, c in ((0, 0), (3000, 1031), (1500, 517), (2999, 4)):
        keep = philox((c // 4, m, 4, 0), (seed, 0))[c % 4] >= int(p * 4294967296.0)
        assert bool(out[m, c] != 0) == keep
    # Of n independent trials the share kept is within 6 standard deviations of 1 - p.
    assert abs(float((out != 0).double().mean()) - 0.75) < 6 * (0.25 * 0.75 / (M * H)) ** 0.5
    assert torch.equal(G.detffn_dropout_backward(x, p, seed, 4), out)
    assert not torch.equal(G.detffn_dropout_forward(x, p, seed, 5), out)


def test_state_on_the_device(G):
    """Seed and base from a tensor, read when the kernel runs: replays of a captured call draw new masks."""
    x = torch.randn((16, 128), device="cuda").bfloat16()
    state = torch.tensor([17, 40], device="cuda")
    assert torch.equal(G.detffn_dropout_forward(x, 0.4, state, 2), G.detffn_dropout_forward(x, 0.4, 17, 42))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = G.detffn_dropout_forward(x, 0.4, state, 2)
        d = G.detffn_dropout_backward(y, 0.4, state, 2)
    for base in (40, 41, -1):
        state[1] = base
        graph.replay()
        want = G.detffn_dropout_forward(x, 0.4, 17, (base + 2) % (1 << 64))
        assert torch.equal(y, want) and torch.equal(d, G.detffn_dropout_backward(want, 0.4, 17, (base + 2) % (1 << 64)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = G.detffn_dropout_forward(x, 0.4, 17, 42, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, G.detffn_dropout_forward(x, 0.4, 17, 42))


def test_no_rows_and_refusals(G):
    x = torch.randn((4, 64), device="cuda").bfloat16()
    assert G.detffn_dropout_forward(x[:0], 0.1, 1).shape == (0, 64)
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(G.DetFFNError) as e:
            G.detffn_dropout_forward(x, p, 1)
        assert e.value.status == 1
    for bad in (dict(seed=-1), dict(seed=1 << 64), dict(seed=1, offset=-1), dict(seed=torch.zeros(2)),
                dict(seed=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(seed=1, residual=x[:2]),
                dict(seed=1, residual=x.float()), dict(seed=1, out=x.float())):
        with pytest.raises(ValueError):
            G.detffn_dropout_forward(x, 0.1, **bad)
    with pytest.raises(TypeError):
        G.detffn_dropout_forward(x, 0.1, 1.5)
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_dropout_forward(x[:2], 0.1, 1, out=x[1:3])
    assert e.value.status == 1


def test_addresses_beyond_32_bits(G):
    """More than 2^32 elements: the words of the last rows, and rows of a wide stride."""
    M, H, p, seed = (1 << 20) + 5, 4104, 0.3, 11
    x = torch.ones((M, H), dtype=torch.bfloat16, device="cuda")
    out = G.detffn_dropout_forward(x, p, seed, 2, out=x)
    limit = int(p * 4294967296.0)
    for m in (0, 1 << 19, M - 1):
        for c in (0, 1, 2051, H - 1):
            assert bool(out[m, c] != 0) == (philox((c // 4, m, 2, 0), (seed, 0))[c % 4] >= limit)
    last = torch.ones((M, 8), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(G.detffn_dropout_forward(last, p, seed, 2)[M - 9:], out[M - 9:, :8])
