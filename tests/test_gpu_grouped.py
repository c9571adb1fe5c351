"""Matrix products grouped by expert against 64-bit products.

Tolerance: a sum of n FP32 products, in any order and each step off by at most
one unit of FP32's last place (2^-23: the tensor cores may cut off), is off by at
most n 2^-23 of the sum of the products' magnitudes; rounding to the stored type
adds half a step of the result, and half the smallest step of FP16."""
import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
AUTO, EXACT, TENSOR = 0, 1, 2


@pytest.fixture(scope="module")
def G():
    import gemm_deterministic_bf16_gb300 as G
    from gemm_deterministic_bf16_gb300 import build
    build.build()
    assert G.detffn_get_status() == 0
    yield G
    assert G.detffn_get_status() == 0


def make(sizes, K, N, dtype, seed=0, first=0, behind=0):
    """x, W, dOut and offsets of experts with `sizes` rows, after `first` rows of none and before `behind`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = first + sum(sizes) + behind
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    ends = [first]
    for n in sizes:
        ends.append(ends[-1] + n)
    return r(R, K), r(len(sizes), N, K), r(R, N), torch.tensor(ends, dtype=torch.int32, device="cuda"), ends


def close(got, want, bound, n, dtype):
    tol = n * 2.0 ** -23 * bound + HALF[dtype] * want.abs() * (1 + 2.0 ** -8) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float((got.double() - want).abs().max()), torch.nonzero(bad)[:4].tolist())


def check_forward(G, x, W, off, ends, out, before):
    for e in range(W.shape[0]):
        a, b = ends[e], ends[e + 1]
        x64, w64 = x[a:b].double(), W[e].double()
        close(out[a:b], x64 @ w64.T, x64.abs() @ w64.abs().T, x.shape[1], x.dtype)
    assert torch.equal(out[:ends[0]], before[:ends[0]]) and torch.equal(out[ends[-1]:], before[ends[-1]:])


def check_backward(G, x, W, d, ends, dX, dW, before):
    for e in range(W.shape[0]):
        a, b = ends[e], ends[e + 1]
        x64, w64, d64 = x[a:b].double(), W[e].double(), d[a:b].double()
        close(dX[a:b], d64 @ w64, d64.abs() @ w64.abs(), W.shape[1], x.dtype)
        close(dW[e], d64.T @ x64, d64.abs().T @ x64.abs(), max(b - a, 1), x.dtype)
    assert torch.equal(dX[:ends[0]], before[:ends[0]]) and torch.equal(dX[ends[-1]:], before[ends[-1]:])


def run(G, sizes, K, N, dtype, path=AUTO, seed=0, first=0, behind=0):
    x, W, d, off, ends = make(sizes, K, N, dtype, seed, first, behind)
    before = torch.randn((x.shape[0], N), device="cuda").to(dtype)
    out = G.detffn_grouped_forward(x, W, off, out=before.clone(), path=path)
    check_forward(G, x, W, off, ends, out, before)
    before = torch.randn((x.shape[0], K), device="cuda").to(dtype)
    dX, dW = G.detffn_grouped_backward(x, W, off, d, dX=before.clone(), path=path)
    check_backward(G, x, W, d, ends, dX, dW, before)
    return out, dX, dW


SIZES = [[1], [0, 1, 0], [16], [64, 64], [17, 0, 0, 255, 31], [300], [257, 1, 511, 128], [5] * 37, [0, 0, 1030]]
WIDTHS = [(64, 64), (128, 256), (8, 8), (264, 520), (1, 1), (65, 33), (1031, 130), (72, 300)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s[:5])))
def test_products(G, sizes, K, N, dtype):
    run(G, sizes, K, N, dtype, seed=K + N)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", SIZES[3:7], ids=lambda s: "-".join(map(str, s[:5])))
@pytest.mark.parametrize("K,N", [(264, 520), (65, 33), (131, 72)])
def test_cuda_core_path(G, sizes, K, N, dtype):
    run(G, sizes, K, N, dtype, path=EXACT, seed=3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K,N", [(1, 1), (65, 33), (131, 72), (136, 77), (1023, 515)])
def test_tensor_path_of_any_width(G, K, N, dtype):
    """Rows that lie on no 16-byte boundary are laid out in the workspace first."""
    run(G, [17, 0, 255, 300], K, N, dtype, path=TENSOR, seed=4, first=3, behind=5)


def test_workspace_of_the_caller(G):
    x, W, d, off, ends = make([30, 50], 65, 33, torch.bfloat16)
    n = G.detffn_grouped_workspace_size(80, 2, 65, 33)
    assert n > 0 and G.detffn_grouped_workspace_size(80, 2, 64, 32) == 0
    assert G.detffn_grouped_workspace_size(80, 2, 65, 33, torch.float32) == 0
    ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    out = G.detffn_grouped_forward(x, W, off, ws=ws)
    dX, dW = G.detffn_grouped_backward(x, W, off, d, ws=ws)
    check_forward(G, x, W, off, ends, out, out)
    check_backward(G, x, W, d, ends, dX, dW, dX)
    assert bool((ws[n:] == 0xFF).all())
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_grouped_forward(x, W, off, ws=ws[:n - 256])
    assert e.value.status == 5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("K,N", [(256, 136), (77, 100)])
def test_rows_of_no_expert_stay(G, K, N, dtype):
    run(G, [40, 0, 333], K, N, dtype, first=19, behind=70)


@pytest.mark.parametrize("dtype,K,N", [(torch.bfloat16, 2048, 768), (torch.float16, 1416, 4096), (torch.bfloat16, 4096, 1536)])
def test_larger(G, dtype, K, N):
    run(G, [700, 0, 1033, 12, 255], K, N, dtype, seed=5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K,N", [(256, 512), (100, 66)])
def test_row_strides(G, K, N, dtype):
    """Rows inside wider buffers, aligned and not."""
    sizes = [33, 0, 200]
    x, W, d, off, ends = make(sizes, K, N, dtype)
    for pad, at in ((64, 0), (64, 8), (3, 1)):
        wide = lambda t: torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        xs, ds, outs, dXs = wide(x), wide(d), wide(d), wide(x)
        cut = lambda t, n: t[:, at:at + n] if pad > at else t[:, :n]  # noqa: E731
        cut(xs, K).copy_(x)
        cut(ds, N).copy_(d)
        out = G.detffn_grouped_forward(cut(xs, K), W, off, out=cut(outs, N))
        dX, dW = G.detffn_grouped_backward(cut(xs, K), W, off, cut(ds, N), dX=cut(dXs, K))
        check_forward(G, x, W, off, ends, out, out)
        check_backward(G, x, W, d, ends, dX, dW, dX)
        for t, n in ((outs, N), (dXs, K)):
            rest = torch.cat((t[:, :at], t[:, at + n:]), 1) if pad > at else t[:, n:]
            assert bool(rest.isnan().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("sizes", [[37, 50, 13], [64, 3, 129], [1, 1, 1]])
def test_rows_that_are_not_finite_stay_their_own(G, dtype, bad, sizes):
    """An expert's rows, and rows of none, that hold an infinity or a NaN reach no other expert's results."""
    K, N = 136, 264
    x, W, d, off, ends = make(sizes, K, N, dtype, first=7, behind=90)
    own = slice(ends[1], ends[2])
    keep = [t.clone() for t in (x, d)]
    for t in (x, d):
        t[:ends[0]] = bad
        t[own] = bad
        t[ends[-1]:] = bad
    out = G.detffn_grouped_forward(x, W, off)
    dX, dW = G.detffn_grouped_backward(x, W, off, d)
    x, d = keep
    for e in (0, 2):
        a, b = ends[e], ends[e + 1]
        x64, w64, d64 = x[a:b].double(), W[e].double(), d[a:b].double()
        close(out[a:b], x64 @ w64.T, x64.abs() @ w64.abs().T, K, dtype)
        close(dX[a:b], d64 @ w64, d64.abs() @ w64.abs(), N, dtype)
        close(dW[e], d64.T @ x64, d64.abs().T @ x64.abs(), b - a, dtype)
    assert not bool(out[own].isfinite().any()) and not bool(dW[1].isfinite().any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ends_out_of_order_or_range(G, dtype):
    """Ends beyond R are R, an end before its beginning gives no rows; nothing else is touched."""
    K, N, R = 128, 64, 100
    x, W, d, _, _ = make([R], K, N, dtype)
    W = torch.randn((3, N, K), device="cuda").to(dtype)
    off = torch.tensor([10, 50, 40, 1000], dtype=torch.int32, device="cuda")
    before = torch.randn((R, N), device="cuda").to(dtype)
    out = G.detffn_grouped_forward(x, W, off, out=before.clone())
    assert torch.equal(out[:10], before[:10])
    x64 = x.double()
    for e, a, b in ((0, 10, 40), (2, 50, 100)):
        w64 = W[e].double()
        close(out[a:b], x64[a:b] @ w64.T, x64[a:b].abs() @ w64.abs().T, K, dtype)
    off = torch.tensor([-5, -1, 0, 0], dtype=torch.int32, device="cuda")
    assert torch.equal(G.detffn_grouped_forward(x, W, off, out=before.clone()), before)
    dX, dW = G.detffn_grouped_backward(x, W, off, d, dX=x.clone())
    assert torch.equal(dX, x) and not bool(dW.any())


def test_gradient_by_differences(G):
    """dX and dW against central differences of the forward in FP32: the sum of
    out * dOut is linear in each input, so a step of 1 has no truncation error
    and leaves the rounding of two sums of 50 * 24 products."""
    x, W, d, off, _ = make([20, 0, 30], 16, 24, torch.float32)
    dX, dW = G.detffn_grouped_backward(x, W, off, d)
    g = torch.Generator(device="cuda").manual_seed(9)
    f = lambda x, W: float((G.detffn_grouped_forward(x, W, off).double() * d.double()).sum())  # noqa: E731
    for t, grad, at in ((x, dX, 0), (W, dW, 1)):
        v = torch.randn(t.shape, generator=g, device="cuda")
        hi, lo = (f(*((t + s * v) if i == at else (x, W)[i] for i in range(2))) for s in (1.0, -1.0))
        want = (hi - lo) / 2
        size = float((d.abs().double() * 16 * 10).sum())   # |x W| summed, entries below 10
        assert abs(float((grad.double() * v.double()).sum()) - want) <= 32 * 2.0 ** -23 * size


@pytest.mark.parametrize("dtype,K,N", [(torch.bfloat16, 256, 384), (torch.float32, 100, 60)])
def test_parts_streams_graphs_and_repeats(G, dtype, K, N):
    x, W, d, off, _ = make([100, 3, 0, 61], K, N, dtype)
    out = G.detffn_grouped_forward(x, W, off)
    dX, dW = G.detffn_grouped_backward(x, W, off, d)
    assert torch.equal(out, G.detffn_grouped_forward(x, W, off))
    a, none = G.detffn_grouped_backward(None, W, off, d, need_dW=False)
    assert none is None and torch.equal(a, dX)
    none, b = G.detffn_grouped_backward(x, W, off, d, need_dX=False)
    assert none is None and torch.equal(b, dW)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2 = G.detffn_grouped_forward(x, W, off, stream=side)
    x2, w2 = G.detffn_grouped_backward(x, W, off, d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, o2) and torch.equal(dX, x2) and torch.equal(dW, w2)
    graph = torch.cuda.CUDAGraph()
    buf = torch.zeros_like(out)
    with torch.cuda.graph(graph):
        G.detffn_grouped_forward(x, W, off, out=buf)
        gx, gw = G.detffn_grouped_backward(x, W, off, d)
    # A replay reads the offsets as they are then.
    for ends in ([0, 100, 103, 103, 164], [0, 1, 64, 100, 164]):
        off.copy_(torch.tensor(ends, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, G.detffn_grouped_forward(x, W, off))
        ex, ew = G.detffn_grouped_backward(x, W, off, d)
        assert torch.equal(gx, ex) and torch.equal(gw, ew)


def test_no_rows(G):
    x, W, d, off, _ = make([0, 0], 64, 32, torch.bfloat16)
    assert G.detffn_grouped_forward(x, W, off).shape == (0, 32)
    dX, dW = G.detffn_grouped_backward(x, W, off, d)
    assert dX.shape == (0, 64) and dW.shape == (2, 32, 64) and not bool(dW.any())


def test_refusals(G):
    x, W, d, off, _ = make([8, 8], 64, 32, torch.bfloat16)
    for bad in ((x.float(), W, off), (x[:, :63], W, off), (x, W[0], off), (x, W, off[:2]), (x, W, off.long()),
                (x.cpu(), W, off), (x, W.transpose(1, 2), off), (x.t(), W, off)):
        with pytest.raises(ValueError):
            G.detffn_grouped_forward(*bad)
    with pytest.raises(ValueError):
        G.detffn_grouped_forward(x, W, off, out=torch.empty((15, 32), dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError):
        G.detffn_grouped_backward(x, W, off, d[:8])
    with pytest.raises(ValueError):
        G.detffn_grouped_backward(None, W, off, d)
    with pytest.raises(ValueError):
        G.detffn_grouped_backward(x, W, off, d, need_dX=False, need_dW=False)
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_grouped_forward(x, torch.randn((2, 64, 64), device="cuda").bfloat16(), off, out=x)
    assert e.value.status == 1
    with pytest.raises(G.DetFFNError) as e:
        G.detffn_grouped_forward(x.float(), W.float(), off, path=TENSOR)
    assert e.value.status == 4


@pytest.mark.parametrize("what", ["forward", "dX", "dW"])
def test_a_wait_that_runs_out_is_reported(G, what):
    """No copies are issued: the first wait ends at its limit, the status says so,
    calls until it is read leave their outputs unwritten, and later ones are whole."""
    x, W, d, off, _ = make([100, 60], 256, 264, torch.bfloat16)
    out = torch.zeros((160, 264), dtype=x.dtype, device="cuda")
    kw = dict(path=TENSOR, spin_limit=2000, flags=G.FLAG_TEST_STALL)
    if what == "forward":
        G.detffn_grouped_forward(x, W, off, out=out, **kw)
    else:
        G.detffn_grouped_backward(x, W, off, d, need_dX=what == "dX", need_dW=what == "dW", **kw)
    torch.cuda.synchronize()
    G.detffn_grouped_forward(x, W, off, out=out, path=TENSOR)
    assert not bool(out.any())
    assert G.detffn_get_status() == 7 and G.detffn_get_status() == 0
    got = G.detffn_grouped_forward(x, W, off, out=out, path=TENSOR)
    want = torch.cat([x[:100].double() @ W[0].double().T, x[100:].double() @ W[1].double().T])
    assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8


@pytest.mark.parametrize("dtype,K,N", [(torch.bfloat16, 64, 40), (torch.float32, 33, 20)])
def test_as_many_experts_as_there_may_be(G, dtype, K, N):
    g = torch.Generator().manual_seed(1)
    run(G, torch.randint(0, 4, (1024,), generator=g).tolist(), K, N, dtype, seed=6)


@pytest.mark.parametrize("dtype,E", [(torch.bfloat16, 65), (torch.float32, 33)])
def test_addresses_beyond_32_bits(G, dtype, E):
    """W and dW of more than 2^32 (FP32: 2^31) elements: the first and the last expert's results."""
    K = N = 8192
    sizes = [70] + [0] * (E - 2) + [130]
    W = torch.zeros((E, N, K), dtype=dtype, device="cuda")
    ends = [0] + [70] * (E - 1) + [200]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    for e in (0, E - 1):
        W[e] = r(N, K)
    x, d = r(200, K), r(200, N)
    out = G.detffn_grouped_forward(x, W, off)
    dX, dW = G.detffn_grouped_backward(x, W, off, d)
    for e in (0, E - 1):
        a, b = ends[e], ends[e + 1]
        assert b - a == sizes[e]
        x64, w64, d64 = x[a:b].double(), W[e].double(), d[a:b].double()
        close(out[a:b], x64 @ w64.T, x64.abs() @ w64.abs().T, K, dtype)
        close(dX[a:b], d64 @ w64, d64.abs() @ w64.abs(), N, dtype)
        close(dW[e], d64.T @ x64, d64.abs().T @ x64.abs(), b - a, dtype)
    assert not bool(dW[1].any()) and not bool(dW[E - 2].any())


def test_two_streams_at_once(G):
    """Calls that overlap on the GPU, tensor cores and CUDA cores, share nothing."""
    jobs = []
    for i, (dtype, K, N) in enumerate(((torch.bfloat16, 512, 1024), (torch.float16, 1031, 260), (torch.float32, 300, 200))):
        x, W, d, off, _ = make([300, 0, 77, 1200], K, N, dtype, seed=i)
        jobs.append((x, W, d, off, G.detffn_grouped_forward(x, W, off), *G.detffn_grouped_backward(x, W, off, d)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for n in range(12):
        x, W, d, off = jobs[n % 3][:4]
        s = streams[n % 2]
        got.append((n % 3, G.detffn_grouped_forward(x, W, off, stream=s), *G.detffn_grouped_backward(x, W, off, d, stream=s)))
    torch.cuda.synchronize()
    for j, out, dX, dW in got:
        assert torch.equal(out, jobs[j][4]) and torch.equal(dX, jobs[j][5]) and torch.equal(dW, jobs[j][6])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_row_does_not_depend_on_the_others(G, dtype):
    """On the tensor cores a row has the same bits in a batch of any size, with any number of experts."""
    x, W, d, off, ends = make([3, 700, 0, 41, 256], 1032, 520, dtype)
    out = G.detffn_grouped_forward(x, W, off)
    dX, _ = G.detffn_grouped_backward(x, W, off, d, need_dW=False)
    for e, a, b in ((0, 1, 2), (1, 100, 133), (4, 744, 1000), (3, 703, 744)):
        o = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        assert torch.equal(G.detffn_grouped_forward(x[a:b], W[e:e + 1], o), out[a:b])
        assert torch.equal(G.detffn_grouped_backward(None, W[e:e + 1], o, d[a:b], need_dW=False)[0], dX[a:b])


FEW = [[1], [2], [3], [8], [9], [1] * 40, [0, 7, 0, 16, 2, 8, 1], [0] * 33 + [5, 0, 11], [40, 0, 0, 0]]


@pytest.mark.parametrize("K,N", [(1, 1), (4, 3), (124, 6), (128, 5), (132, 64), (131, 33), (1031, 130), (2056, 83), (1160, 1028)])
@pytest.mark.parametrize("sizes", FEW, ids=lambda s: "-".join(map(str, s[:5])))
def test_few_rows_in_32_bits(G, sizes, K, N):
    """Up to eight rows of an expert at a time; an expert's row of each length, whole and cut runs of K."""
    out, dX, _ = run(G, sizes, K, N, torch.float32, seed=K + 7 * N, first=2, behind=3)
    again, dX2, _ = run(G, sizes, K, N, torch.float32, seed=K + 7 * N, first=2, behind=3)
    a, b = 2, 2 + sum(sizes)
    assert torch.equal(out[a:b], again[a:b]) and torch.equal(dX[a:b], dX2[a:b])


@pytest.mark.parametrize("per", [15, 16, 17, 64, 65])
@pytest.mark.parametrize("N", [512, 2048])
def test_where_few_rows_end(G, per, N):
    run(G, [per, 0, 2 * per, per], 264, N, torch.float32, seed=per)


@pytest.mark.parametrize("K,N,ld,shift", [(132, 64, 136, 0), (132, 64, 133, 0), (132, 64, 132, 1), (130, 66, 140, 2)])
def test_few_rows_where_they_lie(G, K, N, ld, shift):
    """Rows on and off 16-byte boundaries, and others' values that are not finite beside them."""
    x, W, d, off, ends = make([3, 0, 9, 1], K, N, torch.float32, seed=5)
    R = x.shape[0]
    bad = torch.full((R * ld + shift + 8,), float("nan"), device="cuda")
    xs = bad[shift:shift + R * ld].view(R, ld)[:, :K]
    xs.copy_(x)
    ldd = N + ld - K
    other = torch.full((R * ldd + shift + 8,), float("nan"), device="cuda")
    ds = other[shift:shift + R * ldd].view(R, ldd)[:, :N]
    ds.copy_(d)
    out = torch.full((R, N + 3), 7.0, device="cuda")
    G.detffn_grouped_forward(xs, W, off, out=out[:, :N])
    check_forward(G, x, W, off, ends, out[:, :N], out[:, :N])
    assert bool((out[:, N:] == 7.0).all())
    dX = torch.full((R, K + 5), 7.0, device="cuda")
    _, dW = G.detffn_grouped_backward(xs, W, off, ds, dX=dX[:, :K])
    check_backward(G, x, W, d, ends, dX[:, :K], dW, dX[:, :K])
    assert bool((dX[:, K:] == 7.0).all())


def test_few_rows_keep_what_is_not_finite_to_themselves(G):
    x, W, d, off, ends = make([1, 4, 0, 11], 200, 60, torch.float32, seed=6)
    clean = G.detffn_grouped_forward(x, W, off)
    gone = G.detffn_grouped_backward(x, W, off, d, need_dW=False)[0]
    y, e = x.clone(), d.clone()
    y[2, 5], y[7, 199], e[2, 5], e[7, 59] = float("nan"), float("inf"), float("nan"), float("inf")
    out, dX = G.detffn_grouped_forward(y, W, off), G.detffn_grouped_backward(y, W, off, e, need_dW=False)[0]
    rows = [i for i in range(16) if i not in (2, 7)]
    assert torch.equal(out[rows], clean[rows]) and torch.equal(dX[rows], gone[rows])
    assert not bool(out[[2, 7]].isfinite().any()) and not bool(dX[[2, 7]].isfinite().any())


@pytest.mark.parametrize("sizes,K,N", [
    ([300], 1100, 512), ([300], 512, 1100), ([300], 1025, 513), ([100, 0, 250, 3], 1056, 400), ([64, 63, 65], 1024, 1024),
    ([300], 200, 512), ([300], 65, 512), ([300], 96, 515), ([2000], 128, 128), ([3500, 5, 0], 64, 72), ([900, 1, 33], 130, 66)],
    ids=str)
def test_a_contraction_in_parts(G, sizes, K, N):
    """FP32 with few tiles: parts of whole rounds, a last part that is short or has nothing, experts of few or no rows."""
    a = run(G, sizes, K, N, torch.float32, seed=K + N)
    b = run(G, sizes, K, N, torch.float32, seed=K + N)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    x, W, d, off, ends = make(sizes, K, N, torch.float32, seed=9, first=1, behind=70)
    before = torch.randn((x.shape[0], N), device="cuda")
    check_forward(G, x, W, off, ends, G.detffn_grouped_forward(x, W, off, out=before.clone()), before)
