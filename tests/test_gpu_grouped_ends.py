"""The products grouped by expert at the ends of what they accept: waits that run
out at any point, as many rows as there may be, and sums whose every product
counts.

Sums of whole numbers are exact in FP32 in any order where the magnitudes of all
products add up to less than 2^24, so a result has to be the 64-bit one rounded
once: a product that is left out or taken twice shows at any length."""
import pytest
import torch

from tests.test_gpu_grouped import AUTO, EXACT, G, TENSOR, check_backward, check_forward, make, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["forward", "dX", "dW"])
@pytest.mark.parametrize("sizes,K,N", [([100, 60], 256, 264), ([1, 0, 700], 1032, 520)], ids=str)
def test_waits_of_few_tries(G, sizes, K, N, what):
    """With limits that ordinary waits may well reach, at any point of a call, every call ends; the
    status says whether one ran out, and calls that did not are whole."""
    x, W, d, off, _ = make(sizes, K, N, torch.bfloat16)

    def go(**kw):
        if what == "forward":
            return G.detffn_grouped_forward(x, W, off, path=TENSOR, **kw)
        return next(t for t in G.detffn_grouped_backward(x, W, off, d, need_dX=what == "dX", need_dW=what == "dW", path=TENSOR,
                                                         **kw) if t is not None)
    want = go()
    for limit in (1, 1, 2, 3, 5, 8, 16, 64):
        got = go(spin_limit=limit)
        torch.cuda.synchronize()
        status = G.detffn_get_status()
        assert status in (0, 7)
        assert status == 7 or torch.equal(got, want)
        assert torch.equal(go(), want)
    assert G.detffn_get_status() == 0


@pytest.mark.parametrize("ends", [lambda R: [0, R], lambda R: [3, R - 5000, R]], ids=["one", "two"])
def test_as_many_rows_as_there_may_be(G, ends):
    """2^31 - 256 rows, 34 GB of x: rows at both ends of it, and their sums, in whole numbers."""
    R, K, N = (1 << 31) - 256, 8, 8
    ends = ends(R)
    E = len(ends) - 1
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").bfloat16()  # noqa: E731
    W = r(E, N, K)
    x, d = (torch.zeros((R, K), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    places = [slice(ends[0], 700), slice(R // 2, R // 2 + 513), slice(R - 6000, R)]
    for s in places:
        x[s], d[s] = r(s.stop - s.start, K), r(s.stop - s.start, N)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    G.detffn_grouped_forward(x, W, off, out=out)
    assert bool((out[:ends[0]] == 7.0).all())
    for s in places:
        row = torch.arange(s.start, s.stop, device="cuda")
        of = torch.bucketize(row, off.long()[1:-1], right=True) if E > 1 else torch.zeros_like(row)
        assert torch.equal(out[s], torch.einsum("rk,rnk->rn", x[s].double(), W[of].double()).bfloat16())
    assert not bool(out[1000:R // 2].any())
    del out
    torch.cuda.empty_cache()
    _, dW = G.detffn_grouped_backward(x, W, off, d, need_dX=False)
    want = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
    for s in places:
        for e in range(E):
            a, b = max(s.start, ends[e]), min(s.stop, ends[e + 1])
            if a < b:
                want[e] += d[a:b].double().T @ x[a:b].double()
    assert torch.equal(dW, want.bfloat16())
    assert G.detffn_get_status() == 0


@pytest.mark.parametrize("dtype,path", [(torch.bfloat16, AUTO), (torch.float16, AUTO), (torch.float32, AUTO), (torch.bfloat16, EXACT)],
                         ids=["bf16", "f16", "f32", "bf16-exact"])
@pytest.mark.parametrize("sizes,K,N", [
    ([700, 0, 1033, 12, 255], 4096, 1536), ([64, 1, 100], 8192, 520), ([3, 17, 0, 1], 8189, 77), ([5] * 30, 2056, 1028),
    ([9000, 8191], 64, 72), ([40000], 40, 9), ([300], 1100, 2048), ([20], 9, 65536), ([20], 65536, 9)], ids=str)
def test_sums_of_whole_numbers(G, sizes, K, N, dtype, path):
    """9 times the longest sum, 65536 products, stays below 2^24."""
    x, W, d, off, ends = make(sizes, K, N, torch.float32, seed=K + N)
    x, W, d = (t.round().clamp(-3, 3).to(dtype) for t in (x, W, d))
    out = G.detffn_grouped_forward(x, W, off, path=path)
    dX, dW = G.detffn_grouped_backward(x, W, off, d, path=path)
    for e in range(len(sizes)):
        a, b = ends[e], ends[e + 1]
        x64, w64, d64 = x[a:b].double(), W[e].double(), d[a:b].double()
        assert torch.equal(out[a:b], (x64 @ w64.T).to(dtype))
        assert torch.equal(dX[a:b], (d64 @ w64).to(dtype))
        assert torch.equal(dW[e], (d64.T @ x64).to(dtype))


@pytest.mark.parametrize("what", ["forward", "dX"])
@pytest.mark.parametrize("sizes", [[2, 0, 0, 1, 0], [0] * 70 + [9] + [0] * 40, [0, 0, 1], [0] * 31 + [5, 2] + [0] * 3], ids=lambda s: str(len(s)))
def test_matrices_of_no_row_are_not_laid_out(G, sizes, what):
    """Odd widths and fewer rows than experts: the scratch of those without rows stays as it was."""
    K, N, mark = 65, 33, -23131
    x, W, d, off, ends = make(sizes, K, N, torch.bfloat16)
    R, E = x.shape[0], len(sizes)
    W[[e for e in range(E) if not sizes[e]]] = float("nan")
    ws = torch.full((G.detffn_grouped_workspace_size(R, E, K, N) // 2,), mark, dtype=torch.int16, device="cuda")
    buf = ws.view(torch.uint8)
    if what == "forward":
        got, want = G.detffn_grouped_forward(x, W, off, ws=buf), torch.cat([x[ends[e]:ends[e + 1]].double() @ W[e].double().T for e in range(E)])
    else:
        got, _ = G.detffn_grouped_backward(None, W, off, d, need_dW=False, ws=buf)
        want = torch.cat([d[ends[e]:ends[e + 1]].double() @ W[e].double() for e in range(E)])
    assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8
    assert int((ws == mark).sum()) >= sizes.count(0) * N * 72


def test_matrices_where_ends_are_out_of_order(G):
    """More experts that have rows than there are rows: the last of them, which no other's rows meet, is laid out too."""
    K, N = 65, 33
    x, W, d, _, _ = make([4], K, N, torch.bfloat16)
    W = torch.randn((40, N, K), device="cuda").bfloat16()
    off = torch.tensor([0, 1] * 18 + [0, 0, 1, 2, 4], dtype=torch.int32, device="cuda")   # expert 38 has row 1, 39 rows 2 and 3
    ws = torch.full((G.detffn_grouped_workspace_size(4, 40, K, N),), 0xFF, dtype=torch.uint8, device="cuda")
    out = G.detffn_grouped_forward(x, W, off, ws=ws)
    want = torch.cat([x[1:2].double() @ W[38].double().T, x[2:].double() @ W[39].double().T])
    assert float((out[1:].double() - want).norm() / want.norm()) < 2.0 ** -8
    dX, _ = G.detffn_grouped_backward(None, W, off, d, need_dW=False, ws=ws.fill_(0xFF))
    want = torch.cat([d[1:2].double() @ W[38].double(), d[2:].double() @ W[39].double()])
    assert float((dX[1:].double() - want).norm() / want.norm()) < 2.0 ** -8


@pytest.mark.parametrize("per", [23, 24, 25, 31, 32, 33])
@pytest.mark.parametrize("K,N", [(264, 1040), (1031, 130), (96, 4096)])
def test_where_rows_by_eights_end(G, per, K, N):
    """On both sides of the sizes where FP32 changes kernels, alike and uneven experts."""
    for sizes in ([per] * 9, [3 * per, 0, 0], [per - 3, per + 3, per], [64 * per]):
        run(G, sizes, K, N, torch.float32, seed=per)


@pytest.mark.parametrize("K,N,operand", [(64, 33, "x"), (33, 64, "dOut"), (64, 64, "x"), (64, 64, "dOut")])
def test_rows_off_16_byte_boundaries(G, K, N, operand):
    """An operand whose width is a multiple of 8: refused by the tensor path where a product reads it, right by default."""
    x, W, d, off, ends = make([20, 0, 130], K, N, torch.bfloat16, first=1, behind=2)
    place = lambda t: torch.cat((t[:, :1], t), 1)[:, 1:]  # noqa: E731
    x, d = (place(x), d) if operand == "x" else (x, place(d))
    before = torch.randn((x.shape[0], N), device="cuda").bfloat16()
    check_forward(G, x, W, off, ends, G.detffn_grouped_forward(x, W, off, out=before.clone()), before)
    before = torch.randn((x.shape[0], K), device="cuda").bfloat16()
    dX, dW = G.detffn_grouped_backward(x, W, off, d, dX=before.clone())
    check_backward(G, x, W, d, ends, dX, dW, before)
    for read, call in ((operand == "x", lambda: G.detffn_grouped_forward(x, W, off, path=TENSOR)),
                       (operand == "dOut", lambda: G.detffn_grouped_backward(x, W, off, d, need_dW=False, path=TENSOR)),
                       (True, lambda: G.detffn_grouped_backward(x, W, off, d, need_dX=False, path=TENSOR)),
                       (True, lambda: G.detffn_grouped_backward(x, W, off, d, path=TENSOR))):
        if read:
            with pytest.raises(G.DetFFNError) as e:
                call()
            assert e.value.status == 4
        else:
            call()
