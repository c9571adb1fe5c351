"""4-bit products whose every product counts: x of whole numbers up to 3, scales of
1/2, 1 and 2, so that all sums are whole numbers of halves, below 2^24 of them (24
times 2 halves times 2, by K up to 100003, is 9.6 million), and exact in FP32 in
any order: a result has to be the 64-bit one rounded once."""
import pytest
import torch

from tests.test_gpu_w4 import ALL, G, codes_of, values64  # noqa: F401

pytestmark = pytest.mark.gpu


def whole(G, N, K, group, dtype, codes, seed=0):
    """A matrix with codes of the given ends (all sixteen: 0 to 15)."""
    g = torch.Generator(device="cuda").manual_seed(seed + N + K)
    c = [torch.randint(codes[0], codes[1] + 1, (N, (K + 127) // 128 * 64), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    s = torch.randint(-1, 2, (N, (K + group - 1) // group), generator=g, device="cuda").double().exp2()
    return G.W4(c[0] | c[1] << 4, s.to(dtype), K, group)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(24, 100003), (131, 12288), (40, 4096), (33, 1025), (48, 8320), (20, 129)])
def test_sums_of_whole_numbers(G, N, K, group, dtype):
    w = whole(G, N, K, group, dtype, (0, 15))
    v = values64(w)
    for T in (1, 3, 8, 9, 17, 33, 64):
        x = torch.randint(-3, 4, (T, K), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").to(dtype)
        assert torch.equal(G.detffn_w4_matvec(x, w), (x.double() @ v.T).to(dtype)), T


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("H,I,group", [(512, 12288, 128), (500, 3001, 64), (129, 1030, 32)])
def test_ffn_of_whole_numbers(G, H, I, group, dtype):
    """Gates of 20 and more, whose SiLU is the gate in FP32, and a hidden activation
    of whole numbers below 2^16, which 16 bits hold."""
    Wg, Wu, Wd = whole(G, I, H, group, dtype, (9, 10)), whole(G, I, H, group, dtype, (7, 9), 1), whole(G, H, I, group, dtype, (7, 9), 2)
    Wg, Wu, Wd = (w._replace(scales=torch.full_like(w.scales, s)) for w, s in ((Wg, 1), (Wu, 1), (Wd, 1 / 16)))   # (FP16's range)
    g64, u64, d64 = values64(Wg), values64(Wu), values64(Wd)
    for T in (1, 5, 8, 9, 17, 33, 64):
        x = (torch.rand((T, H), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda") < 64 / H).float()
        x[:, :20] = 1.0
        g, u = x.double() @ g64.T, x.double() @ u64.T
        h = g * u
        want = h @ d64.T
        assert float(g.min()) >= 20 and float(h.abs().max()) < 2 ** 16 and float((h.abs() @ d64.abs().T).max()) < 2 ** 20   # (of sixteenths)
        if dtype == torch.float16:
            assert float(want.abs().max()) < 65504
        assert torch.equal(G.detffn_w4_forward(x.to(dtype), Wg, Wu, Wd), want.to(dtype)), T
