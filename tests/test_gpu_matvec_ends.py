"""GPU tests of the 4-bit matrix-vector product at the ends of its scales' and its
tokens' ranges, on both kernels: sizes with K no multiple of 128, or small ones, go to
mma.sync, K = 8192 and above to the block-scaled tensor cores.  Bounds as in
test_gpu_matvec.py."""
import math

import pytest
import torch

from test_gpu_matvec import BF16, check, decode, generator, random_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe(moelib):
    import moe_expert_layer_08_b200 as m
    return m


@pytest.mark.parametrize("K", [32, 8192])
def test_a_result_near_the_end_of_the_range(moe, K):
    """One weight of 1.0 with the scale 2^115 times one: 2^115, up to 2^127."""
    x = torch.zeros((1, K), dtype=BF16, device="cuda")
    x[0, 5] = 1
    w = torch.zeros((16, K // 2), dtype=torch.uint8, device="cuda")
    w[:, 2] = 2 << 4               # element 5 is 1.0
    sf = torch.full((16, K // 32), 127, dtype=torch.uint8, device="cuda")
    for byte in range(240, 255):
        sf[:, 0] = byte
        want = torch.full((1, 16), 2.0 ** (byte - 127), dtype=BF16, device="cuda")
        assert torch.equal(moe.fp4_matvec(x, w, sf), want), byte


@pytest.mark.parametrize("T,N,K", [(8, 40, 1056), (3, 33, 96), (1, 130, 8192), (8, 130, 8192)])
@pytest.mark.parametrize("byte", [0, 1, 20, 200, 240, 243, 247, 251, 254])
def test_scales_near_their_ends(moe, T, N, K, byte):
    """A matrix whose scales are all near one end, and tokens from the size that
    keeps every sum of magnitudes below 2^126 (at most 2^120) down by 2^15 a token:
    no sum passes fp32's range."""
    x, w, sf = random_case(T, N, K, "mx", 81)
    g = generator(82)
    sf[:] = (byte + torch.randint(-3, 4, sf.shape, device="cuda", generator=g)).clamp(0, min(byte + 2, 254)).to(torch.uint8)
    # |x| <= 8 before scaling (normal), |code| <= 6: a sum is below K * 48 * 2^(byte + 2 - 127) * 2^p
    p = min(126 - (min(byte + 2, 254) - 127) - math.ceil(math.log2(K * 48)), 117)
    assert float(x.abs().max()) <= 8
    x *= torch.exp2(p - 15.0 * torch.arange(T, device="cuda", dtype=torch.float64)).to(BF16)[:, None]
    check(moe, x, w, sf, "mx")


@pytest.mark.parametrize("T,N,K", [(8, 40, 1056), (5, 70, 256), (2, 130, 8192), (4, 130, 8320)])
def test_nvfp4_tokens_of_every_size(moe, T, N, K):
    """Tokens from 2^-130 to the largest whose sums stay below 2^126."""
    x, w, sf = random_case(T, N, K, "nvfp4", 83)
    top = 126 - 9 - math.ceil(math.log2(K * 48))
    assert float(x.abs().max()) <= 8
    e = torch.linspace(-130, top, T, device="cuda", dtype=torch.float64).round()
    x = (x.double() * torch.exp2(e)[:, None]).to(BF16)
    check(moe, x, w, sf, "nvfp4")


@pytest.mark.parametrize("N,K", [(40, 96), (9001, 96), (40, 8192)])
def test_a_small_token_that_is_not_finite_beside_large_scales(moe, N, K):
    x, w, sf = random_case(3, N, K, "mx", 84)
    x *= 2.0 ** -40
    sf[:] = 250
    w |= 0x22                      # no zero weights
    x[0, 3], x[1, 7], x[1, 8] = float("inf"), float("nan"), float("inf")
    y = moe.fp4_matvec(x, w, sf)
    exact = x.double() @ decode(w, sf, "mx").T
    assert torch.equal(y[0].double(), exact[0]) and bool(torch.isinf(y[0]).all())
    assert bool(torch.isnan(y[1]).all())
    assert bool(torch.isfinite(y[2]).all())
    check(moe, x[2:].contiguous(), w, sf, "mx")


def wide_tokens(T, K, seed):
    """Tokens of every kind, T of them: elements over 60 powers of two, zeros, a
    small one, a large one, one large element, every other zero, the smallest bf16
    numbers, one element of 2^100."""
    g = generator(seed)
    x = torch.randn((8, K), dtype=BF16, device="cuda", generator=g)
    x[0] *= torch.exp2(torch.randint(-40, 20, (K,), device="cuda", generator=g).to(BF16))
    x[1] = 0
    x[2] *= 2.0 ** -110
    x[3] *= 2.0 ** 60
    x[4, 5] = 3e30
    x[5, ::2] = 0
    x[6] = 2.0 ** -133 * torch.randint(-9, 10, (K,), device="cuda", generator=g).to(BF16)
    x[7, K // 2] = 2.0 ** 100
    return x[:T] if seed % 2 else x[8 - T:].contiguous()


@pytest.mark.parametrize("fmt,T,K", [("mx", 8, 8192), ("mx", 8, 8320), ("mx", 3, 8320), ("nvfp4", 4, 8320), ("nvfp4", 2, 8192),
                                     ("nvfp4", 1, 8320), ("nvfp4", 8, 8320)])
@pytest.mark.parametrize("seed", [91, 92])
def test_wide_tokens_times_long_rows(moe, fmt, T, K, seed):
    """test_tokens_of_a_wide_range at the tensor cores' sizes."""
    w, sf = random_case(1, 200, K, fmt, seed)[1:]
    check(moe, wide_tokens(T, K, seed), w, sf, fmt)


@pytest.mark.parametrize("fmt,T,n", [("mx", 8, 1056), ("mx", 8, 8192), ("mx", 1, 8192), ("nvfp4", 4, 8192), ("nvfp4", 2, 8192),
                                     ("nvfp4", 8, 1056)])
@pytest.mark.parametrize("seed", [93, 94])
def test_every_element_by_itself(moe, fmt, T, n, seed):
    """The unit matrix gives the tokens back: an element exactly down to 2^-31 of
    its token's largest one, below that within 2^-40 of it (and one rounding)."""
    w = torch.zeros((n, n // 2), dtype=torch.uint8, device="cuda")
    row = torch.arange(n, device="cuda")
    w[row, row // 2] = torch.where(row % 2 == 1, 2 << 4, 2).to(torch.uint8)     # 1.0
    one, group = (127, 32) if fmt == "mx" else (0x38, 16)
    sf = torch.full((n, n // group), one, dtype=torch.uint8, device="cuda")
    x = wide_tokens(T, n, seed)
    x[0, 77] = 2.0 ** 127
    y = moe.fp4_matvec(x, w, sf, fmt=fmt)
    largest = x.double().abs().amax(1, keepdim=True)
    high = x.double().abs() >= 2.0 ** -31 * largest
    assert torch.equal(y[high], x[high])
    off = 2.0 ** -40 * largest
    assert bool(((y.double() - x.double()).abs() <= off + 2.0 ** -8 * (x.double().abs() + off))[~high].all())


def test_mx_scales_at_their_ends_of_long_rows(moe):
    x, w, sf = random_case(8, 40, 8320, "mx", 95)
    x *= 2.0 ** 20
    sf[0], sf[1], sf[2] = 0, 200, 1
    for T in (1, 5, 8):
        check(moe, x[:T].contiguous(), w, sf, "mx")
    sf[7, 259], sf[30, 0] = 255, 255   # NaN
    fine = [n for n in range(40) if n not in (7, 30)]
    for T in (1, 8):
        y = moe.fp4_matvec(x[:T].contiguous(), w, sf)
        assert bool(torch.isnan(y[:, [7, 30]]).all()) and bool(torch.isfinite(y[:, fine]).all())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("fmt,T,K", [("mx", 8, 8192), ("mx", 5, 8320), ("nvfp4", 4, 8320), ("nvfp4", 2, 8192)])
def test_a_token_does_not_reach_another_in_long_rows(moe, bad, fmt, T, K):
    x, w, sf = random_case(T, 300, K, fmt, 96)
    w |= 0x22                      # no zero weights
    if fmt == "nvfp4":
        sf.clamp_(1, 126)          # and no zero or NaN scales
    clean = moe.fp4_matvec(x, w, sf, fmt=fmt)
    x[1, 100] = bad
    y = moe.fp4_matvec(x, w, sf, fmt=fmt)
    others = [t for t in range(T) if t != 1]
    assert torch.equal(y[others], clean[others]) and not bool(torch.isfinite(y[1]).any())
    assert bool(torch.isnan(y[1]).all() if bad != bad else torch.isinf(y[1]).all())


@pytest.mark.parametrize("fmt,K", [("mx", 96), ("mx", 8192), ("nvfp4", 96), ("nvfp4", 8192)])
def test_an_infinity_beside_the_largest_elements(moe, fmt, K):
    """Finite products, however large before their scale, leave an infinite result
    as it is."""
    x = torch.zeros((1, K), dtype=BF16, device="cuda")
    x[0, 0], x[0, 5], x[0, 40] = float("inf"), 1.5 * 2.0 ** 127, -1.5 * 2.0 ** 127
    w = torch.full((8, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    w[:4, 2] = 0xF2                # element 5 is -6
    w[2:6, 20] = 0x27              # element 40 is 6
    small = 100 if fmt == "mx" else 1
    sf = torch.full((8, K // (32 if fmt == "mx" else 16)), small, dtype=torch.uint8, device="cuda")
    w[1, 0] = w[3, 0] = 0x2A       # element 0 is -1
    y = moe.fp4_matvec(x, w, sf, fmt=fmt)
    exact = x.double() @ decode(w, sf, fmt).T
    assert bool(torch.isinf(exact).all()) and torch.equal(y.double(), exact)
