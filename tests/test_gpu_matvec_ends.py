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


@pytest.mark.parametrize("K", [96, 8192])
def test_a_small_token_that_is_not_finite_beside_large_scales(moe, K):
    x, w, sf = random_case(3, 40, K, "mx", 84)
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
