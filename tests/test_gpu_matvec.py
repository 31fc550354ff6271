"""GPU tests of the 4-bit matrix-vector product against the definition in 64
bits, with the weights decoded here from the formats' bit fields.

Tolerance, element by element: one rounding to bf16 (2^-8 relative) of an fp32
sum of K products, whose additions (in groups, over the groups, over the eight
slices) number at most K + 16 and are off by at most 2^-23 of a partial sum <=
S = sum |x w| each; a group's factor adds at most one rounding per addition
already counted.  An element of x enters as fp16 scaled by its slice's largest
magnitude: off by at most 2^-40 of that, so by 2^-40 max|x| sum |w| in all."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64
ROUND = torch.finfo(BF16).eps / 2


@pytest.fixture(scope="module")
def moe(moelib):
    import moe_expert_layer_08_b200 as m
    return m


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def decode(w, sf, fmt):
    """The weights as fp64 values."""
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device="cuda")
    codes = torch.stack([w & 15, w >> 4], 2).reshape(w.shape[0], -1).to(torch.int64)
    v = mag[codes & 7] * torch.where(codes > 7, -1.0, 1.0)
    b = sf.to(F64)
    if fmt == "mx":
        s = torch.where(sf == 255, float("nan"), torch.exp2(b - 127))
    else:
        c = sf.to(torch.int64) & 127
        e, m = c >> 3, (c & 7).to(F64)
        s = torch.where(e > 0, torch.exp2((e - 7).to(F64)) * (1 + m / 8), m * 2.0 ** -9)
        s = torch.where(c == 127, float("nan"), s)
    return v * s.repeat_interleave(v.shape[1] // sf.shape[1], 1)


def check(moe, x, w, sf, fmt):
    T, K = x.shape
    y = moe.fp4_matvec(x, w, sf, fmt=fmt)
    wv, xv = decode(w, sf, fmt), x.to(F64)
    exact, s = xv @ wv.T, xv.abs() @ wv.abs().T
    x_off = 2.0 ** -40 * xv.abs().amax(1, keepdim=True) * wv.abs().sum(1)[None]
    bound = ROUND * exact.abs() + (1 + ROUND) * ((K + 16) * 2.0 ** -23 * s + x_off) + 2.0 ** -133
    assert y.shape == exact.shape and bool(torch.isfinite(y).all())
    over = (y.to(F64) - exact).abs() > bound
    assert not bool(over.any()), f"{int(over.sum())} of {over.numel()} outside the bound"
    assert torch.equal(y, moe.fp4_matvec(x, w, sf, fmt=fmt))
    return y


def random_case(T, N, K, fmt, seed):
    g = generator(seed)
    x = torch.randn((T, K), dtype=BF16, device="cuda", generator=g)
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    low, high, group = (100, 140, 32) if fmt == "mx" else (0, 127, 16)
    sf = torch.randint(low, high, (N, K // group), dtype=torch.uint8, device="cuda", generator=g)
    return x, w, sf


@pytest.mark.parametrize("fmt", ["mx", "nvfp4"])
@pytest.mark.parametrize("T,N,K", [
    (1, 1, 32), (1, 16, 64), (2, 17, 256), (3, 15, 288), (7, 33, 2080), (8, 4099, 544), (9, 48, 1024),
    (17, 31, 7168), (1, 2500, 4128), (5, 40, 16384), (2, 18, 57344), (16, 5000, 96),
])
def test_sizes(moe, T, N, K, fmt):
    check(moe, *random_case(T, N, K, fmt, T * 7 + N), fmt)


@pytest.mark.parametrize("fmt,T,N,K", [
    ("mx", 8, 65600, 128), ("mx", 8, 30000, 384), ("mx", 7, 20011, 640),    # fewer than four stages, and an odd half
    ("mx", 1, 4099, 7168), ("mx", 8, 4099, 7168), ("mx", 12, 11000, 4096),  # tiles of any number of rows, two passes
    ("mx", 1, 50000, 256), ("mx", 8, 20011, 512), ("mx", 6, 19000, 1152),   # several tiles to a block
    ("mx", 1, 260, 26624), ("mx", 4, 65, 53248), ("mx", 2, 1, 7296),        # long parts
    ("nvfp4", 1, 1, 8192), ("nvfp4", 2, 200, 8320), ("nvfp4", 1, 129, 16512), ("nvfp4", 2, 40000, 256),
    ("nvfp4", 1, 4099, 7168), ("nvfp4", 2, 4099, 7168), ("nvfp4", 1, 65600, 128), ("nvfp4", 2, 19000, 1152),
    ("nvfp4", 1, 260, 26624), ("nvfp4", 2, 65, 26752),
    ("nvfp4", 3, 4099, 7168), ("nvfp4", 4, 4099, 7168), ("nvfp4", 3, 65600, 128), ("nvfp4", 4, 19000, 1152),
    ("nvfp4", 3, 50000, 384), ("nvfp4", 4, 65, 26752),
])
def test_whole_stages(moe, fmt, T, N, K):
    """K a multiple of 128, which the block-scaled tensor cores take (NVFP4: for
    four tokens at most)."""
    check(moe, *random_case(T, N, K, fmt, T * 11 + N), fmt)


@pytest.mark.parametrize("fmt,T,N,K", [
    ("mx", 17, 6300, 7168), ("mx", 8, 9, 57344), ("nvfp4", 2, 9, 57344),   # three passes; the longest rows
    ("mx", 3, 18, 57312), ("nvfp4", 3, 18, 57312), ("nvfp4", 8, 20, 28000),  # rows that leave room for few tokens
    ("nvfp4", 5, 300, 14336),
])
def test_largest(moe, fmt, T, N, K):
    check(moe, *random_case(T, N, K, fmt, T * 3 + N), fmt)


@pytest.mark.parametrize("fmt,T,bad", [("mx", 7, (1, 3, 5)), ("nvfp4", 2, (1,)), ("nvfp4", 1, (0,))])
def test_infinities_by_definition(moe, fmt, T, bad):
    """Tokens that are not finite give what the sum of their products gives."""
    x, w, sf = random_case(T, 300, 8320, fmt, 51)
    if fmt == "nvfp4":
        sf[sf == 127] = 0
    for t, at in zip(bad, ([7], [8319], [0, 900])):
        x[t, at] = float("-inf") if t == 3 else float("inf")
    y = moe.fp4_matvec(x, w, sf, fmt=fmt)
    exact = x.to(F64) @ decode(w, sf, fmt).T
    for t in bad:
        assert torch.equal(torch.isnan(y[t]), torch.isnan(exact[t]))
        inf = torch.isinf(exact[t])
        assert bool(inf.any()) and torch.equal(y[t][inf].to(F64), exact[t][inf])
    fine = [t for t in range(T) if t not in bad]
    if fine:
        check(moe, x[fine].contiguous(), w, sf, fmt)


def test_nvfp4_scales_at_their_ends(moe):
    x, w, sf = random_case(2, 40, 8192, "nvfp4", 71)
    sf[0], sf[1], sf[2] = 0, 126, 1
    sf[3] |= 128                   # bit 7 is not read
    sf[3][(sf[3] & 127) == 127] = 0
    for T in (1, 2):
        check(moe, x[:T].contiguous(), w, sf, "nvfp4")
    sf[5, 511] = 127
    for T in (1, 2):
        y = moe.fp4_matvec(x[:T].contiguous(), w, sf, fmt="nvfp4")
        assert bool(torch.isnan(y[:, 5]).all()) and bool(torch.isfinite(y[:, :5]).all() and torch.isfinite(y[:, 6:]).all())


def test_weights_at_16_bytes(moe):
    x, w, sf = random_case(2, 130, 8192, "mx", 61)
    room = torch.empty(w.numel() + 64, dtype=torch.uint8, device="cuda")
    at = (16 - room.data_ptr()) % 32
    moved = room[at:at + w.numel()].view(w.shape)
    assert moved.data_ptr() % 32 == 16
    moved.copy_(w)
    check(moe, x, moved, sf, "mx")


@pytest.mark.parametrize("fmt", ["mx", "nvfp4"])
def test_quantised_weights(moe, fmt):
    """Weights as the framework's quantisers write them."""
    g = generator(3)
    w = torch.randn((1000, 1536), dtype=BF16, device="cuda", generator=g).mul_(0.04)
    q, sf = (moe.quantize_fp4 if fmt == "mx" else moe.quantize_nvfp4)(w)
    x = torch.randn((4, 1536), dtype=BF16, device="cuda", generator=g)
    y = check(moe, x, q, sf, fmt)
    # E2M1 with its group's scale is off by at most a quarter of the weight's binade: far from a layout mistake
    rel = (y.to(F64) - x.to(F64) @ w.to(F64).T).norm() / (x.to(F64) @ w.to(F64).T).norm()
    assert rel < 0.25


@pytest.mark.parametrize("fmt", ["mx", "nvfp4"])
def test_tokens_of_a_wide_range(moe, fmt):
    """Outliers next to small elements, tokens of zeros, of the smallest and of
    large magnitudes."""
    x, w, sf = random_case(8, 100, 1056, fmt, 11)
    g = generator(12)
    x[0] *= torch.exp2(torch.randint(-40, 20, (1056,), device="cuda", generator=g).to(BF16))
    x[1] = 0
    x[2] *= 2.0 ** -110
    x[3] *= 2.0 ** 60
    x[4, 5] = 3e30
    x[5, ::2] = 0
    x[6] = 2.0 ** -133
    check(moe, x, w, sf, fmt)


def test_scales_at_their_ends(moe):
    x, w, sf = random_case(2, 16, 128, "mx", 21)
    x *= 2.0 ** 20
    sf[0] = 0                      # 2^-127
    sf[1] = 200                    # 2^73
    check(moe, x, w, sf, "mx")
    sf[2, 1] = 255                 # NaN
    y = moe.fp4_matvec(x, w, sf)
    assert bool(torch.isnan(y[:, 2]).all()) and bool(torch.isfinite(y[:, [0, 1] + list(range(3, 16))]).all())
    x, w, sf = random_case(2, 16, 128, "nvfp4", 22)
    sf[3] |= 128                   # bit 7 is not read
    sf[3][(sf[3] & 127) == 127] = 0
    check(moe, x, w, sf, "nvfp4")
    sf[5, 0] = 127
    assert bool(torch.isnan(moe.fp4_matvec(x, w, sf, fmt="nvfp4")[:, 5]).all())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_token_does_not_reach_another(moe, bad):
    x, w, sf = random_case(8, 64, 512, "mx", 31)
    w |= 0x22                      # no zero weights
    clean = moe.fp4_matvec(x, w, sf)
    x[3, 100] = bad
    y = moe.fp4_matvec(x, w, sf)
    others = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(y[others], clean[others]) and not bool(torch.isfinite(y[3]).any())


def test_graph_stream_and_given_output(moe):
    x, w, sf = random_case(3, 77, 640, "mx", 41)
    y = torch.empty((3, 77), dtype=BF16, device="cuda")
    assert moe.fp4_matvec(x, w, sf, out=y) is y
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.fp4_matvec(x, w, sf, out=y)
    x.copy_(random_case(3, 77, 640, "mx", 42)[0])
    graph.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = moe.fp4_matvec(x, w, sf, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, other)
    del graph


def test_refusals(moe):
    x, w, sf = random_case(2, 16, 64, "mx", 1)
    with pytest.raises(ValueError):
        moe.fp4_matvec(x, w, sf, fmt="int4")
    with pytest.raises(ValueError):
        moe.fp4_matvec(x, w, sf, fmt="nvfp4")            # twice as many scales there
    with pytest.raises(ValueError):
        moe.fp4_matvec(x[:, :32].contiguous(), w, sf)
    with pytest.raises(TypeError):
        moe.fp4_matvec(x.half(), w, sf)
    with pytest.raises(ValueError):
        moe.fp4_matvec(x.t(), w, sf)
    with pytest.raises(moe.MoEError) as e:
        moe.fp4_matvec(x[:, :48].contiguous(), w[:, :24].contiguous(), sf[:, :1].contiguous())
    assert e.value.status == 2
    assert moe.fp4_matvec(x[:0], w, sf).shape == (0, 16)
