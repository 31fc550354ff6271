"""GPU tests of the experts' bf16 products over ragged groups and their
gradients against the definition in 64 bits.

Tolerance, element by element: the result is one rounding to bf16 (2^-8
relative) of an fp32 sum of C products, which are exact; each of at most C
additions is off by at most 2^-23 of a partial sum (truncation allowed), and
partial sums stay below S = sum |a b|.  So |got - exact| <= 2^-8 |exact| +
(1 + 2^-8) C 2^-23 S; 2^-133 for results below bf16's normal range."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64
ROUND = torch.finfo(BF16).eps / 2


@pytest.fixture(scope="module")
def moe(moelib):
    import moe_expert_layer_08_b200 as m
    return m


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, dtype=BF16, device="cuda", generator=g)


def offsets_of(sizes, before=0):
    ends = [before]
    for n in sizes:
        ends.append(ends[-1] + n)
    return ends, torch.tensor(ends, dtype=torch.int32, device="cuda")


def close(got, exact, magnitude, length):
    assert got.shape == exact.shape
    bound = ROUND * exact.abs() + (1 + ROUND) * length * 2.0 ** -23 * magnitude + 2.0 ** -133
    over = (got.to(F64) - exact).abs() > bound
    assert bool(torch.isfinite(got).all())
    assert not bool(over.any()), f"{int(over.sum())} of {over.numel()} outside the bound"


def check_all(moe, sizes, N, K, before=0, behind=0, seed=0):
    ends, off = offsets_of(sizes, before)
    E, R = len(sizes), ends[-1] + behind
    x, dy, w = normal(seed, R, K), normal(seed + 1, R, N), normal(seed + 2, E, N, K)
    ws = torch.full((moe.grouped_workspace_bytes(),), 0xAB, dtype=torch.uint8, device="cuda")
    y = moe.grouped_matmul(x, w, off, workspace=ws)
    assert moe.check_device_error(ws) == 0
    dx = moe.grouped_matmul_grad_input(dy, w, off, workspace=ws)
    assert moe.check_device_error(ws) == 0
    dw = moe.grouped_matmul_grad_weight(dy, x, off, workspace=ws)
    assert moe.check_device_error(ws) == 0
    assert y.shape == (R, N) and dx.shape == (R, K) and dw.shape == (E, N, K)
    for t in (y, dx):
        assert not bool(t[:ends[0]].any()) and not bool(t[ends[-1]:].any())
    for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        xe, de, we = x[a:b].to(F64), dy[a:b].to(F64), w[e].to(F64)
        close(y[a:b], xe @ we.T, xe.abs() @ we.abs().T, K)
        close(dx[a:b], de @ we, de.abs() @ we.abs(), N)
        close(dw[e], de.T @ xe, de.abs().T @ xe.abs(), b - a)
    # the same bits again
    assert torch.equal(y, moe.grouped_matmul(x, w, off))
    assert torch.equal(dx, moe.grouped_matmul_grad_input(dy, w, off))
    assert torch.equal(dw, moe.grouped_matmul_grad_weight(dy, x, off))


@pytest.mark.parametrize("sizes,N,K,before,behind", [
    ([1], 8, 8, 0, 0),                                       # the smallest call
    ([1], 264, 520, 0, 0),
    ([3, 0, 2], 128, 64, 0, 0),
    ([0, 1, 15, 16, 17, 0, 33, 64, 65, 0], 264, 136, 0, 0),  # every edge of the 16-row steps
    ([5, 0, 3, 1], 72, 1000, 2, 3),                          # rows of no expert on both sides
    ([255, 256, 257], 136, 72, 0, 0),                        # every edge of a row chunk
    ([600, 0, 3], 520, 264, 0, 40),
    ([5000], 256, 128, 0, 0),                                # more row chunks than a block of them
    ([4500, 0, 4200], 776, 200, 7, 0),                       # chunk blocks, several strips
    ([0, 0, 0], 64, 64, 0, 5),                               # rows, but none of an expert
    ([1] * 1024, 16, 24, 0, 0),                              # as many experts as there may be
    ([40, 1, 0, 7, 130], 7168, 2048, 0, 0),                  # the layer's widths
])
def test_products_and_gradients(moe, sizes, N, K, before, behind):
    check_all(moe, sizes, N, K, before, behind)


@pytest.mark.parametrize("turned", [False, True])  # for the input gradient as for the product
@pytest.mark.parametrize("sizes,N,K", [
    # the contraction in 8 and in 4 parts (in 2: [10] * 20, turned)
    ([33], 264, 2056), ([1], 264, 1032), ([9, 0, 5, 26], 264, 1032), ([70, 1], 1032, 520),
    # 64, 160 and 256 columns, each with one tile a strip and with two
    ([50, 0, 250], 520, 264), ([10] * 20, 1032, 136),
    ([90, 0, 210], 4096, 264), ([130] * 19 + [131], 1032, 136), ([80, 130, 50, 0, 88, 110, 100, 42], 4096, 264),
    ([190, 0, 150, 300, 200, 260, 300], 2056, 136), ([250, 150] * 10, 1032, 136), ([1990, 0], 4096, 136),
])
def test_every_shape_of_a_work_item(moe, sizes, N, K, turned):
    check_all(moe, sizes, *((K, N) if turned else (N, K)), before=3, behind=9, seed=3)


@pytest.mark.parametrize("sizes,N,K", [
    ([70], 192, 320), ([300, 0, 20], 320, 448), ([100, 37, 0, 260], 320, 512), ([65, 1, 64], 64, 256),
    ([700, 900], 1088, 768), ([129] * 12, 832, 1280),
])
def test_widths_of_whole_chunks(moe, sizes, N, K):
    """Widths that are multiples of 64, odd and even, and of 256: operands come
    two chunks of 64 columns at a time."""
    check_all(moe, sizes, N, K, before=2, behind=3, seed=8)


def test_decode_load_with_one_hot_expert(moe):
    """A mean load of at most 8 rows (32-row chunks) with an expert of 150."""
    check_all(moe, [0] * 20 + [150] + [1] * 30 + [2, 33, 32], 392, 328, seed=5)


def test_no_rows(moe):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty((0, 64), dtype=BF16, device="cuda"), torch.empty((0, 128), dtype=BF16, device="cuda")
    w = normal(1, 3, 128, 64)
    assert moe.grouped_matmul(x, w, off).shape == (0, 128)
    assert moe.grouped_matmul_grad_input(dy, w, off).shape == (0, 64)
    dw = torch.full((3, 128, 64), 7.0, dtype=BF16, device="cuda")
    assert moe.grouped_matmul_grad_weight(dy, x, off, out=dw) is dw and not bool(dw.any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_result_depends_on_its_own_group_alone(moe, bad):
    """Infinities and NaN in rows of no expert, in another expert's rows and in
    an unused expert's weights leave every other result as it was."""
    sizes, N, K = [5, 0, 21, 9, 70], 136, 200
    ends, off = offsets_of(sizes, 3)
    R = ends[-1] + 4
    x, dy, w = normal(1, R, K), normal(2, R, N), normal(3, 5, N, K)
    clean = (moe.grouped_matmul(x, w, off), moe.grouped_matmul_grad_input(dy, w, off),
             moe.grouped_matmul_grad_weight(dy, x, off))
    for t in (x, dy):
        t[:3] = bad
        t[ends[2]:ends[3]] = bad   # expert 2's rows
        t[ends[-1]:] = bad
    w[1] = bad                     # expert 1 has no rows
    y, dx, dw = (moe.grouped_matmul(x, w, off), moe.grouped_matmul_grad_input(dy, w, off),
                 moe.grouped_matmul_grad_weight(dy, x, off))
    keep = [r for r in range(R) if not ends[2] <= r < ends[3]]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(dx[keep], clean[1][keep])
    assert torch.equal(dw[[0, 1, 3, 4]], clean[2][[0, 1, 3, 4]])
    assert not bool(torch.isfinite(y[ends[2]:ends[3]]).any()) and not bool(torch.isfinite(dw[2]).any())


def test_rows_of_no_expert_in_a_given_output(moe):
    """left as they were, while a new output has zeros there."""
    sizes, N, K = [4, 0, 30], 72, 40
    ends, off = offsets_of(sizes, 2)
    R = ends[-1] + 300
    x, dy, w = normal(1, R, K), normal(2, R, N), normal(3, 3, N, K)
    for fn, rows, width in ((moe.grouped_matmul, x, N), (moe.grouped_matmul_grad_input, dy, K)):
        fresh = fn(rows, w, off)
        out = torch.full((R, width), 7.0, dtype=BF16, device="cuda")
        assert fn(rows, w, off, out=out) is out
        inside = slice(ends[0], ends[-1])
        assert torch.equal(out[inside], fresh[inside])
        assert bool((out[:2] == 7).all()) and bool((out[ends[-1]:] == 7).all())
        assert not bool(fresh[:2].any()) and not bool(fresh[ends[-1]:].any())


@pytest.mark.parametrize("given,read", [
    ([0, 9, 4, 20], [0, 9, 9, 20]),       # decreasing: the running maximum
    ([-5, 6, 8, 99], [0, 6, 8, 20]),      # outside [0, R]: clamped
    ([2 ** 31 - 1, 0, -2 ** 31, 3], [20, 20, 20, 20]),
])
def test_bad_offsets_are_reported(moe, given, read):
    R, N, K = 20, 64, 48
    x, dy, w = normal(1, R, K), normal(2, R, N), normal(3, 3, N, K)
    bad = torch.tensor(given, dtype=torch.int32, device="cuda")
    good = torch.tensor(read, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.grouped_workspace_bytes(), dtype=torch.uint8, device="cuda")
    for fn, args in ((moe.grouped_matmul, (x, w)), (moe.grouped_matmul_grad_input, (dy, w)),
                     (moe.grouped_matmul_grad_weight, (dy, x))):
        got = fn(*args, bad, workspace=ws)
        assert moe.check_device_error(ws) == 5  # MOE_ERR_BAD_ROUTING
        assert torch.equal(got, fn(*args, good, workspace=ws))
        assert moe.check_device_error(ws) == 0


def test_gradients_are_the_products_differences(moe):
    """With small whole numbers every sum is exact, in bf16 too (|sum| <= 256):
    the change of <dy, y> for a step in x or w is the gradient times the step."""
    sizes, N, K = [3, 0, 10, 6], 24, 16
    ends, off = offsets_of(sizes)
    R, E = ends[-1], len(sizes)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)

    def whole(*shape):
        return torch.randint(-1, 2, shape, device="cuda", generator=g).to(BF16)

    x, dy, w, sx, sw = whole(R, K), whole(R, N), whole(E, N, K), whole(R, K), whole(E, N, K)

    def loss(x, w):
        return (moe.grouped_matmul(x, w, off).to(F64) * dy.to(F64)).sum()

    dx, dw = moe.grouped_matmul_grad_input(dy, w, off).to(F64), moe.grouped_matmul_grad_weight(dy, x, off).to(F64)
    assert float(loss(x + sx, w) - loss(x, w)) == float((dx * sx.to(F64)).sum())
    assert float(loss(x, w + sw) - loss(x, w)) == float((dw * sw.to(F64)).sum())


def test_captured_call_follows_its_buffers(moe):
    """A graph of the three calls, replayed after the rows and the offsets
    changed in place; eager calls on another stream in between."""
    E, N, K, R = 6, 264, 136, 200
    w = normal(3, E, N, K)
    x, dy = normal(1, R, K), normal(2, R, N)
    off = offsets_of([50, 0, 70, 10, 0, 40])[1]
    ws = torch.empty(moe.grouped_workspace_bytes(), dtype=torch.uint8, device="cuda")
    y, dx = torch.empty((R, N), dtype=BF16, device="cuda"), torch.empty((R, K), dtype=BF16, device="cuda")
    dw = torch.empty((E, N, K), dtype=BF16, device="cuda")

    def calls():
        moe.grouped_matmul(x, w, off, out=y, workspace=ws)
        moe.grouped_matmul_grad_input(dy, w, off, out=dx, workspace=ws)
        moe.grouped_matmul_grad_weight(dy, x, off, out=dw, workspace=ws)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed, sizes in ((10, [0, 0, 200, 0, 0, 0]), (20, [33, 1, 0, 90, 76, 0])):
        x.copy_(normal(seed, R, K))
        dy.copy_(normal(seed + 1, R, N))
        off.copy_(offsets_of(sizes)[1])
        graph.replay()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        eager = (moe.grouped_matmul(x, w, off, stream=other), moe.grouped_matmul_grad_input(dy, w, off, stream=other),
                 moe.grouped_matmul_grad_weight(dy, x, off, stream=other))
        torch.cuda.synchronize()
        assert moe.check_device_error(ws) == 0
        assert torch.equal(y, eager[0]) and torch.equal(dx, eager[1]) and torch.equal(dw, eager[2])
    del graph


def test_routing_metadata_gives_the_groups(moe):
    """Offsets as read_routing returns them."""
    import workloads as W
    from cases import gpu_layer
    w = W.WORKLOADS[0]
    g = gpu_layer(w)
    ws = torch.empty(moe.workspace_bytes(w.T, w.E, w.k, w.H, w.I), dtype=torch.uint8, device="cuda")
    moe.forward(g["xq"], g["xs"], g["idx"], g["tw"], g["l1_t"], g["l2_t"], w.E, w.H, w.I, workspace=ws)
    r = moe.read_routing(ws, w.T, w.E, w.k, w.H, w.I)
    x, weights = normal(1, w.T, 64), normal(2, w.E, 40, 64)
    rows = x[(r["perm"] // w.k).to("cuda", torch.int64)]
    y = moe.grouped_matmul(rows, weights, r["offset"].cuda())
    expert = g["idx"].flatten()[r["perm"].to("cuda", torch.int64)]
    exact = torch.einsum("rk,rnk->rn", rows.to(F64), weights[expert].to(F64))
    close(y, exact, torch.einsum("rk,rnk->rn", rows.to(F64).abs(), weights[expert].to(F64).abs()), 64)


def test_refusals(moe):
    x, dy, w = normal(1, 4, 64), normal(2, 4, 32), normal(3, 2, 32, 64)
    off = offsets_of([2, 2])[1]
    with pytest.raises(TypeError):
        moe.grouped_matmul(x.float(), w, off)
    with pytest.raises(TypeError):
        moe.grouped_matmul(x, w, off.long())
    with pytest.raises(TypeError):
        moe.grouped_matmul(x.cpu(), w, off)
    with pytest.raises(ValueError):
        moe.grouped_matmul(x[:, ::2], w[:, :, :32].contiguous(), off)  # strided rows
    with pytest.raises(ValueError):
        moe.grouped_matmul(dy, w, off)                                 # K of the rows
    with pytest.raises(ValueError):
        moe.grouped_matmul_grad_input(x, w, off)
    with pytest.raises(ValueError):
        moe.grouped_matmul(x, w, off[:-1])
    with pytest.raises(ValueError):
        moe.grouped_matmul(x, w, off, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        moe.grouped_matmul_grad_weight(dy[:3].contiguous(), x, off)
    with pytest.raises(moe.MoEError) as e:
        moe.grouped_matmul(x[:, :60].contiguous(), w[:, :, :60].contiguous(), off)  # K % 8
    assert e.value.status == 2
    with pytest.raises(moe.MoEError) as e:
        moe.grouped_matmul(x, w, off, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(moe.MoEError) as e:
        moe.grouped_matmul(normal(1, 1, 4 * 64 + 1)[0, 1:].view(4, 64), w, off)     # 2-byte aligned rows
    assert e.value.status == 1
