"""The operators around the expert layer in a run, as a block uses them: a decode
step (norm -> routed experts and a shared expert held in 4 bits -> norm into the
residual stream) and a training step over unquantised experts with its
gradients."""
import os
import subprocess
import sys

import pytest
import torch

import workloads as W
from cases import gpu_layer

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64
ROUND = torch.finfo(BF16).eps / 2


@pytest.fixture(scope="module")
def moe(moelib):
    import moe_expert_layer_08_b200 as m
    return m


def normal(seed, *shape, scale=1.0, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, dtype=BF16, device="cuda", generator=g) * scale + mean


def norm64(x, w, eps):
    x = x.to(F64)
    return x * (x.pow(2).mean(1, keepdim=True) + eps).rsqrt() * w.to(F64)


@pytest.mark.parametrize("fmt", ["mx", "nvfp4"])
def test_decode_step(moe, fmt):
    """Eager and captured; the norm's quantised output runs the layer as the
    quantiser's would, and every step follows from the one before it within its
    own rounding: bf16 results to 2^-8 and a few fp32 roundings (2^-16 of the
    terms)."""
    w = W.custom("block", T=8, E=8, k=2, H=256, I=256, seed=3)
    g = gpu_layer(w)
    T, H, SI, eps = w.T, w.H, 384, 1e-6
    stream_in, before, after, gate = normal(1, T, H), normal(2, H, mean=1.0), normal(3, H, mean=1.0), normal(4, H)
    quantise = moe.quantize_fp4 if fmt == "mx" else moe.quantize_nvfp4
    up, up_sf = quantise(normal(5, 2 * SI, H, scale=0.05))
    down, down_sf = quantise(normal(6, H, SI, scale=0.05))

    def step():
        n = moe.norm_before(stream_in, before, eps, fp8=True)
        routed = moe.forward(n.x_fp8, n.x_sf, g["idx"], g["tw"], g["l1_t"], g["l2_t"], w.E, w.H, w.I)
        gu = moe.fp4_matvec(n.y, up, up_sf, fmt=fmt)
        h = torch.nn.functional.silu(gu[:, :SI].float()).mul(gu[:, SI:].float()).to(BF16)
        shared = moe.fp4_matvec(h, down, down_sf, fmt=fmt)
        both = routed + shared
        return n, routed, gu, h, shared, both, moe.norm_after(both, stream_in, after, eps, gate=gate).out

    n, routed, gu, h, shared, both, out = step()
    y = norm64(stream_in, before, eps)
    assert bool(((n.y.to(F64) - y).abs() <= (ROUND + 2.0 ** -16) * y.abs()).all())
    codes, sf = moe.quantize_fp8(n.y)
    assert torch.equal(routed, moe.forward(codes, sf, g["idx"], g["tw"], g["l1_t"], g["l2_t"], w.E, w.H, w.I))
    assert bool(shared.any()) and bool(torch.isfinite(shared).all())
    added = gate.to(F64) * norm64(both, after, eps)
    exact = stream_in.to(F64) + added
    bound = ROUND * exact.abs() + 2.0 ** -16 * (stream_in.to(F64).abs() + added.abs())
    assert bool(((out.to(F64) - exact).abs() <= bound).all())

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()[-1]
    stream_in.copy_(normal(9, T, H))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, step()[-1])
    del graph


def test_training_step(moe):
    """Forward and backward through norm, experts' products, gated activation,
    combine and norm against autograd in 64 bits.  A gradient passes at most 12
    tensors that are rounded to bf16 (2^-8 relative each, at most), so its
    relative 2-norm error stays below 12 * 2^-8."""
    T, E, k, H, I, eps, alpha = 96, 6, 2, 256, 128, 1e-5, 0.9
    x, n1, n2, gate = normal(1, T, H), normal(2, H, mean=1.0), normal(3, H, mean=1.0), normal(4, T, 1, mean=1.0)
    w1, w2 = normal(5, E, 2 * I, H, scale=0.06), normal(6, E, H, I, scale=0.09)
    dout = normal(7, T, H)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    idx = torch.rand((T, E - 1), device="cuda", generator=g).topk(k, 1).indices  # the last expert stays empty
    tw = torch.softmax(torch.randn((T, k), device="cuda", generator=g), 1)
    order = torch.argsort(idx.flatten(), stable=True)
    token, weight = order // k, tw.flatten()[order][:, None]
    offsets = torch.cat([torch.zeros(1, device="cuda"), torch.bincount(idx.flatten(), minlength=E).cumsum(0)]).int()

    # forward
    a = moe.norm_before(x, n1, eps, rstd=True)
    rows = a.y[token].contiguous()
    gu = moe.grouped_matmul(rows, w1, offsets)
    gt, up = gu[:, :I].float(), gu[:, I:].float()
    sig = torch.sigmoid(gt)
    h = (gt * sig * up).to(BF16)
    y = moe.grouped_matmul(h, w2, offsets)
    combined = torch.zeros((T, H), device="cuda").index_add_(0, token, weight * y.float()).to(BF16)
    b = moe.norm_after(combined, x, n2, eps, gate=gate, residual_scale=alpha, rstd=True)
    # backward
    dcombined, dresidual, dn2, dgate = moe.norm_after_backward(dout, combined, n2, b.rstd, gate=gate,
                                                               residual_scale=alpha)
    dy = (weight * dcombined.float()[token]).to(BF16)
    dh = moe.grouped_matmul_grad_input(dy, w2, offsets).float()
    dw2 = moe.grouped_matmul_grad_weight(dy, h, offsets)
    dgu = torch.cat([dh * up * (sig + gt * sig * (1 - sig)), dh * gt * sig], 1).to(BF16)
    drows = moe.grouped_matmul_grad_input(dgu, w1, offsets)
    dw1 = moe.grouped_matmul_grad_weight(dgu, rows, offsets)
    dnorm = torch.zeros((T, H), device="cuda").index_add_(0, token, drows.float()).to(BF16)
    dx, dn1 = moe.norm_before_backward(dnorm, x, n1, a.rstd, dresidual=dresidual)

    v = [t.to(F64).requires_grad_() for t in (x, n1, n2, gate, w1, w2)]
    X, N1, N2, G, W1, W2 = v
    r = (X * (X.pow(2).mean(1, keepdim=True) + eps).rsqrt() * N1)[token]
    expert = idx.flatten()[order]
    q = torch.einsum("rk,rnk->rn", r, W1[expert])
    z = torch.einsum("rk,rnk->rn", torch.nn.functional.silu(q[:, :I]) * q[:, I:], W2[expert])
    c = torch.zeros((T, H), dtype=F64, device="cuda").index_add(0, token, weight.to(F64) * z)
    out = alpha * X + G * (c * (c.pow(2).mean(1, keepdim=True) + eps).rsqrt() * N2)
    exact = torch.autograd.grad((out * dout.to(F64)).sum(), v)

    room = 12 * ROUND
    for name, got, want in zip(("out", "dx", "dn1", "dn2", "dgate", "dw1", "dw2"),
                               (b.out, dx, dn1, dn2, dgate, dw1, dw2), (out.detach(), *exact)):
        off = float((got.to(F64) - want).norm() / want.norm())
        assert off <= room, (name, off)
    assert not bool(dw1[E - 1].any()) and not bool(dw2[E - 1].any())


def test_two_streams_at_once(moe):
    """Calls of the same shapes under way on two streams, a graph's among them."""
    x, w = normal(1, 16, 2048), normal(2, 2, 520, 2048)
    off = torch.tensor([0, 7, 16], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    codes = torch.randint(0, 256, (9000, 1024), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(120, 130, (9000, 64), dtype=torch.uint8, device="cuda", generator=g)
    inputs = [(x, x[:8].contiguous()), (x * 2, (x[:8] * 3).contiguous())]
    expect = [(moe.grouped_matmul(a, w, off), moe.fp4_matvec(b, codes, scales)) for a, b in inputs]
    graph_out = torch.empty_like(expect[0][1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.fp4_matvec(inputs[0][1], codes, scales, out=graph_out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((moe.grouped_matmul(inputs[i][0], w, off), moe.fp4_matvec(inputs[i][1], codes, scales)))
        graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for y, z in got[i]:
            assert torch.equal(y, expect[i][0]) and torch.equal(z, expect[i][1])
    assert torch.equal(graph_out, expect[0][1])
    del graph


def test_small_clusters_of_two_streams(moe):
    """Launches of a few clusters each, which would fit an SM side by side: no
    block waits for what another cluster holds."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    cases = []
    for N in (200, 130):
        codes = torch.randint(0, 256, (N, 8192), dtype=torch.uint8, device="cuda", generator=g)
        scales = torch.randint(120, 130, (N, 512), dtype=torch.uint8, device="cuda", generator=g)
        cases.append((normal(N, 1, 16384), codes, scales))
    expect = [moe.fp4_matvec(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for _ in range(100):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i % 2, moe.fp4_matvec(*cases[i % 2])))
    torch.cuda.synchronize()
    assert all(torch.equal(y, expect[i]) for i, y in got)


def test_memory_of_calls_on_another_stream(moe):
    """Outputs and workspaces that a call on a given stream makes for itself are
    not handed to the current stream while that work is still to come."""
    x, dy, w = normal(1, 600, 4096), normal(2, 600, 4096), normal(3, 4096)
    off = torch.tensor([0, 250, 600], dtype=torch.int32, device="cuda")
    we = normal(4, 2, 264, 4096)
    rstd = moe.norm_before(x, w, rstd=True).rstd
    expect = [moe.norm_before_backward(dy, x, w, rstd), (moe.grouped_matmul(x, we, off),), tuple(moe.norm_before(x, w)[:1])]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    got = [moe.norm_before_backward(dy, x, w, rstd, stream=s), (moe.grouped_matmul(x, we, off, stream=s),),
           tuple(moe.norm_before(x, w, stream=s)[:1])]
    sizes = (moe.norm_workspace_bytes(600, 4096), moe.grouped_workspace_bytes(), 600 * 4096 * 2, 4096 * 4)
    mine = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    for a, b in zip(expect, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert all(bool((m == 0x5A).all()) for m in mine)


FIRST = """
import torch
import moe_expert_layer_08_b200 as moe
torch.manual_seed(0)
B = torch.bfloat16
x, w = torch.randn((16, 2048), dtype=B, device="cuda"), torch.randn((2, 520, 2048), dtype=B, device="cuda")
off = torch.tensor([0, 7, 16], dtype=torch.int32, device="cuda")
codes = torch.randint(0, 256, (9000, 1024), dtype=torch.uint8, device="cuda")
scales = torch.randint(120, 130, (9000, 64), dtype=torch.uint8, device="cuda")
gain = torch.randn(2048, dtype=B, device="cuda")
y, z = torch.empty((16, 520), dtype=B, device="cuda"), torch.empty((8, 9000), dtype=B, device="cuda")
ws = torch.empty(moe.grouped_workspace_bytes(), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    n = moe.norm_before(x, gain).y
    moe.grouped_matmul(n, w, off, out=y, workspace=ws)
    y2 = moe.grouped_matmul(n, w, off)
    moe.fp4_matvec(n[:8], codes, scales, out=z)
graph.replay()
torch.cuda.synchronize()
n2 = moe.norm_before(x, gain).y
assert torch.equal(n, n2)
assert torch.equal(y, moe.grouped_matmul(n2, w, off)) and torch.equal(z, moe.fp4_matvec(n2[:8], codes, scales))
assert moe.check_device_error(ws) == 0 and torch.equal(y, y2)
kept = y.clone()
del graph, n, y2
torch.cuda.empty_cache()
fill = [torch.full((4096,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(64)]
assert torch.equal(kept, moe.grouped_matmul(n2, w, off))
torch.cuda.synchronize()
assert all(bool((f == 0x5A).all()) for f in fill)
print("same")
"""


def test_first_calls_inside_a_capture(moelib):
    """A process whose first use of the operators is captured into a graph."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip() == "same", done.stderr[-2000:]
