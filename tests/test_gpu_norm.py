"""GPU tests of the norms before and after the layer and their gradients
against the definition in 64 bits, the quantised output against the quantiser.

Tolerances, element by element.  A result is rounded to bf16 once (2^-8
relative).  In front of that: a row's sums take at most 128 additions in a
thread and 10 across threads, off by 2^-24 of the sum of magnitudes each
(2^-16.9 in all; half of that in rstd), and the products around them a few
2^-24 more: FP = 2^-16 of the terms' magnitudes covers them.  A column sum over
T tokens takes at most T + 16 additions: (T + 16) 2^-24 of the magnitudes more."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ROUND = torch.finfo(BF16).eps / 2
FP = 2.0 ** -16
TINY = 2.0 ** -133
SIZES = [(1, 8), (1, 32), (3, 40), (2, 1000), (5, 7168), (1, 16384), (150, 264), (300, 7168), (333, 4096),
         (4097, 96), (149, 16384), (700, 2056)]
GATES = ["none", "channel", "token", "full"]


@pytest.fixture(scope="module")
def moe(moelib):
    import moe_expert_layer_08_b200 as m
    return m


class Case:
    def __init__(self, T, H, gate="none", seed=0, scale=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, dtype=BF16, device="cuda", generator=g)
        self.T, self.H, self.eps, self.alpha = T, H, 1e-5, -0.75
        self.x, self.w, self.res = normal(T, H) * scale, normal(H) + 1, normal(T, H)
        self.dy, self.dres = normal(T, H), normal(T, H)
        shape = {"channel": (H,), "token": (T, 1), "full": (T, H)}.get(gate)
        self.gate = normal(*shape) if shape else None

    def exact(self):
        x, w = self.x.to(F64), self.w.to(F64)
        rstd = (x.pow(2).mean(1, keepdim=True) + self.eps).rsqrt()
        return x * rstd, w, rstd


def within(got, exact, bound, what):
    assert got.shape == exact.shape, what
    assert bool(torch.isfinite(got).all()), what
    over = (got.to(F64) - exact).abs() > bound + TINY
    assert not bool(over.any()), f"{what}: {int(over.sum())} of {over.numel()} outside the bound"


@pytest.mark.parametrize("T,H", SIZES)
def test_before(moe, T, H):
    c = Case(T, H, seed=T)
    xhat, w, rstd = c.exact()
    n = moe.norm_before(c.x, c.w, c.eps, rstd=True)
    assert n.x_fp8 is None and n.x_sf is None
    within(n.rstd, rstd[:, 0], FP * rstd[:, 0], "rstd")
    y = xhat * w
    within(n.y, y, (ROUND + FP) * y.abs(), "y")
    if H % 32 == 0:
        both = moe.norm_before(c.x, c.w, c.eps, fp8=True)
        only = moe.norm_before(c.x, c.w, c.eps, bf16=False, fp8=True)
        codes, sf = moe.quantize_fp8(n.y)
        assert torch.equal(both.y, n.y) and only.y is None
        for q in (both, only):
            assert torch.equal(q.x_fp8, codes) and torch.equal(q.x_sf, sf)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,H", SIZES)
def test_after(moe, T, H, gate):
    c = Case(T, H, gate, seed=T + 1)
    xhat, w, rstd = c.exact()
    g = torch.ones((), dtype=F64, device="cuda") if c.gate is None else c.gate.to(F64)
    kept, added = c.alpha * c.res.to(F64), g * xhat * w
    n = moe.norm_after(c.x, c.res, c.w, c.eps, gate=c.gate, residual_scale=c.alpha, rstd=True)
    within(n.rstd, rstd[:, 0], FP * rstd[:, 0], "rstd")
    within(n.out, kept + added, ROUND * (kept + added).abs() + FP * (kept.abs() + added.abs()), "out")
    # into the residual itself
    res = c.res.clone()
    assert moe.norm_after(c.x, res, c.w, c.eps, gate=c.gate, residual_scale=c.alpha, out=res).out is res
    assert torch.equal(res, n.out)


def check_dx(dx, c, dz, rstd, dres):
    """dx from dz, the gradient that reaches xhat * w, with the kernel's rstd."""
    r = rstd.to(F64)[:, None]
    xhat, dxhat = c.x.to(F64) * r, dz * c.w.to(F64)
    exact = r * (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True)) + dres
    terms = r * (dxhat.abs() + xhat.abs() * (dxhat * xhat).abs().mean(1, keepdim=True)) + dres.abs()
    within(dx, exact, ROUND * exact.abs() + FP * terms, "dx")


@pytest.mark.parametrize("with_residual", [True, False])
@pytest.mark.parametrize("T,H", SIZES)
def test_before_gradients(moe, T, H, with_residual):
    c = Case(T, H, seed=T + 2)
    rstd = moe.norm_before(c.x, c.w, c.eps, rstd=True).rstd
    dres = c.dres if with_residual else None
    dx, dw = moe.norm_before_backward(c.dy, c.x, c.w, rstd, dresidual=dres)
    check_dx(dx, c, c.dy.to(F64), rstd, c.dres.to(F64) if with_residual else torch.zeros((), dtype=F64, device="cuda"))
    terms = c.dy.to(F64) * c.x.to(F64) * rstd.to(F64)[:, None]
    within(dw, terms.sum(0), (FP + (T + 16) * 2.0 ** -24) * terms.abs().sum(0), "dweight")
    again = moe.norm_before_backward(c.dy, c.x, c.w, rstd, dresidual=dres)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,H", SIZES)
def test_after_gradients(moe, T, H, gate):
    c = Case(T, H, gate, seed=T + 3)
    rstd = moe.norm_after(c.x, c.res, c.w, c.eps, gate=c.gate, rstd=True).rstd
    dx, dres, dw, dg = moe.norm_after_backward(c.dy, c.x, c.w, rstd, gate=c.gate, residual_scale=c.alpha)
    dout = c.dy.to(F64)
    dz = dout if c.gate is None else dout * c.gate.to(F64)
    check_dx(dx, c, dz, rstd, torch.zeros((), dtype=F64, device="cuda"))
    within(dres, c.alpha * dout, (ROUND + FP) * (c.alpha * dout).abs(), "dresidual")
    xhat = c.x.to(F64) * rstd.to(F64)[:, None]
    column = FP + (T + 16) * 2.0 ** -24
    within(dw, (dz * xhat).sum(0), column * (dz * xhat).abs().sum(0), "dweight")
    terms = dout * xhat * c.w.to(F64)
    if gate == "none":
        assert dg is None
    elif gate == "channel":
        within(dg, terms.sum(0), column * terms.abs().sum(0), "dgate")
    elif gate == "token":
        within(dg, terms.sum(1, keepdim=True), FP * terms.abs().sum(1, keepdim=True), "dgate")
    else:
        assert dg.dtype == BF16
        within(dg, terms, (ROUND + FP) * terms.abs(), "dgate")
    again = moe.norm_after_backward(c.dy, c.x, c.w, rstd, gate=c.gate, residual_scale=c.alpha)
    for a, b in zip((dx, dres, dw, dg), again):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("gate", GATES)
def test_gradients_against_differences(moe, gate):
    """Central differences of <out, dout> in 64 bits, along a random direction
    of every input, against the gradients along it.  The difference is off by
    h^2 times a third derivative of order one in units of the terms: h = 2^-12
    leaves 2^-24 of them, next to the gradients' own rounding."""
    c = Case(6, 264, gate, seed=9)
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    rstd = moe.norm_after(c.x, c.res, c.w, c.eps, gate=c.gate, rstd=True).rstd
    grads = moe.norm_after_backward(c.dy, c.x, c.w, rstd, gate=c.gate, residual_scale=c.alpha)
    inputs = [c.x, c.res, c.w] + ([] if c.gate is None else [c.gate])
    values = [t.to(F64) for t in inputs]

    def loss(v):
        x, res, w = v[:3]
        z = x * (x.pow(2).mean(1, keepdim=True) + c.eps).rsqrt() * w
        return ((c.alpha * res + (z if len(v) < 4 else v[3] * z)) * c.dy.to(F64)).sum()

    h = 2.0 ** -12
    for i, grad in enumerate(t for t in grads if t is not None):
        d = torch.randn(values[i].shape, dtype=F64, device="cuda", generator=g)
        up, down = [v.clone() for v in values], [v.clone() for v in values]
        up[i] += h * d
        down[i] -= h * d
        difference = float((loss(up) - loss(down)) / (2 * h))
        along = (grad.to(F64).reshape(d.shape) * d)
        room = float((along.abs() * ROUND).sum()) + 2.0 ** -12 * float(along.abs().sum())
        assert abs(float(along.sum()) - difference) <= room, i


def test_magnitudes(moe):
    """Rows of zeros (eps alone), of tiny and of huge elements, and a row with
    NaN, which stays in its row."""
    c = Case(6, 512, seed=4)
    c.x[0] = 0
    c.x[1] *= 2.0 ** -100
    c.x[2] *= 2.0 ** 50
    c.x[3, 7:] = 0
    xhat, w, _ = c.exact()
    n = moe.norm_before(c.x, c.w, c.eps, fp8=True)
    within(n.y, xhat * w, (ROUND + FP) * (xhat * w).abs(), "y")
    assert not bool(n.y[0].any()) and bool((n.x_sf[0] == 127).all())
    codes, sf = moe.quantize_fp8(n.y)
    assert torch.equal(n.x_fp8, codes) and torch.equal(n.x_sf, sf)
    c.x[5, 100] = float("nan")
    bad = moe.norm_before(c.x, c.w, c.eps).y
    assert torch.equal(bad[:5], n.y[:5]) and bool(torch.isnan(bad[5]).all())


def test_no_tokens(moe):
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    n = moe.norm_before(e, w, fp8=True, rstd=True)
    assert n.y.shape == (0, 64) and n.x_sf.shape == (0, 2)
    dx, dw = moe.norm_before_backward(e, e, w, n.rstd)
    assert dx.shape == (0, 64) and not bool(dw.any())
    _, _, dw, dg = moe.norm_after_backward(e, e, w, n.rstd, gate=w)
    assert not bool(dw.any()) and not bool(dg.any())


def test_graph_and_stream(moe):
    """One captured step, forward and backward, replayed on changed inputs,
    against eager calls on another stream."""
    c, other = Case(200, 1024, "channel", seed=5), Case(200, 1024, "channel", seed=6)

    def step(stream=None):
        n = moe.norm_before(c.x, c.w, c.eps, rstd=True, stream=stream)
        a = moe.norm_after(n.y, c.res, c.w, c.eps, gate=c.gate, rstd=True, stream=stream)
        back = moe.norm_after_backward(c.dy, n.y, c.w, a.rstd, gate=c.gate, stream=stream)
        return (a.out, *back, *moe.norm_before_backward(back[0], c.x, c.w, n.rstd, dresidual=back[1], stream=stream))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for name in ("x", "res", "dy", "gate"):
        getattr(c, name).copy_(getattr(other, name))
    graph.replay()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        eager = step(s)
    torch.cuda.synchronize()
    for a, b in zip(captured, eager):
        assert torch.equal(a, b)
    del graph


def test_refusals(moe):
    c = Case(4, 64, "channel")
    r = torch.ones(4, dtype=F32, device="cuda")
    with pytest.raises(ValueError):
        moe.norm_before(c.x, c.w, bf16=False)
    with pytest.raises(ValueError):
        moe.norm_before(c.x, c.w[:32].contiguous())
    with pytest.raises(TypeError):
        moe.norm_before(c.x, c.w.float())
    with pytest.raises(ValueError):
        moe.norm_before(c.x.t(), c.w)
    with pytest.raises(ValueError):
        moe.norm_after(c.x, c.res[:2].contiguous(), c.w)
    with pytest.raises(ValueError):
        moe.norm_after(c.x, c.res, c.w, gate=c.gate[:4].contiguous())
    with pytest.raises(ValueError):
        moe.norm_after_backward(c.dy, c.x, c.w, r[:3].contiguous())
    for kw in (dict(eps=0.0), dict(eps=float("nan"))):
        with pytest.raises(moe.MoEError) as e:
            moe.norm_before(c.x, c.w, **kw)
        assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.norm_after(c.x, c.res, c.w, residual_scale=float("inf"))
    assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.norm_before(torch.zeros((2, 40), dtype=BF16, device="cuda"), torch.ones(40, dtype=BF16, device="cuda"),
                        fp8=True)
    assert e.value.status == 2
    with pytest.raises(moe.MoEError) as e:
        moe.norm_before_backward(c.dy, c.x, c.w, r, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
