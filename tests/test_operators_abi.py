"""CPU checks of the entry points around the expert layer: arguments are
validated on the host before any CUDA call (p is never dereferenced)."""
import ctypes

import pytest

p, odd, q2 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10002)
BIG = 1 << 40
INVALID, SHAPE, SMALL = 1, 2, 3


def test_grouped_products(moelib):
    for f in (moelib.moe_grouped_matmul, moelib.moe_grouped_matmul_grad_input):
        def call(x=p, w=p, off=p, y=p, R=4, E=2, N=64, K=32, zero=1, ws=p, n=BIG):
            return f(x, w, off, y, R, E, N, K, zero, ws, n, None)
        assert call(R=0, x=None, y=None, ws=None, n=0) == 0
        for kw in (dict(R=-1), dict(E=0), dict(N=0), dict(K=-8), dict(x=None), dict(w=None), dict(off=None),
                   dict(y=None), dict(ws=None), dict(x=q2), dict(w=q2), dict(off=q2), dict(y=q2),
                   dict(ws=ctypes.c_void_p(0x10010))):
            assert call(**kw) == INVALID, kw
        for kw in (dict(N=60), dict(K=36), dict(E=1025), dict(N=131080), dict(K=131080), dict(R=2 ** 31 - 1, N=8, K=8)):
            assert call(**kw) == SHAPE, kw
        assert call(n=64) == SMALL
    g = moelib.moe_grouped_matmul_grad_weight

    def call(dy=p, x=p, off=p, dw=p, R=4, E=2, N=64, K=32, ws=p, n=BIG):
        return g(dy, x, off, dw, R, E, N, K, ws, n, None)
    for kw in (dict(R=-1), dict(dy=None), dict(x=None), dict(off=None), dict(dw=None), dict(ws=None), dict(dy=q2),
               dict(R=0, dw=None)):
        assert call(**kw) == INVALID, kw
    assert call(N=4) == SHAPE and call(n=0) == SMALL
    assert moelib.moe_grouped_workspace_bytes(None) == INVALID


def test_matvec(moelib):
    def call(x=p, w=p, sf=p, y=p, T=1, N=16, K=64, fmt=0):
        return moelib.moe_fp4_matvec(x, w, sf, y, T, N, K, fmt, None)
    assert call(T=0, x=None, w=None, sf=None, y=None) == 0
    for kw in (dict(T=-1), dict(N=0), dict(K=0), dict(fmt=2), dict(fmt=-1), dict(x=None), dict(w=None), dict(sf=None),
               dict(y=None), dict(x=q2), dict(w=q2), dict(sf=q2), dict(y=odd)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(K=48), dict(K=57376), dict(T=65536), dict(N=2 ** 31 - 1)):
        assert call(**kw) == SHAPE, kw


NAN, INF = float("nan"), float("inf")


def test_norm_before(moelib):
    def call(x=p, w=p, T=2, H=64, eps=1e-6, y=p, q=p, sf=p, r=p):
        return moelib.moe_norm_before(x, w, T, H, eps, y, q, sf, r, None)
    assert call(T=0, x=None, w=None, y=None, q=None, sf=None, r=None) == 0
    for kw in (dict(T=-1), dict(H=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(x=None),
               dict(w=None), dict(y=None, q=None, sf=None), dict(q=None), dict(sf=None), dict(x=q2), dict(w=q2),
               dict(y=q2), dict(q=q2), dict(r=q2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=60), dict(H=16392), dict(H=40), dict(T=2 ** 31 - 1)):
        assert call(**kw) == SHAPE, kw


def test_norm_after(moelib):
    def call(x=p, res=p, w=p, g=p, kind=1, T=2, H=64, eps=1e-6, a=1.0, out=p, r=None):
        return moelib.moe_norm_after(x, res, w, g, kind, T, H, eps, a, out, r, None)
    assert call(T=0, x=None, res=None, w=None, g=None, out=None) == 0
    for kw in (dict(T=-1), dict(H=-8), dict(kind=-1), dict(kind=4), dict(a=NAN), dict(a=INF), dict(eps=0.0),
               dict(x=None), dict(res=None), dict(w=None), dict(g=None), dict(out=None), dict(g=q2),
               dict(g=odd, kind=2), dict(res=q2), dict(out=q2)):
        assert call(**kw) == INVALID, kw
    assert call(H=12) == SHAPE and call(H=16392) == SHAPE


def test_norm_gradients(moelib):
    n = ctypes.c_size_t()
    assert moelib.moe_norm_workspace_bytes(4, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert moelib.moe_norm_workspace_bytes(4, 60, ctypes.byref(n)) == SHAPE
    assert moelib.moe_norm_workspace_bytes(-1, 64, ctypes.byref(n)) == INVALID
    assert moelib.moe_norm_workspace_bytes(4, 64, None) == INVALID

    def before(dy=p, x=p, w=p, r=p, res=None, T=2, H=64, dx=p, dw=p, ws=p, size=BIG):
        return moelib.moe_norm_before_backward(dy, x, w, r, res, T, H, dx, dw, ws, size, None)
    for kw in (dict(T=-1), dict(dy=None), dict(x=None), dict(w=None), dict(r=None), dict(dx=None), dict(dw=None),
               dict(ws=None), dict(dy=q2), dict(res=q2), dict(T=0, dw=None)):
        assert before(**kw) == INVALID, kw
    assert before(H=20) == SHAPE and before(size=16) == SMALL

    def after(do=p, x=p, w=p, r=p, g=p, kind=1, T=2, H=64, a=1.0, dx=p, dres=p, dw=p, dg=p, ws=p, size=BIG):
        return moelib.moe_norm_after_backward(do, x, w, r, g, kind, T, H, a, dx, dres, dw, dg, ws, size, None)
    for kw in (dict(kind=5), dict(a=NAN), dict(do=None), dict(x=None), dict(w=None), dict(r=None), dict(g=None),
               dict(dx=None), dict(dres=None), dict(dw=None), dict(dg=None), dict(dg=None, kind=2),
               dict(dg=None, kind=3), dict(ws=None), dict(g=q2, kind=3), dict(T=0, dg=None)):
        assert after(**kw) == INVALID, kw
    assert after(H=20) == SHAPE and after(size=16) == SMALL


@pytest.mark.parametrize("name", ["grouped_matmul", "fp4_matvec", "norm_before", "norm_after"])
def test_the_binding_takes_cuda_tensors_only(moelib, name):
    import torch
    import moe_expert_layer_08_b200 as m
    t = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        getattr(m, name)(t, t, t)


def test_the_bindings_workspace_of_the_grouped_products(moelib):
    import moe_expert_layer_08_b200 as m
    assert m._GROUPED_WORKSPACE == m.grouped_workspace_bytes()
