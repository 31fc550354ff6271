"""Gradients that autograd would leave out: a result of the operators around the
layer refuses a backward pass through it and names what to call instead."""
import pytest
import torch


def test_a_tied_result(moelib):
    import moe_expert_layer_08_b200 as m
    x, w = torch.randn(4, 8, requires_grad=True), torch.randn(8)
    y = torch.randn(4, 8)
    assert m._tied(y, "f", "its gradient is g", w, None) is y
    with torch.no_grad():
        assert m._tied(y, "f", "its gradient is g", x, w) is y
    tied = m._tied(y, "f", "its gradient is g", x, w)
    assert tied.data_ptr() == y.data_ptr() and tied.requires_grad and not tied._is_view()
    with pytest.raises(RuntimeError, match="f has no backward pass for autograd: its gradient is g"):
        (tied * 2 + x).sum().backward()
    before = tied.detach().clone()
    tied += 1                      # written in place, with a graph and without one
    with torch.no_grad():
        tied.mul_(2)
    assert torch.equal(tied.detach(), (before + 1) * 2)
    with pytest.raises(RuntimeError, match="f has no backward pass"):
        tied.sum().backward()


@pytest.mark.gpu
def test_a_backward_pass_through_an_operator_is_refused(moelib):
    import moe_expert_layer_08_b200 as moe
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=g)

    x, res, gain, gate, w = normal(6, 64), normal(6, 64), normal(64), normal(64), normal(2, 40, 64)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    codes, sf = moe.quantize_fp4(normal(32, 64))
    calls = {
        "grouped_matmul": ((x, w), lambda x, w: moe.grouped_matmul(x, w, off)),
        "fp4_matvec": ((x,), lambda x: moe.fp4_matvec(x, codes, sf)),
        "norm_before": ((x, gain), lambda x, gain: moe.norm_before(x, gain, fp8=True).y),
        "norm_after": ((x, res, gain, gate), lambda x, r, gain, gate: moe.norm_after(x, r, gain, gate=gate).out),
    }
    for name, (inputs, call) in calls.items():
        want = call(*inputs)
        assert not want.requires_grad
        for i in range(len(inputs)):
            leaves = [t.clone().requires_grad_(i == j) for j, t in enumerate(inputs)]
            y = call(*leaves)
            assert torch.equal(y.detach(), want)
            with pytest.raises(RuntimeError, match=name + " has no backward pass"):
                y.mul_(2).float().sum().backward()
            with torch.no_grad():
                assert not call(*leaves).requires_grad
    # a given output stays the caller's, and the gradients' own calls give plain tensors
    leaf = x.clone().requires_grad_()
    out = torch.empty_like(x)
    assert moe.norm_after(leaf, res, gain, out=out).out is out and not out.requires_grad
    y = torch.empty((6, 40), dtype=torch.bfloat16, device="cuda")
    assert moe.grouped_matmul(leaf, w, off, out=y) is y and not y.requires_grad
    n = moe.norm_before(leaf, gain, rstd=True)
    dx, dgain = moe.norm_before_backward(x, leaf, gain, n.rstd)
    assert not dx.requires_grad and not dgain.requires_grad
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert moe.norm_before(leaf, gain, stream=s).y.requires_grad
    torch.cuda.synchronize()
