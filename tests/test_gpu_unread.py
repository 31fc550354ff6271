"""Grouped products without a workspace share memory with nobody: what they write
beside their outputs reaches no tensor, whichever stream or graph the process's
first such call is on (each case in a process of its own)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HEAD = """
import torch
import moe_expert_layer_08_b200 as moe
torch.manual_seed(0)
B, U8 = torch.bfloat16, torch.uint8
x, dy = torch.randn((16, 64), dtype=B, device="cuda"), torch.randn((16, 40), dtype=B, device="cuda")
w = torch.randn((2, 40, 64), dtype=B, device="cuda")
off = torch.tensor([0, 7, 16], dtype=torch.int32, device="cuda")
none = torch.zeros(3, dtype=torch.int32, device="cuda")
want = torch.cat([x[:7].double() @ w[0].double().T, x[7:].double() @ w[1].double().T])

def calls():
    moe.grouped_matmul_grad_input(dy, w, off)
    moe.grouped_matmul_grad_weight(dy[:0], x[:0], none)
    return moe.grouped_matmul(x, w, off)

size = torch.cat([x[:7].abs().double() @ w[0].abs().double().T, x[7:].abs().double() @ w[1].abs().double().T])

def right(y):  # one rounding to bf16, 64 additions in fp32 at 2^-23 each (and the sum's rounding)
    return bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 66 * 2.0 ** -23 * size).all())
"""

STREAMS = HEAD + """
a, b = torch.cuda.Stream(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.stream(a):
    kept = [torch.empty(n, dtype=U8, device="cuda") for n in (512, 1024, 2048)]
    early = [torch.full_like(k, 0x5A) for k in kept]
    torch.cuda._sleep(400_000_000)
    for k, e in zip(kept, early):
        k.copy_(e)
    del early, e
    first = calls()
with torch.cuda.stream(b):
    second = calls()
torch.cuda.synchronize()
assert all(bool((k == 0x5A).all()) for k in kept)
assert right(first) and torch.equal(first, second)
print("same")
"""

GRAPH = HEAD + """
kept = [torch.empty(n, dtype=U8, device="cuda") for n in (512, 1024, 2048)]
b = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    early = [torch.full_like(k, 0x5A) for k in kept]
    torch.cuda._sleep(20_000_000)
    for k, e in zip(kept, early):
        k.copy_(e)
    del early, e
    first = calls()
for _ in range(3):
    for k in kept:
        k.zero_()
    graph.replay()
    with torch.cuda.stream(b):
        second = [calls() for _ in range(20)][-1]
    torch.cuda.synchronize()
    assert all(bool((k == 0x5A).all()) for k in kept)
    assert right(first) and torch.equal(first, second)
del graph
print("same")
"""


@pytest.mark.parametrize("script", [STREAMS, GRAPH], ids=["streams", "graph"])
def test_calls_without_a_workspace_reach_no_tensor(moelib, script):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip() == "same", done.stderr[-2000:]
