"""The 4-bit product on the tensor cores (K = 7168, whose rows go there whatever
their number) on two streams at once, a graph among them, and first used inside a
capture."""
import os
import subprocess
import sys

import pytest
import torch

from test_gpu_matvec import random_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe(moelib):
    import moe_expert_layer_08_b200 as m
    return m


@pytest.mark.parametrize("fmt,T", [("mx", 8), ("nvfp4", 4)])
def test_two_streams_and_a_graph(moe, fmt, T):
    x, w, sf = random_case(T, 9000, 7168, fmt, 1)
    inputs = [x, (x * 3).contiguous()]
    expect = [moe.fp4_matvec(v, w, sf, fmt=fmt) for v in inputs]
    out = torch.empty_like(expect[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.fp4_matvec(inputs[0], w, sf, fmt=fmt, out=out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(moe.fp4_matvec(inputs[i], w, sf, fmt=fmt))
        graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, expect[i]) for y in got[i])
    assert torch.equal(out, expect[0])
    del graph


FIRST = """
import torch
import moe_expert_layer_08_b200 as moe
torch.manual_seed(0)
x = torch.randn((8, 7168), dtype=torch.bfloat16, device="cuda")
codes = torch.randint(0, 256, (9000, 3584), dtype=torch.uint8, device="cuda")
scales = torch.randint(120, 130, (9000, 224), dtype=torch.uint8, device="cuda")
y = torch.empty((8, 9000), dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.fp4_matvec(x, codes, scales, out=y)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, moe.fp4_matvec(x, codes, scales))
del graph
print("same")
"""


def test_first_call_inside_a_capture(moelib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip() == "same", done.stderr[-2000:]
