"""A process's first calls may be captured into a graph: what the library sets up on the way (kernels loaded,
attributes, the status word) is no part of a capture and does not end it."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
import torch
from warp_specialized_tma_gb300 import ffn

bf = torch.bfloat16
gen = torch.Generator().manual_seed(0)
ints = lambda *s: torch.randint(-1, 2, s, generator=gen).to(bf).cuda()
M = int(sys.argv[1])
x, dy = ints(M, 520), ints(M, 264)
wg, wu, wd = ints(1000, 520), ints(1000, 520), ints(264, 1000)
b = ints(264)


def run():
    h, saved = ffn.gated(x, wg, wu, "relu", save=sys.argv[2])
    y, z = ffn.linear(h, wd, b, "relu", dy, save=True)
    y32 = ffn.linear(x, wg, out_dtype=torch.float32)
    first = ffn.linear_backward(dy, h, wd, z, "relu", bias=True, grad_dtype=torch.float32)
    return (h, y, z, y32) + first + ffn.gated_backward(dy, x, saved, wg, wu, wd, "relu")


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
want = run()
torch.cuda.synchronize()
assert all(a.equal(b) for a, b in zip(got, want)), [a.equal(b) for a, b in zip(got, want)]
assert ffn.device_status() == (ffn.OK, 0)
print("captured")
"""


@pytest.mark.parametrize("save", ["bf16", "e4m3"])
@pytest.mark.parametrize("M", [1, 12, 200, 5000])
def test_a_first_call_may_be_captured(M, save):
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    run = subprocess.run([sys.executable, "-c", PROGRAM, str(M), save], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.endswith("captured\n"), run.stdout + run.stderr
