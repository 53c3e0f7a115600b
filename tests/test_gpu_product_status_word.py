"""All products report in one word of the device: reading it takes one kernel, and a 4-bit product may be the first
call of a process inside a graph's capture (the word's address is asked for then)."""
import os
import subprocess
import sys

import pytest
import torch
from torch.profiler import ProfilerActivity, profile

import combine_ep_route_gb300 as ep
from tests.test_gpu_w4 import built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

FIRST = """
import sys, torch
import combine_ep_route_gb300 as ep
rows, k, n = int(sys.argv[1]), 512, 256
x = torch.ones(rows, k, device="cuda", dtype=torch.bfloat16)
codes = torch.full((n, k // 2), 0x21, device="cuda", dtype=torch.uint8)
scales = torch.full((k // 32, n), 0.5, device="cuda", dtype=torch.bfloat16)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = ep.linear_w4(x, codes, scales)
graph.replay()
ep.check_products()
assert (y == k * 0.75).all()     # fields of 1 and 2 by turns, times 0.5
"""


def kernels(call):
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [e.key for e in p.key_averages() for _ in range(e.count)]


def test_one_kernel_reads_the_status():
    x = torch.ones(4, device="cuda")
    kernels(lambda: x + 1)                      # (the profiler's first use may record nothing)
    names = kernels(lambda: (x + 1, ep.check_products()))
    if not any("elementwise" in n for n in names):
        pytest.skip("the profiler sees no launches here")
    assert sum("take_status" in n for n in names) == 1


@pytest.mark.parametrize("rows", (1, 64))
def test_a_captured_call_may_be_the_first(rows):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST, str(rows)], cwd=root, check=True, timeout=300)
