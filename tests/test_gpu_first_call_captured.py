"""The first call of a process inside a stream capture: what a kernel's launch looks up once does not disturb it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import combine_topk_ids_histogram_gb300 as ep
bf = torch.bfloat16
L = ep.dispatch_layout(torch.arange(64, dtype=torch.int32, device="cuda").view(-1, 1) % 2, 2)
x, w, g = (torch.randn(*s, device="cuda").to(bf) for s in ((64, 128), (2, 96, 128), (64, 96)))
a, b = (torch.randn(*s, device="cuda").to(bf) for s in ((2, 16, 128), (2, 128, 16)))
def step():
    return (ep.expert_linear(x, w, L), *ep.expert_linear(x, w, L, swiglu=True, save=True), *ep.expert_linear_bwd(g, x, w, L),
            ep.lora_add(x, x, a, b, L))
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
assert all(torch.equal(p, q) for p, q in zip(held, step())) and ep.read_status(L) == 0
print("same")
"""


def test_first_call_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
