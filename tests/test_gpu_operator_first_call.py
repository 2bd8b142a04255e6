"""The first call of a process inside a graph capture: kernels are loaded, their
limits raised and the error word looked up while a capture is under way."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
import torch
import context_attention_partial_gb300 as cp
what, dtype = sys.argv[1], {"bf16": torch.bfloat16, "f32": torch.float32}[sys.argv[2]]
g = torch.Generator("cpu").manual_seed(1)
M, N = {"rotary": (50, 50), "few": (2, 9000), "rows": (300, 200), "parts": (100, 9000)}[what]
q, k, v, dout = (torch.randn(1, 4, s, 64, generator=g).to(dtype).cuda() for s in (M, N, N, M))
pos = torch.arange(M, dtype=torch.float32, device="cuda")[:, None]

def step():
    if what == "rotary":
        return [cp.rotary(q, pos, (64,)), cp.rotary(q, pos, (64,), interleaved=False)]
    out, lse = cp.cross_attention(q, k, v)
    return [out, lse, *cp.cross_attention_backward(q, k, v, out, lse, dout)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert cp.last_device_status() == 0
"""


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["rotary", "few", "rows", "parts"])
def test_first_call_in_a_capture(what, dtype):
    p = subprocess.run([sys.executable, "-c", PROGRAM, what, dtype], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, p.stderr[-2000:]
