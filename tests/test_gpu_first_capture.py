"""The first call that a process makes of an entry point may be a captured one: what the library sets up
for good then (its pool, its modules) is not part of the capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
import gated_delta_rule_linear_gb300 as la

H, d, lens = 16, 64, [200] * 40
N = sum(lens)
q, k, v, e = (torch.randn(N, H, d, device="cuda", dtype=torch.bfloat16) * d ** -0.5 for _ in range(4))
c = torch.arange(0, N + 1, 200, dtype=torch.int32, device="cuda")
g, w = torch.full((H,), -0.1, device="cuda"), torch.ones(d, device="cuda")
dense = [t.view(1, N, H, d).transpose(1, 2).contiguous() for t in (q, k, v)]
call = {
    "packed_fwd": lambda: la.packed_fwd(q, k, v, c, "retnet", g=g),
    "packed_bwd": lambda: la.packed_bwd(q, k, v, e, c, "retnet", g=g),
    "epilogue_bwd": lambda: tuple(la.epilogue_bwd(q, k, w=w, gate=v).values()),
    "chunk_fwd": lambda: la.chunk_fwd(*dense, "retnet", g=g),
}["NAME"]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
want = call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)
assert la.la_stream_status(torch.cuda.current_stream().cuda_stream) == 0
"""


@pytest.mark.parametrize("name", ["packed_fwd", "packed_bwd", "epilogue_bwd", "chunk_fwd"])
def test_first_call_is_captured(name):
    r = subprocess.run([sys.executable, "-c", CODE.replace("NAME", name)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
