"""The first call that a process makes of a serving entry point may be a captured one."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
import gated_delta_rule_linear_gb300 as la

dev, i32 = "cuda", torch.int32
q, k = torch.randn(6, 8, 64, device=dev, dtype=torch.bfloat16), torch.randn(6, 2, 64, device=dev, dtype=torch.bfloat16)
kc, vc = (torch.randn(6 * 64, 16, 2, 64, device=dev, dtype=torch.bfloat16) for _ in range(2))
table = torch.randperm(6 * 64, device=dev).to(i32).reshape(6, 64)
lens = torch.tensor([1, 900, 30, 0, 512, 77], device=dev, dtype=i32)
freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device=dev) / 32)
logits, scores = torch.randn(2, 3, 5001, device=dev), torch.randn(2, 3, device=dev)
parent = torch.tensor([[1, 0, 2], [2, 2, 2]], device=dev, dtype=i32)
pool = torch.randn(6, 4, 64, 64, device=dev)
call = {
    "cache_append": lambda: (la.cache_append(q, k, k, kc, vc, table, lens, freq=freq), kc, vc),
    "paged_attn": lambda: la.paged_attn(q, kc, vc, table, lens, with_lse=True),
    "beam_select": lambda: la.beam_select(logits, scores, 4),
    "beam_states": lambda: (la.beam_states(pool, torch.zeros_like(parent)),),
    "beam_cache": lambda: la.beam_cache(kc, vc, table, lens, torch.zeros_like(parent)),
}["NAME"]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = call()  # (with every parent 0, and for the same tokens, once more changes nothing)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
"""


@pytest.mark.parametrize("name", ["cache_append", "paged_attn", "beam_select", "beam_states", "beam_cache"])
def test_first_call_is_captured(name):
    r = subprocess.run([sys.executable, "-c", CODE.replace("NAME", name)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
