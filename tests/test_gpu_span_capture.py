"""A process's first call of each operator inside a stream capture (needs a B200)."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.path.insert(0, %r)
import torch
from temporal_block_sparse_b200 import lite_attn as la
which = sys.argv[1]
g = torch.Generator(device="cuda").manual_seed(1)
new = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
plan = la.RopePlan((44, 42, 42))
if which == "rope":
    q, k = new(1, 300, 100, 128), new(1, 300, 4, 128)
    outs = torch.zeros_like(q), torch.zeros_like(k)
    call = lambda out: la.lite_qk_rope(q, k, plan, grid=(3, 10, 10), q_out=out[0], k_out=out[1])
elif which == "fwd":
    q, k, v = new(1, 300, 4, 128), new(1, 300, 4, 128), new(1, 300, 4, 128)
    masks = la.new_mask(1, 4, 300, 128), la.new_mask(1, 4, 300, 128)
    outs = torch.zeros_like(q), torch.zeros(1, 4, 300, device="cuda")
    call = lambda out: la.lite_attn_fwd(q, k, v, *masks, tau=-3.0, o=out[0], lse=out[1])
else:
    q, k, v = new(2, 1, 4, 128), new(2, 5000, 4, 128), new(2, 5000, 4, 128)
    outs = torch.zeros_like(q), torch.zeros(2, 4, 1, device="cuda")
    if which == "span":
        call = lambda out: la.lite_attn_span(q, k, v, o=out[0], lse=out[1])
    else:
        call = lambda out: la.lite_attn_prefix(q, k[0], v[0], k, v, o=out[0], lse=out[1])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call(outs)
graph.replay()
torch.cuda.synchronize()
eager = [torch.zeros_like(x) for x in outs]
call(eager)
torch.cuda.synchronize()
assert all(torch.equal(a, b) and a.float().abs().sum() > 0 for a, b in zip(outs, eager))
assert la.lite_get_device_status() == 0
"""


@pytest.mark.parametrize("which", ["rope", "span", "prefix", "fwd"])
def test_first_call_of_a_process_in_a_capture(which):
    done = subprocess.run([sys.executable, "-c", PROGRAM % ROOT, which], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert done.returncode == 0, done.stdout + done.stderr[-2000:]
