"""Scratch of split span and prefix calls: the pool stays within the gigabyte that lite_attn.h names (needs a B200)."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A process of its own, whose pool holds nothing yet: hundreds of variants drawn from one history, one token each.
PROGRAM = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np
import torch
from oracle import span as ref
from temporal_block_sparse_b200 import lite_attn as la
from test_gpu_span import check, f64, make

B, H, d, Np, Nk = 512, 40, 128, 32760, 64
q, k, v, kp, vp = make(1, (B, 1, H, d), (B, Nk, H, d), (B, Nk, H, d), (Np, H, d), (Np, H, d))
before = la.scratch_pool_bytes()
o, lse = la.lite_attn_prefix(q, kp, vp, k, v)
torch.cuda.synchronize()
held = la.scratch_pool_bytes()
print(before, held)
assert before == 0 and 0 < held <= (1 << 30) + (32 << 20), held
few = [0, 1, 300, B - 1]
check((o[few][:, :, 5:7], lse[few][:, 5:7]),
      ref.span_attention(*(f64(x[few][:, :, 5:7]) for x in (q, k, v)), None, f64(kp[:, 5:7]), f64(vp[:, 5:7])))
assert la.lite_get_device_status() == 0
"""


def test_many_variants_of_one_token_stay_within_a_gigabyte():
    program = PROGRAM % (ROOT, os.path.join(ROOT, "tests"))
    done = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert done.returncode == 0, done.stdout + done.stderr[-2000:]


# The scratch of a split call does not fit beside what the program holds: the call says so, and the calls after it, which
# need none, are not blamed for it.
NO_ROOM = """
import sys
sys.path[:0] = [%r, %r]
import torch
from temporal_block_sparse_b200 import lite_attn as la
from test_gpu_span import make

B, H, d, Np, Nk = 512, 40, 128, 32760, 64
q, k, v, kp, vp = make(1, (B, 1, H, d), (B, Nk, H, d), (B, Nk, H, d), (Np, H, d), (Np, H, d))
plan = la.RopePlan((44, 42, 42))
few = q[:4].contiguous(), k[:4].contiguous()
small = lambda: (la.lite_attn_span(q[:1], k[:1], v[:1]), la.lite_attn_dense(k[:1], k[:1], v[:1]),
                 la.lite_qk_rope(*few[:1], None, plan, grid=(4, 1, 1)))
want = small()
torch.cuda.synchronize()
torch.cuda.empty_cache()
outs = torch.empty(B, 1, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, 1, device="cuda")
room = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
free, _ = torch.cuda.mem_get_info()
hold = torch.empty(max(0, free - (200 << 20)), dtype=torch.uint8, device="cuda")
del room  # what the small calls' outputs take, in torch's own cache
for _ in range(2):
    try:
        la.lite_attn_prefix(q, kp, vp, k, v, o=outs[0], lse=outs[1])
        raise SystemExit("the scratch found room: nothing was tested")
    except la.LiteAttnError as e:
        assert e.status == la.LITE_ERR_CUDA, e
    got = small()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(x is y or torch.equal(x, y) for x, y in zip(a, b))
del hold
torch.cuda.empty_cache()
la.lite_attn_prefix(q, kp, vp, k, v, o=outs[0], lse=outs[1])
torch.cuda.synchronize()
assert torch.isfinite(outs[1]).all() and la.lite_get_device_status() == 0
"""


def test_a_call_without_room_for_its_scratch_fails_alone():
    program = NO_ROOM % (ROOT, os.path.join(ROOT, "tests"))
    done = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert done.returncode == 0, done.stdout + done.stderr[-2000:]
