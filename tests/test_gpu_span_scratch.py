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
