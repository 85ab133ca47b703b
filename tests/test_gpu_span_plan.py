"""How lite_attn_span and lite_attn_prefix split their work, as far as a caller can tell (needs a B200).

Split calls take scratch from the library's pool, unsplit ones with an item a CTA or less take none, so a process's first
call shows which it was.
"""

import os
import subprocess
import sys

import pytest
import torch

from oracle import span as ref
from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import spans as sp
from test_gpu_span import check, f64, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST_CALL = """
import sys
sys.path.insert(0, %r)
import torch
from temporal_block_sparse_b200 import lite_attn as la
B, Nq, Nk, H, d = %r
q = torch.randn(B, Nq, H, d, device="cuda").to(torch.bfloat16)
kv = torch.randn(1, Nk, H, d, device="cuda").to(torch.bfloat16).expand(B, -1, -1, -1)
la.lite_attn_span(q, kv, kv)
torch.cuda.synchronize()
print("held", la.scratch_pool_bytes())
"""


@pytest.mark.parametrize("B,Nq,Nk,H,d,split", [
    # 33 .. 128 rows: unsplit, one softmax group does all key tiles; split, both do. Items for nearly all SMs
    (8, 64, 32768, 18, 128, True),
    (1, 100, 8192, 148, 64, True),
    (2, 64, 512, 40, 128, False),  # few key tiles: a join costs more than it saves
])
def test_a_single_query_tile_is_split_where_both_groups_save_time(B, Nq, Nk, H, d, split):
    done = subprocess.run([sys.executable, "-c", FIRST_CALL % (ROOT, (B, Nq, Nk, H, d))], capture_output=True, text=True,
                          timeout=300, cwd=ROOT)
    assert done.returncode == 0, done.stdout + done.stderr[-2000:]
    held = int(done.stdout.split("held")[1])
    assert (held > 0) == split, held


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,G", [(33, 1), (64, 1), (128, 1), (7, 5), (129, 1)])
def test_rows_of_one_tile_split_and_unsplit(d, Nq, G):
    Hk = 2
    for Nk in (100, 2500):
        q, k, v = make(Nq, (2, Nq, Hk * G, d), (2, Nk, Hk, d), (2, Nk, Hk, d))
        spans = sp.padded_spans([Nk, Nk // 2 + 1], Nq, causal=True)
        check(la.lite_attn_span(q, k, v, spans), ref.span_attention(f64(q), f64(k), f64(v), f64(spans)))
