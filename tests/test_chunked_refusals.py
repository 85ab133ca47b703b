"""A refused first chunk leaves a ChunkedAttention as it was (CPU only: the operators refuse tensors that are not on a GPU)."""

import pytest
import torch

from temporal_block_sparse_b200.attention import AxisRope, ChunkedAttention


def test_a_refused_first_chunk_does_not_fix_the_shapes():
    attn = ChunkedAttention(AxisRope((24, 20, 20), (4, 2, 2)), frames=2, frame_tokens=4)
    for B, Hk in ((1, 2), (3, 2), (3, 1)):
        q, k = (torch.zeros(B, 4, h, 64, dtype=torch.bfloat16) for h in (2, Hk))
        with pytest.raises(ValueError, match="CUDA"):  # and not that something must stay as in the first chunk
            attn(q, k, k)
        assert attn.cached_frames == 0
    hist = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    attn.set_history(hist, hist)  # still before the first chunk
