"""A chunk of ChunkedAttention captured into a graph (needs a B200): replays repeat it at its place in the cache."""

import pytest
import torch

from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import workload as wl
from temporal_block_sparse_b200.attention import AxisRope, ChunkedAttention

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("history", [False, True])
def test_one_frame_replayed_with_new_inputs(d, history):
    B, H, rows, cols = 2, 3, 4, 9
    ft = rows * cols
    g = torch.Generator(device="cuda").manual_seed(d)
    new = lambda: [torch.randn(B, ft, H, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    hist = [torch.randn(50, H, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    rope = AxisRope(wl.axis_split(d), (20, rows, cols))

    def fresh():
        a = ChunkedAttention(rope, frames=4, frame_tokens=ft)
        if history:
            a.set_history(*hist)
        return a

    first, passes, last = new(), [new() for _ in range(3)], new()
    attn = fresh()
    attn(*first)
    held = [x.clone() for x in passes[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = attn(*held)
    assert attn.cached_frames == 2
    for p in passes:
        for x, y in zip(held, p):
            x.copy_(y)
        graph.replay()
        plain = fresh()
        plain(*first)
        assert torch.equal(out, plain(*p))
    # the next frame sees the last pass's keys and values
    assert torch.equal(attn(*last), plain(*last))
    torch.cuda.synchronize()
    assert la.lite_get_device_status() == 0
