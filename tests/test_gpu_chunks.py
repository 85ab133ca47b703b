"""AxisRope, LiteAttention(rope=...) and ChunkedAttention on the GPU against the 64-bit oracle (needs a B200).

The chunked run goes through all three operators together: norm and rotation of the chunk at its place in the
stream, k into the cache, attention over shared history, cache and chunk. q and k of the oracle are the
oracle's own rotation rounded to bf16 as the operator rounds it; where that rounding falls the other way
(a value within 2^-18 of a tie) a score moves by at most 2^-8 of one product, which the bound of
test_gpu_span.check holds (see there) with the 2^-8 of P counted once more.
"""

import numpy as np
import pytest
import torch

from oracle import span as ref
from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import workload as wl
from temporal_block_sparse_b200.attention import AxisRope, ChunkedAttention, LiteAttention

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(autouse=True)
def _clean_state():
    la.load()
    yield
    assert la.lite_get_device_status() == 0


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def bf16(a):
    return torch.from_numpy(a).to(torch.bfloat16).double().numpy()


def check(o, want):
    ro, _, rw = want
    err = np.abs(f64(o) - ro)
    lim = (2.0 ** -7 + 1e-3) * rw + 2.0 ** -8 * np.abs(ro) + 1e-30
    assert (err <= lim).all(), float((err / lim).max())


def layer(H, Hk, d, grid, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    wq, wk = (1 + 0.2 * torch.randn(n, generator=g, device="cuda") for n in (H * d, Hk * d))
    return AxisRope(wl.axis_split(d), grid, q_weight=wq, k_weight=wk, eps=1e-5), g


def turned(rope, x, weight, start):
    N = x.shape[1]
    at = np.broadcast_to(ref.grid_positions(rope.grid, start, N), (x.shape[0], 3, N))
    return bf16(ref.rope(f64(x), at, rope.plan.freq, rope.plan.axis, rope.plan.pairing, f64(weight), rope.eps))


@pytest.mark.parametrize("d,H,Hk", [(64, 2, 2), (128, 4, 2)])
@pytest.mark.parametrize("history,window", [(0, None), (2, None), (2, 2)])
def test_chunked_generation(d, H, Hk, history, window):
    rows, cols, B = 3, 7, 2
    ft = rows * cols
    rope, g = layer(H, Hk, d, (50, rows, cols), d + history)
    slopes = torch.linspace(0.001, 0.01, H, device="cuda")
    attn = ChunkedAttention(rope, frames=6, frame_tokens=ft, window=window, cap=20.0, slopes=slopes)
    hk = hv = None
    if history:
        raw = torch.randn(1, history * ft, H + 2 * Hk, d, generator=g, device="cuda").to(torch.bfloat16)
        hk = rope(raw[:, :, :H], raw[:, :, H : H + Hk])[1][0]
        hv = raw[0, :, H + Hk :].contiguous()
        attn.set_history(hk, hv)
    keys, values = [], []
    for n in (1, 3, 1):
        done = attn.cached_frames
        qkv = torch.randn(B, n * ft, H + 2 * Hk, d, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = qkv[:, :, :H], qkv[:, :, H : H + Hk], qkv[:, :, H + Hk :]
        o, lse = attn(q, k, v, return_softmax_lse=True)
        start = (history + done) * ft
        keys.append(turned(rope, k, rope.k_weight, start))
        values.append(f64(v))
        frame = np.arange(n * ft) // ft + done
        first = np.zeros_like(frame) if window is None else np.maximum(frame + 1 - window, 0)
        spans = np.stack([first * ft, (frame + 1) * ft], -1)
        check(o, ref.span_attention(turned(rope, q, rope.q_weight, start), np.concatenate(keys, 1),
                                    np.concatenate(values, 1), spans, f64(hk), f64(hv), cap=20.0, slopes=f64(slopes)))
        assert attn.cached_frames == done + n and lse.shape == (B, H, n * ft)
    with pytest.raises(ValueError):
        attn(qkv[:, :, :H].repeat(1, 2, 1, 1), qkv[:, :, :Hk].repeat(1, 2, 1, 1), qkv[:, :, :Hk].repeat(1, 2, 1, 1))
    attn.reset()
    assert attn.cached_frames == 0


def test_lite_attention_with_rope_equals_rotating_first():
    w = wl.small_workload(1, 3, 4, 8, 16, 128, steps=2, locality=4.0, tau=-2.0, seed_offset=300)
    rope, g = layer(3, 3, 128, (4, 8, 16), 1)
    with_rope, plain = LiteAttention(threshold=-2.0, rope=rope), LiteAttention(threshold=-2.0)
    for _ in range(w.steps):
        q, k, v = (torch.randn(1, w.N, 3, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
        a = with_rope(q, k, v)
        b = plain(*rope(q, k), v)
        assert torch.equal(a, b)
    check(LiteAttention(enable_skipping=False, rope=rope)(q, k, v),
          ref.span_attention(turned(rope, q, rope.q_weight, 0), turned(rope, k, rope.k_weight, 0), f64(v)))
