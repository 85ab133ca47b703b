"""Distance bias far from the keys, with steep slopes and at given positions, against the 64-bit oracle (needs a B200).

The bounds are those of test_gpu_span (derived there); they hold at any distance because the bias is kept out of the
32-bit scores: a key's exponent is its score (bound of that file), plus the difference of its bias and the least bias
of the keys seen in its tile (one rounding, 2^-24 of at most 64 for a weight above 2^-64: 4e-6), minus the
reference, which is the same 32-bit number for all keys. Where a tile is seen entirely and has all rows on one
side, the difference is to the reference itself. The slope in log2 units is off by 2^-24 of itself, for the
differences of the keys that matter (below 64 again) 4e-6. Distances of whole positions below 2^24 are
exact.
"""

import numpy as np
import pytest
import torch

from oracle import span as ref
from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import spans as sp
from test_gpu_span import check, f64, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(autouse=True)
def _clean_state():
    la.load()
    yield
    assert la.lite_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 3, 200])
@pytest.mark.parametrize("cap", [0.0, 6.0])
def test_short_sequences_at_the_start_of_a_long_cache(d, Nq, cap):
    # the queries' own positions are at the end of the padded cache, 2^20 keys away from what they see
    Nk, H, lengths = 1 << 20, 2, [90, 700]
    top = max(lengths)
    q, head_k, head_v = make(Nq, (2, Nq, H, d), (2, top, H, d), (2, top, H, d))
    k = torch.zeros((2, Nk, H, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[:, :top], v[:, :top] = head_k, head_v
    slopes = torch.tensor([0.5, 0.031], device="cuda")
    spans = sp.padded_spans(lengths, Nq)
    got = la.lite_attn_span(q, k, v, spans, cap=cap, slopes=slopes)
    check(got, ref.span_attention(f64(q), f64(head_k), f64(head_v), f64(spans), cap=cap, slopes=f64(slopes),
                                  q_pos=np.arange(Nk - Nq, Nk), k_pos=np.arange(top)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [2, 150])
def test_prefix_far_behind(d, Nq):
    # a prefix that ends inside a tile, 2^20 positions back; some rows see their own last keys too
    Nk, Np, H, tail = 1 << 20, 300, 2, 40
    q, kp, vp, tail_k, tail_v = make(Nq, (1, Nq, H, d), (Np, H, d), (Np, H, d), (1, tail, H, d), (1, tail, H, d))
    k = torch.zeros((1, Nk, H, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[:, -tail:], v[:, -tail:] = tail_k, tail_v
    slopes = torch.tensor([0.25, 1e-5], device="cuda")  # the second head sees both
    spans = torch.zeros(Nq, 2, dtype=torch.int32)
    spans[::2, 0], spans[::2, 1] = Nk - tail + 3, Nk
    spans = spans.cuda()
    got = la.lite_attn_prefix(q, kp, vp, k, v, spans, slopes=slopes)
    near = np.maximum(f64(spans) - (Nk - tail), 0)
    check(got, ref.span_attention(f64(q), f64(tail_k), f64(tail_v), near, f64(kp), f64(vp), slopes=f64(slopes),
                                  q_pos=np.arange(Np + Nk - Nq, Np + Nk), k_pos=np.arange(Np + Nk - tail, Np + Nk)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_given_positions_far_away_in_any_order(d, Nq, sign):
    B, Nk, H = 2, 400, 2
    q, k, v = make(Nq + d, (B, Nq, H, d), (B, Nk, H, d), (B, Nk, H, d))
    g = torch.Generator(device="cuda")
    g.manual_seed(Nq)
    # three clusters of keys, mixed within every tile; rows before, between and after them
    place = torch.tensor([2.0e6, 9.0e6, 9.1e6], device="cuda")
    k_pos = place[torch.randint(0, 3, (B, Nk), generator=g, device="cuda")] + torch.randint(0, 30, (B, Nk), generator=g, device="cuda")
    q_pos = torch.tensor([0.0, 1.0e6, 5.0e6, 9.05e6, 1.6e7], device="cuda")[torch.randint(0, 5, (B, Nq), generator=g, device="cuda")]
    slopes = sign * torch.tensor([0.5, 0.07], device="cuda")
    for spans in (None, sp.padded_spans([Nk, 37], Nq)):
        got = la.lite_attn_span(q, k, v, spans, slopes=slopes, q_pos=q_pos, k_pos=k_pos)
        check(got, ref.span_attention(f64(q), f64(k), f64(v), f64(spans), slopes=f64(slopes), q_pos=f64(q_pos),
                                      k_pos=f64(k_pos)))
    # queries far from keys at their default positions, before and after them
    far = torch.where(q_pos > 4e6, 1.0e8, -6.0e7)
    for spans in (None, sp.padded_spans([Nk, 37], Nq)):
        got = la.lite_attn_span(q, k, v, spans, slopes=slopes * 0.5, q_pos=far)
        check(got, ref.span_attention(f64(q), f64(k), f64(v), f64(spans), slopes=f64(slopes * 0.5), q_pos=f64(far)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 11.0])
def test_slopes_on_both_sides_of_the_short_way(d, cap):
    # 1.3 a token (0.65 with a cap) is where a tile's bias spreads too far for the short way
    N = 300
    slopes = torch.tensor([0.6, 0.7, 1.29, 1.31, 5.0, 1000.0, -0.5, -2.0], device="cuda")
    H = slopes.numel()
    q, k, v = make(d, (1, N, H, d), (1, N, H, d), (1, N, H, d))
    for spans in (None, sp.prefix_spans(N, 0), sp.document_spans([100, 33, 167])):
        got = la.lite_attn_span(q, k, v, spans, cap=cap, slopes=slopes)
        check(got, ref.span_attention(f64(q), f64(k), f64(v), f64(spans), cap=cap, slopes=f64(slopes)))
        one = None if spans is None else spans[-2:-1]
        got = la.lite_attn_span(q[:, -2:-1], k, v, one, cap=cap, slopes=slopes, q_pos=torch.full((1,), N - 2.0, device="cuda"))
        check(got, ref.span_attention(f64(q[:, -2:-1]), f64(k), f64(v), None if one is None else f64(one), cap=cap,
                                      slopes=f64(slopes), q_pos=np.full(1, N - 2.0)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 70])
@pytest.mark.parametrize("at", [1e9, -3e9, 1e14, 1e30])
def test_positions_past_the_exact_range_stay_finite(d, Nq, at):
    # distances are 32-bit numbers: what remains of the order of keys is theirs, but every row is an average of values
    q, k, v = make(Nq, (1, Nq, 2, d), (1, 300, 2, d), (1, 300, 2, d))
    slopes = torch.tensor([0.5, 1.2], device="cuda")
    pos = torch.full((Nq,), at, device="cuda")
    for spans in (None, sp.padded_spans([200], Nq)):
        for kw in ({}, {"cap": 3.0}, {"k_pos": torch.arange(300, device="cuda").float()}):
            o, lse = la.lite_attn_span(q, k, v, spans, slopes=slopes, q_pos=pos, **kw)
            assert torch.isfinite(lse).all() and torch.isfinite(o).all()
            assert (o.float().abs() <= v.float().abs().max() * (1 + 2.0 ** -7)).all() and (o != 0).any()
