"""lite_attn_span and lite_attn_prefix against the 64-bit oracle (needs a B200).

Bound of an output element: P is rounded to bf16 once (at most 2^-8 of each weight, so 2^-8 of the
weighted |v|), the output once (2^-8 of itself). The 32-bit part: a score is a sum of d exact products,
off by at most d 2^-24 sum |q k| scale, below 2e-4 for these inputs, plus a few 2^-23 of its size
for the cap, the bias and the exponent; twice that, relative, in a weight (its own and the row
sum's): 1e-3 of the weighted |v| covers it. lse: the score's error, 4e-4 + 2^-20 |score|.
"""

import numpy as np
import pytest
import torch

from oracle import span as ref
from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import spans as sp

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(autouse=True)
def _clean_state():
    la.load()
    yield
    assert la.lite_get_device_status() == 0


def make(seed, *shapes, gain=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * gain).to(torch.bfloat16) for s in shapes]


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(got, want, big=0.0):
    o, lse = got
    ro, rl, rw = want
    err = np.abs(f64(o) - ro)
    lim = (2.0 ** -8 + 1e-3) * rw + 2.0 ** -8 * np.abs(ro) + 1e-30
    assert (err <= lim).all(), (float((err / lim).max()), np.argwhere(err > lim)[:4])
    if lse is not None:
        a = f64(lse)
        assert (np.isneginf(a) == np.isneginf(rl)).all()
        fine = ~np.isneginf(rl)
        if fine.any():
            assert np.abs(a[fine] - rl[fine]).max() <= 4e-4 + 2.0 ** -20 * max(big, np.abs(rl[fine]).max())


def span_case(B, Nq, Nk, H, Hk, d, spans, seed=0, **kw):
    q, k, v = make(seed, (B, Nq, H, d), (B, Nk, Hk, d), (B, Nk, Hk, d))
    got = la.lite_attn_span(q, k, v, spans, **kw)
    rk = {x: (f64(y) if isinstance(y, torch.Tensor) else y) for x, y in kw.items() if x not in ("return_lse", "stream")}
    check(got, ref.span_attention(f64(q), f64(k), f64(v), f64(spans) if spans is not None else None, **rk))
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 128, 129, 255, 257, 400])
def test_all_keys_and_causal_at_tile_edges(d, N):
    span_case(1, N, N, 2, 2, d, None, seed=N)
    span_case(2, N, N, 2, 1, d, sp.prefix_spans(N, 0), seed=N + 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (7.0, False), (0.0, True), (20.0, True)])
def test_masks_with_cap_and_bias(d, cap, bias):
    N = 333
    slopes = torch.tensor([0.5, 0.03], device="cuda") if bias else None
    for spans in (sp.document_spans([100, 1, 131, 0, 101]), sp.prefix_spans(N, 70), sp.frame_spans(9, 37),
                  sp.frame_spans(9, 37, window=2), sp.document_spans([200, 133], causal=True)):
        span_case(1, N, N, 2, 2, d, spans, seed=5, cap=cap, slopes=slopes)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_keys_and_spans_outside_the_keys(d):
    N = 200
    spans = torch.zeros(2, N, 2, dtype=torch.int32)
    spans[0, :, 1] = N
    spans[0, 5:150] = torch.tensor([7, 7])
    spans[0, 160] = torch.tensor([-100, 3])
    spans[0, 161] = torch.tensor([190, 2 ** 31 - 1])
    spans[0, 162] = torch.tensor([2 ** 31 - 1, -2 ** 31])
    spans[0, 163] = torch.tensor([199, 200])
    spans[1, :] = torch.tensor([50, 40])  # a batch entry that sees nothing
    o, lse = span_case(2, N, N, 3, 3, d, spans.cuda(), seed=3)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("H,Hk", [(4, 2), (5, 1), (6, 2), (12, 1), (128, 1), (40, 8)])
@pytest.mark.parametrize("Nq", [1, 3, 45])
def test_grouped_heads(H, Hk, Nq):
    Nk = 150
    spans = sp.padded_spans([150, 77], Nq, causal=True)
    span_case(2, Nq, Nk, H, Hk, 64, spans, seed=H + Nq)
    slopes = torch.rand(H, device="cuda")
    span_case(2, Nq, Nk, H, Hk, 128, spans, seed=H + Nq, slopes=slopes)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nk", [1, 500, 5000, 20011])
def test_single_tokens_of_a_padded_batch(d, Nk):
    lengths = [Nk, max(1, Nk // 3), 1, 0]
    span_case(4, 1, Nk, 3, 3, d, sp.padded_spans(lengths, 1), seed=Nk)
    span_case(4, 1, Nk, 3, 3, d, sp.padded_spans(lengths, 1), seed=Nk, cap=5.0)


def test_more_items_than_ctas_in_uneven_order():
    # 2 * 9 heads, 60 documents: items of very different lengths handed out one by one
    lengths = [1, 700, 3, 256, 11, 129, 300, 2, 64, 434]
    span_case(2, sum(lengths), sum(lengths), 9, 3, 64, sp.document_spans(lengths), seed=8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Nq,Nk,Np,H,Hk", [
    (1, 1, 1, 1, 1, 1), (3, 1, 5, 1000, 4, 2), (5, 17, 93, 512, 3, 3), (2, 130, 130, 300, 2, 2), (4, 40, 0, 257, 6, 2),
    (3, 9, 70, 0, 2, 1), (16, 1, 64, 4000, 5, 1), (2, 300, 301, 129, 1, 1), (7, 33, 128, 128, 4, 4)])
def test_prefix(d, B, Nq, Nk, Np, H, Hk):
    q, k, v, kp, vp = make(B + Nq, (B, Nq, H, d), (B, Nk, Hk, d), (B, Nk, Hk, d), (Np, Hk, d), (Np, Hk, d))
    for spans in (None, sp.padded_spans([max(0, Nk - 3 * b) for b in range(B)], Nq, causal=True) if Nk else None):
        for kw in ({}, {"cap": 9.0, "slopes": torch.linspace(0.01, 0.4, H, device="cuda")}):
            got = la.lite_attn_prefix(q, kp, vp, k, v, spans, **kw)
            rk = {x: f64(y) if isinstance(y, torch.Tensor) else y for x, y in kw.items()}
            check(got, ref.span_attention(f64(q), f64(k), f64(v), f64(spans), f64(kp), f64(vp), **rk))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 40, 300])
@pytest.mark.parametrize("batches", [1, 2])
def test_given_positions(d, Nq, batches):
    B, Nk, Np, H = 2, 300, 150, 2
    q, k, v, kp, vp = make(Nq, (B, Nq, H, d), (B, Nk, H, d), (B, Nk, H, d), (Np, H, d), (Np, H, d))
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    slopes = torch.tensor([0.3, 0.01], device="cuda")
    qpos = torch.randint(0, 50, (batches, Nq), generator=g, device="cuda").float()  # e.g. frame numbers
    kpos = torch.randint(0, 50, (batches, Nk), generator=g, device="cuda").float()
    ppos = torch.randint(-20, 20, (Np,), generator=g, device="cuda").float() + 0.5
    for some in ({"q_pos": qpos, "k_pos": kpos}, {"k_pos": kpos}, {"q_pos": qpos}):
        for cap in (0.0, 4.0):
            rk = {x: f64(y) for x, y in some.items()}
            got = la.lite_attn_span(q, k, v, slopes=slopes, cap=cap, **some)
            check(got, ref.span_attention(f64(q), f64(k), f64(v), slopes=f64(slopes), cap=cap, **rk))
    spans = sp.padded_spans([Nk, 33], Nq)
    got = la.lite_attn_prefix(q, kp, vp, k, v, spans, slopes=slopes, q_pos=qpos, k_pos=kpos, prefix_pos=ppos)
    check(got, ref.span_attention(f64(q), f64(k), f64(v), f64(spans), f64(kp), f64(vp), slopes=f64(slopes),
                                  q_pos=f64(qpos), k_pos=f64(kpos), prefix_pos=f64(ppos)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [1e-3, 0.5, 3.0, 30.0, 1e6])
def test_caps_from_saturated_to_idle(d, cap):
    # scores reach +-20 here: the smaller caps saturate, the largest change nothing. 32-bit scores of
    # size 20 are good to 20 * 2^-20 after the cap's arithmetic; the bounds of check() hold unchanged.
    q, k, v = make(11, (1, 150, 2, d), (1, 200, 2, d), (1, 200, 2, d), gain=2.2)
    got = la.lite_attn_span(q, k, v, sp.padded_spans([170], 150), cap=cap)
    check(got, ref.span_attention(f64(q), f64(k), f64(v), f64(sp.padded_spans([170], 150)), cap=cap))
