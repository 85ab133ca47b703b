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


def check_special(got, want):
    """check() where the oracle's values are finite; the same NaN and infinities elsewhere."""
    o, lse = got
    ro, rl, rw = want
    a = f64(o)
    fine = np.isfinite(ro)
    assert (np.isfinite(a) == fine).all(), np.argwhere(np.isfinite(a) != fine)[:4]
    assert (np.isnan(a) == np.isnan(ro)).all() and (a[np.isinf(ro)] == ro[np.isinf(ro)]).all()
    rw = np.where(fine, rw, 0.0)
    err = np.abs(np.where(fine, a - ro, 0.0))
    assert (err <= (2.0 ** -8 + 1e-3) * rw + 2.0 ** -8 * np.abs(np.where(fine, ro, 0.0)) + 1e-30).all()
    x = f64(lse)
    ok = np.isfinite(rl)
    assert (np.isfinite(x) == ok).all() and np.abs(x[ok] - rl[ok]).max() <= 4e-4 + 2.0 ** -20 * np.abs(rl[ok]).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 7, 100, 300])
@pytest.mark.parametrize("kw", [{}, {"cap": 5.0}])
def test_garbage_behind_the_sequences(d, Nq, kw):
    # what lies behind a sequence's end in a padded batch is anything: NaN, infinities, huge values
    B, Nk, H = 3, 700, 2
    lengths = [700, 333, 1]
    q, k, v, kp, vp = make(Nq, (B, Nq, H, d), (B, Nk, H, d), (B, Nk, H, d), (140, H, d), (140, H, d))
    spans = sp.padded_spans(lengths, Nq)
    want = ref.span_attention(f64(q), f64(k), f64(v), f64(spans), **kw)
    both = ref.span_attention(f64(q), f64(k), f64(v), f64(spans), f64(kp), f64(vp), **kw)
    for b, n in enumerate(lengths):
        k[b, n:] = float("nan")
        v[b, n:, 0] = float("nan")
        v[b, n:, 1] = float("-inf")
        k[b, n + 1 :: 3] = 3e38
        v[b, n + 2 :: 5] = float("inf")
    check(la.lite_attn_span(q, k, v, spans, **kw), want)
    check(la.lite_attn_prefix(q, kp, vp, k, v, spans, **kw), both)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(2, 2), (6, 2)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them_only(d, H, Hk):
    N = 420
    q, k, v = make(1, (1, N, H, d), (1, N, Hk, d), (1, N, Hk, d))
    inf, nan = float("inf"), float("nan")
    v[0, 3, 0, 5] = inf
    v[0, 60, 1, 0] = nan
    v[0, 130, 0, 5] = -inf
    v[0, 200, 0, 9] = inf
    v[0, 201, 1, d - 1] = -inf
    v[0, 410, :, 33] = nan
    with np.errstate(invalid="ignore"):
        for spans in (sp.prefix_spans(N, 0), sp.document_spans([50, 100, 20, 250]), sp.frame_spans(21, 20, window=3), None):
            want = ref.span_attention(f64(q), f64(k), f64(v), f64(spans))
            check_special(la.lite_attn_span(q, k, v, spans), want)
        one = sp.padded_spans([205], 3, causal=True)
        want = ref.span_attention(f64(q[:, :3]), f64(k), f64(v), f64(one))
        check_special(la.lite_attn_span(q[:, :3].contiguous(), k, v, one), want)


def test_not_finite_values_in_more_tiles_than_an_item_lists():
    N, d = 1500, 64
    q, k, v = make(4, (1, N, 1, d), (1, N, 1, d), (1, N, 1, d))
    v[0, 7::97, 0, 3] = float("nan")
    n = torch.arange(N)
    spans = torch.stack([(n * 7919) % N, torch.clamp((n * 7919) % N + 40, max=N)], -1).int().cuda()
    with np.errstate(invalid="ignore"):
        check_special(la.lite_attn_span(q, k, v, spans), ref.span_attention(f64(q), f64(k), f64(v), f64(spans)))


def test_strided_views_and_a_batch_that_shares_its_keys():
    B, N, H, d = 3, 190, 2, 128
    qkv, kv = make(6, (B, N, 3 * H, d), (1, N, 2 * H, d))
    q, k, v = qkv[:, :, :H], qkv[:, :, H : 2 * H], qkv[:, :, 2 * H :]
    check(la.lite_attn_span(q, k, v, sp.prefix_spans(N, 3)),
          ref.span_attention(f64(q), f64(k), f64(v), f64(sp.prefix_spans(N, 3))))
    k1, v1 = kv[:, :, :H].expand(B, -1, -1, -1), kv[:, :, H:].expand(B, -1, -1, -1)
    check(la.lite_attn_span(q, k1, v1), ref.span_attention(f64(q), f64(k1), f64(v1)))
    q1 = q[:1].expand(B, -1, -1, -1)
    check(la.lite_attn_prefix(q1[:, :5], kv[0, :, :H], kv[0, :, H:], k, v),
          ref.span_attention(f64(q1[:, :5]), f64(k), f64(v), None, f64(kv[0, :, :H]), f64(kv[0, :, H:])))
    # one token a sequence out of a wider buffer: evenly spaced, so it can be stacked
    check(la.lite_attn_prefix(q[:, :1], kv[0, :, :H], kv[0, :, H:], k, v),
          ref.span_attention(f64(q[:, :1]), f64(k), f64(v), None, f64(kv[0, :, :H]), f64(kv[0, :, H:])))


def test_a_cache_past_32_bit_offsets():
    Nk, Hk, d = 600_000, 30, 128  # 2.3e9 elements; all but the end is uninitialised memory
    k = torch.empty((1, Nk, Hk, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    (q,) = make(7, (1, 2, Hk, d))
    tail = 300
    k[:, -tail:], v[:, -tail:] = make(8, (1, tail, Hk, d), (1, tail, Hk, d))
    spans = torch.tensor([[Nk - tail, Nk], [Nk - 17, Nk - 1]], dtype=torch.int32, device="cuda")
    want = ref.span_attention(f64(q), f64(k[:, -tail:]), f64(v[:, -tail:]), np.array([[0, tail], [tail - 17, tail - 1]]))
    check(la.lite_attn_span(q, k, v, spans), want)
    q2 = q.expand(1, 2, Hk, d)
    k2 = k.as_strided((2, 200, Hk, d), ((Nk - 250) * Hk * d, Hk * d, d, 1))  # a batch stride past 2^31
    k2[0], k2[1] = make(9, (200, Hk, d), (200, Hk, d))
    q2 = torch.cat([q, q])
    check(la.lite_attn_span(q2, k2, k2), ref.span_attention(f64(q2), f64(k2), f64(k2)))


def test_equal_calls_give_equal_bits_on_any_grid():
    lengths = [1, 700, 3, 256, 11, 129, 300, 2]
    N = sum(lengths)
    q, k, v = make(10, (2, N, 4, 128), (2, N, 4, 128), (2, N, 4, 128))
    spans = sp.document_spans(lengths)
    (q1,) = make(12, (2, 1, 4, 128))
    first = la.lite_attn_span(q, k, v, spans), la.lite_attn_span(q1, k, v)
    try:
        for ctas in (0, 1, 7):
            la.lite_set_option(la.LITE_OPT_MAX_CTAS, ctas)
            again = la.lite_attn_span(q, k, v, spans), la.lite_attn_span(q1, k, v)
            for a, b in zip(first, again):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    finally:
        la.lite_set_option(la.LITE_OPT_MAX_CTAS, 0)


def _calls():
    """Calls of each kind with their inputs: split and joined, stacked, handed out by a counter, direct."""
    q, k, v, kp, vp = make(20, (4, 1, 5, 128), (4, 900, 5, 128), (4, 900, 5, 128), (2000, 5, 128), (2000, 5, 128))
    big = make(21, (1, 2600, 24, 64), (1, 2600, 24, 64), (1, 2600, 24, 64))
    docs = sp.document_spans([1000, 7, 1593])
    ragged = sp.padded_spans([900, 3, 451, 0], 1)
    return [
        lambda **kw: la.lite_attn_span(q, k, v, ragged, **kw),
        lambda **kw: la.lite_attn_prefix(q, kp, vp, k, v, **kw),
        lambda **kw: la.lite_attn_span(*big, docs, cap=10.0, **kw),
    ]


def test_captured_and_replayed_beside_an_eager_call():
    for call in _calls():
        want = call()
        o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        torch.cuda.synchronize()
        g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
        with torch.cuda.graph(g):
            call(o=o, lse=lse)
        with torch.cuda.graph(h):
            call(o=o2, lse=lse2)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            o.zero_(), lse.zero_()
            g.replay()
            with torch.cuda.stream(s):
                h.replay()
            eager = call()
            torch.cuda.synchronize()
            for a, b in ((o, lse), (o2, lse2), eager):
                assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_two_streams_at_once():
    for call in _calls():
        want = call()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = [call(stream=s) for s in streams for _ in range(3)]
        torch.cuda.synchronize()
        for a, b in got:
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_a_stalled_kernel_gives_up_and_says_so():
    q, k, v = make(30, (1, 300, 2, 128), (1, 300, 2, 128), (1, 300, 2, 128))
    (q1,) = make(31, (1, 1, 2, 128))
    want = la.lite_attn_span(q, k, v), la.lite_attn_span(q1, k, v)
    assert la.lite_get_device_status() == 0
    la.lite_set_option(la.LITE_OPT_WAIT_LIMIT_NS, 2_000_000)
    la.lite_set_option(la.LITE_OPT_DEBUG_STALL, 1)
    try:
        for x in (q, q1):
            la.lite_attn_span(x, k, v)
            assert la.lite_get_device_status() == la.LITE_ERR_TIMEOUT
    finally:
        la.lite_set_option(la.LITE_OPT_DEBUG_STALL, 0)
        la.lite_set_option(la.LITE_OPT_WAIT_LIMIT_NS, 4_000_000_000)
    for x, w in zip((q, q1), want):
        got = la.lite_attn_span(x, k, v)
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


@pytest.mark.parametrize("d", [64, 128])
def test_many_items_of_few_rows(d):
    # more items than CTAs, handed out one by one; row counts on both sides of 32
    lengths = [(37 * b) % 300 for b in range(48)]
    span_case(48, 1, 300, 8, 8, d, sp.padded_spans(lengths, 1), seed=1)
    span_case(12, 32, 140, 16, 16, d, sp.padded_spans(lengths[:12], 32, causal=True), seed=2)
    span_case(12, 33, 140, 16, 16, d, sp.padded_spans(lengths[:12], 33, causal=True), seed=3)


@pytest.mark.parametrize("d", [64, 128])
def test_prefix_pass_and_own_pass_of_different_kinds(d):
    # 64 stacked rows against the prefix, 8 rows of each sequence against its own keys
    B, Nq, Nk, Np, H = 8, 8, 60, 6000, 20
    q, k, v, kp, vp = make(d, (B, Nq, H, d), (B, Nk, H, d), (B, Nk, H, d), (Np, H, d), (Np, H, d))
    spans = sp.padded_spans([60, 1, 0, 33, 8, 59, 60, 17], Nq, causal=True)
    o, lse = la.lite_attn_prefix(q, kp, vp, k, v, spans, return_lse=False)
    assert lse is None
    check((o, None), ref.span_attention(f64(q), f64(k), f64(v), f64(spans), f64(kp), f64(vp)))


def test_outputs_given_and_rows_outside_them_untouched():
    q, k, v = make(5, (2, 70, 3, 64), (2, 90, 3, 64), (2, 90, 3, 64))
    want = la.lite_attn_span(q, k, v)
    big = torch.full((4, 70, 3, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 3, 70), 5.0, device="cuda")
    got = la.lite_attn_span(q, k, v, o=big[1:3], lse=lse[1:3])
    assert got[0].data_ptr() == big[1:3].data_ptr()
    assert torch.equal(big[1:3], want[0]) and torch.equal(lse[1:3], want[1])
    assert (big[0] == 5).all() and (big[3] == 5).all() and (lse[0] == 5).all() and (lse[3] == 5).all()
    for bad in (dict(o=big), dict(o=big[1:3].float()), dict(lse=lse), dict(spans=torch.zeros(70, 2, device="cuda")),
                dict(spans=torch.zeros(3, 70, 2, dtype=torch.int32, device="cuda")), dict(cap=-1.0),
                dict(slopes=torch.zeros(2, device="cuda")), dict(q_pos=torch.zeros(70, device="cuda"))):
        with pytest.raises(ValueError):
            la.lite_attn_span(q, k, v, **bad)
    with pytest.raises(ValueError):
        la.lite_attn_span(q, k[..., ::2], v[..., ::2])
    with pytest.raises(ValueError):
        la.lite_attn_span(q, k[:, :, :2], v[:, :, :2])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,scale", [(1e-30, None), (1e-9, None), (1e-4, 100.0), (3e38, None), (40.0, 1e-6)])
def test_caps_and_scales_at_the_ends_of_the_range(d, cap, scale):
    # a cap next to nothing makes all scores equal, an enormous one changes none
    q, k, v = make(13, (1, 130, 2, d), (1, 260, 2, d), (1, 260, 2, d))
    for spans in (None, sp.padded_spans([200], 130)):
        want = ref.span_attention(f64(q), f64(k), f64(v), f64(spans), cap=cap if cap < 1e30 else 0.0, scale=scale)
        check(la.lite_attn_span(q, k, v, spans, cap=cap, scale=scale), want)
