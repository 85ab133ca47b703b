"""lite_attn_span with values that are not finite: what rows see of them does not depend on which softmax group
comes first (needs a B200).

A weight that underflows to 0 makes NaN of an infinity in the product and leaves an infinity where the value was
taken out before the product and added afterwards, so both groups of an item have to treat a key tile
alike. The oracle's 64-bit weights do not underflow here (e^-190 at most), its infinities stay infinities.
"""

import numpy as np
import pytest
import torch

from oracle import span as ref
from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import spans as sp
from test_gpu_span import check_special, f64, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(autouse=True)
def _clean_state():
    la.load()
    yield
    assert la.lite_get_device_status() == 0


def bits(t):
    """Bit patterns, so that equal NaN compare equal."""
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).clone()


def same_bits(call, times=8):
    first = [bits(t) for t in call()]
    for _ in range(times):
        assert all(torch.equal(a, bits(t)) for a, t in zip(first, call()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 9.0])
def test_infinity_in_a_tile_that_one_group_sees_all_of(d, cap):
    # Causal rows 0 .. 255 are one item: the tiles of keys 0 .. 127 are cut for rows 0 .. 127 (the first group) and
    # seen entirely by rows 128 .. 255, whose weight for key 5 is below 2^-200 (0 in 32 bits).
    N, H = 256, 160
    q, k, v = make(d, (1, N, H, d), (1, N, H, d), (1, N, H, d))
    v[0, 5, :, 7] = float("inf")
    v[0, 60, ::2, 1] = float("-inf")
    v[0, 61, ::3, 2] = float("nan")
    slopes = torch.full((H,), 1.2 if not cap else 0.6, device="cuda")
    causal = sp.prefix_spans(N, 0)
    o, lse = la.lite_attn_span(q, k, v, causal, cap=cap, slopes=slopes)
    with np.errstate(invalid="ignore"):
        want = ref.span_attention(f64(q[:, :, :4]), f64(k[:, :, :4]), f64(v[:, :, :4]), f64(causal), cap=cap,
                                  slopes=f64(slopes[:4]))
    check_special((o[:, :, :4], lse[:, :4]), want)
    assert torch.isposinf(o[0, 5:, :, 7]).all() and torch.isfinite(o[0, :5]).all()
    same_bits(lambda: la.lite_attn_span(q, k, v, causal, cap=cap, slopes=slopes))


@pytest.mark.parametrize("d", [64, 128])
def test_infinities_at_documents_edges_give_equal_bits_on_any_grid(d):
    # edges inside tiles: either group, both or neither has a tile cut
    lengths = [150, 333, 1, 64, 300, 17, 190]
    N, H = sum(lengths), 6
    q, k, v = make(d + 1, (2, N, H, d), (2, N, H, d), (2, N, H, d))
    v[:, 3::41, :, 5] = float("inf")
    v[:, 9::77, :, 6] = float("-inf")
    slopes = torch.linspace(0.2, 1.3, H, device="cuda")
    for spans in (sp.document_spans(lengths), sp.document_spans(lengths, causal=True)):
        call = lambda: la.lite_attn_span(q, k, v, spans, slopes=slopes)
        same_bits(call)
        first = [bits(t) for t in call()]
        try:
            for ctas in (1, 7):
                la.lite_set_option(la.LITE_OPT_MAX_CTAS, ctas)
                assert all(torch.equal(a, bits(t)) for a, t in zip(first, call()))
        finally:
            la.lite_set_option(la.LITE_OPT_MAX_CTAS, 0)
        # a row that sees such a value is not finite in its column, no other row or column is touched
        seen = torch.zeros(2, N, H, d, dtype=torch.bool, device="cuda")
        at = torch.arange(N, device="cuda")
        sees = (at >= spans[:, :1]) & (at < spans[:, 1:])  # [row, key]
        for c in (5, 6):
            bad = ~torch.isfinite(v[0, :, 0, c])
            seen[:, :, :, c] = (sees & bad).any(1)[None, :, None]
        assert torch.equal(~torch.isfinite(call()[0]), seen)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nk", [600, 9000])
def test_infinity_far_from_a_single_token(d, Nk):
    # The key's weight underflows in every join: of the quarters and groups of a CTA, and of the split keys. Its column
    # is not finite all the same, whether a span ends in its tile (start 1) or not (start 0).
    H = 3
    q, k, v = make(Nk + d, (2, 1, H, d), (2, Nk, H, d), (2, Nk, H, d))
    v[:, 3, :, 4] = float("inf")
    v[:, Nk // 2, :, 9] = float("-inf")
    spans = torch.tensor([[[0, Nk]], [[1, Nk]]], dtype=torch.int32, device="cuda")
    slopes = torch.tensor([1.0, 0.9, 1.2], device="cuda")
    call = lambda: la.lite_attn_span(q, k, v, spans, slopes=slopes)
    o, lse = call()
    assert torch.isfinite(lse).all()
    fine = torch.ones(d, dtype=torch.bool, device="cuda")
    fine[[4, 9]] = False
    assert not torch.isfinite(o[..., ~fine]).any() and torch.isfinite(o[..., fine]).all()
    same_bits(call, 30)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 40])
def test_more_cut_tiles_with_infinities_than_an_item_lists_in_split_calls(d, Nq):
    # Every second token of the batch sees another part of the keys, most tiles are cut and hold an infinity; parts
    # of a split call add those of their own tiles only.
    Nk, H = 40 * d, 2
    q, k, v = make(Nq + d, (3, Nq, H, d), (3, Nk, H, d), (3, Nk, H, d))
    v[:, 11 :: d, :, 3] = float("inf")
    n = torch.arange(Nq)
    first = (n * 131) % (Nk - 700)
    spans = torch.stack([first, first + 13 + (n * 61) % 687], -1).int()[None].repeat(3, 1, 1)
    spans[1, ::2, 1] = Nk
    spans[2, :, 0] = 12  # behind the first infinity
    spans[2, :, 1] = torch.clamp(15 + n * 5, max=Nk)
    spans = spans.cuda()
    call = lambda: la.lite_attn_span(q, k, v, spans)
    o, lse = call()
    at = torch.arange(Nk, device="cuda")
    sees = ((at >= spans[..., :1]) & (at < spans[..., 1:]) & (at % d == 11)).any(-1)  # [B, Nq]
    assert torch.equal(~torch.isfinite(o[..., 3]), sees[..., None].expand(-1, -1, H))
    assert torch.isfinite(o[..., 4:]).all() and torch.isfinite(o[..., :3]).all()
    same_bits(call, 30)
