"""Tables of some of the batch entries are refused by the C entry points (CPU only: refused before any CUDA call)."""

import pytest

from temporal_block_sparse_b200 import lite_attn as la
from test_span_refusals import FAKE, INVALID, span


@pytest.mark.parametrize("fn", ["lite_attn_span", "lite_attn_prefix"])
@pytest.mark.parametrize("batches", [-1, 0, 2, 4, 6])
def test_tables_for_neither_one_nor_all_entries(fn, batches):
    # 3 entries: a table of 2 would be read past its end, one of 4 or 6 is not what the caller can mean
    assert span(fn, B=3, spans=FAKE, span_batches=batches) == INVALID
    for pos in ({"q_pos": FAKE}, {"k_pos": FAKE}):
        assert span(fn, B=3, slopes=FAKE, pos_batches=batches, **pos) == INVALID


@pytest.mark.parametrize("batches", [1, 3])
def test_counts_without_tables_are_not_looked_at(batches):
    # refused for the alignment of q: the checks after the tables' are reached
    assert span(B=3, q=FAKE + 8, span_batches=7, pos_batches=7) == la.LITE_ERR_UNSUPPORTED
    assert span(B=3, q=FAKE + 8, spans=FAKE, span_batches=batches) == la.LITE_ERR_UNSUPPORTED
    assert span(B=3, q=FAKE + 8, slopes=FAKE, q_pos=FAKE, pos_batches=batches) == la.LITE_ERR_UNSUPPORTED
