"""lite_qk_rope refuses outputs whose rows fall on one another by a stride of 0 (CPU only: refused before any CUDA call)."""

import pytest

from temporal_block_sparse_b200 import lite_attn as la
from test_span_refusals import INVALID, rope


@pytest.mark.parametrize("name", ["qos0", "qos1", "qos2", "kos0", "kos1", "kos2"])
def test_output_strides_of_zero(name):
    assert rope(**{name: 0}) == la.LITE_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [{"qs0": 0}, {"qs1": 0}, {"qs2": 0}, {"ks0": 0}, {"B": 1, "qos0": 0, "kos0": 0}, {"Hk": 1, "kos2": 0}])
def test_other_strides_of_zero_pass_that_check(kw):
    # without a device the call ends at its first CUDA call, not in a refusal of its arguments
    import torch

    if torch.cuda.is_available():
        pytest.skip("the pointers are fake")
    assert rope(**kw) not in (INVALID, la.LITE_ERR_UNSUPPORTED)
