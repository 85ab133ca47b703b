"""lite_qk_rope against the 64-bit oracle (needs a B200).

Bound of an output element: one rounding to bf16, 2^-8 of its value. The 32-bit part before it: the norm's
mean and scale (a few 2^-24 of d or heads * d squares, summed in a tree), cos and sin (2^-22), two
products and a sum: 2^-18 of the pair's length covers it.
"""

import numpy as np
import pytest
import torch

from oracle import span as ref
from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import workload as wl

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def pair_length(y, pairing):
    d = y.shape[-1]
    if pairing == "interleaved":
        n = np.sqrt(y[..., 0::2] ** 2 + y[..., 1::2] ** 2)
        return np.repeat(n, 2, -1)
    n = np.sqrt(y[..., : d // 2] ** 2 + y[..., d // 2 :] ** 2)
    return np.concatenate([n, n], -1)


def check(got, want, pairing):
    err = np.abs(got.double().cpu().numpy() - want)
    lim = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * pair_length(want, pairing) + 1e-30
    assert (err <= lim).all(), (float((err / lim).max()), np.argwhere(err > lim)[:4])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("norm", ["none", "head", "row"])
def test_types_norms_and_pairings(d, pairing, dtype, norm):
    for B, N, H, Hk, start in ((2, 37, 3, 3, 0), (1, 1, 5, 1, 99999 * 35), (1, 129, 1, 2, 11), (2, 5, 40, 40, 7)):
        g = torch.Generator(device="cuda")
        g.manual_seed(N)
        qkv = (torch.randn(B, N, H + 2 * Hk, d, generator=g, device="cuda") * 1.5).to(dtype)
        q, k = qkv[:, :, :H], qkv[:, :, H : H + Hk]
        plan = la.RopePlan(wl.axis_split(d), pairing=pairing)
        wq = wk = None
        if norm != "none":
            wq = 1 + 0.2 * torch.randn(d if norm == "head" else H * d, generator=g, device="cuda")
            wk = 1 + 0.2 * torch.randn(d if norm == "head" else Hk * d, generator=g, device="cuda")
        grid = (100000, 5, 7)
        yq, yk = la.lite_qk_rope(q, k, plan, grid=grid, start=start, q_weight=wq, k_weight=wk, eps=1e-5)
        at = np.broadcast_to(ref.grid_positions(grid, start, N), (B, 3, N))
        for x, y, w in ((q, yq, wq), (k, yk, wk)):
            want = ref.rope(x.double().cpu().numpy(), at, plan.freq, plan.axis, pairing,
                            None if w is None else w.double().cpu().numpy(), 1e-5)
            check(y, want, pairing)


@pytest.mark.parametrize("dtype", [torch.float32, torch.int32])
def test_given_positions_and_partial_heads(dtype):
    B, N, H, d = 2, 50, 4, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.randn(B, N, H, d, generator=g, device="cuda").to(torch.bfloat16)
    plan = la.RopePlan((32, 16), theta=500.0, head_dim=128)  # the last 40 pairs stay as they are
    for shape in ((B, 2, N), (2, N), (1, 2, N)):
        pos = (torch.rand(shape, generator=g, device="cuda") * 1e6 - 3e5).to(dtype)
        y, none = la.lite_qk_rope(q, None, plan, pos=pos)
        assert none is None
        at = np.broadcast_to(pos.double().cpu().numpy(), (B, 2, N))
        check(y, ref.rope(q.double().cpu().numpy(), at, plan.freq, plan.axis, "interleaved"), "interleaved")
        assert torch.equal(y[..., 48:], q[..., 48:])


def test_in_place_and_into_a_cache_slice():
    B, N, H, Hk, d = 2, 21, 4, 2, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    q = torch.randn(B, N, H, d, generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn(B, N, Hk, d, generator=g, device="cuda").to(torch.bfloat16)
    plan = la.RopePlan(wl.axis_split(d))
    w = torch.ones(d, device="cuda")
    yq, yk = la.lite_qk_rope(q, k, plan, grid=(3, 1, 7), q_weight=w, k_weight=w)
    cache = torch.full((B, 64, Hk, d), 7.0, device="cuda", dtype=torch.bfloat16)
    q2 = q.clone()
    la.lite_qk_rope(q2, k, plan, grid=(3, 1, 7), q_weight=w, k_weight=w, q_out=q2, k_out=cache[:, 9 : 9 + N])
    assert torch.equal(q2, yq) and torch.equal(cache[:, 9 : 9 + N], yk)
    assert (cache[:, :9] == 7).all() and (cache[:, 9 + N :] == 7).all()
