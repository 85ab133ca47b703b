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


@pytest.mark.parametrize("B,N,H,Hk,d,dtype", [
    (300, 2, 20, 20, 128, torch.bfloat16),   # a block passes several batch entries from one step to the next
    (700, 1, 40, 1, 64, torch.float16),      # many tokens a block for the one key head, one for the queries
    (1, 3, 128, 128, 128, torch.float32),    # the widest row
    (2, 3, 256, 1, 64, torch.bfloat16),
    (1, 5000, 1, 1, 64, torch.float32)])
@pytest.mark.parametrize("norm", ["head", "row"])
def test_many_entries_and_wide_rows(B, N, H, Hk, d, dtype, norm):
    g = torch.Generator(device="cuda")
    g.manual_seed(B + H)
    q = torch.randn(B, N, H, d, generator=g, device="cuda").to(dtype)
    k = torch.randn(B, N, Hk, d, generator=g, device="cuda").to(dtype)
    plan = la.RopePlan(wl.axis_split(d))
    wq, wk = (1 + 0.2 * torch.randn(n, generator=g, device="cuda") for n in ((d, d) if norm == "head" else (H * d, Hk * d)))
    # cells past 2^40 of a huge grid, so that the index takes 64 bits
    grid, start = (1 << 40, 50, 100), (1 << 30) * 5000 + 123
    yq, yk = la.lite_qk_rope(q, k, plan, grid=grid, start=start, q_weight=wq, k_weight=wk)
    at = np.broadcast_to(ref.grid_positions(grid, start, N), (B, 3, N))
    # positions of 2^30 x frequency: the oracle's own product is off by 2^-53 of 2^30 turns, 10^-7
    for x, y, w in ((q, yq, wq), (k, yk, wk)):
        check(y, ref.rope(x.double().cpu().numpy(), at, plan.freq, plan.axis, "interleaved", w.double().cpu().numpy()),
              "interleaved")


def test_queries_alone_with_norm_and_negative_positions():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    q = torch.randn(2, 9, 3, 64, generator=g, device="cuda").to(torch.bfloat16)
    plan, w = la.RopePlan((64,), pairing="half"), torch.rand(3 * 64, generator=g, device="cuda")
    pos = torch.arange(-4, 5, dtype=torch.int32, device="cuda")[None] * 1000
    y, _ = la.lite_qk_rope(q, None, plan, pos=pos, q_weight=w)
    at = np.broadcast_to(pos.double().cpu().numpy(), (2, 1, 9))
    check(y, ref.rope(q.double().cpu().numpy(), at, plan.freq, plan.axis, "half", w.double().cpu().numpy()), "half")


def test_captured_and_on_two_streams():
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    q, k = (torch.randn(1, 2000, h, 128, generator=g, device="cuda").to(torch.bfloat16) for h in (12, 3))
    plan = la.RopePlan(wl.axis_split(128))
    want = la.lite_qk_rope(q, k, plan, grid=(2, 25, 40))
    out = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.lite_qk_rope(q, k, plan, grid=(2, 25, 40), q_out=out[0], k_out=out[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [la.lite_qk_rope(q, k, plan, grid=(2, 25, 40), stream=s) for s in streams]
    graph.replay()
    torch.cuda.synchronize()
    for a, b in got + [out]:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_python_refusals():
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    plan = la.RopePlan((24, 20, 20))
    w = torch.ones(64, device="cuda")
    for bad in (dict(grid=(1, 2, 3), start=3), dict(grid=(1, 2, 3), start=-1), dict(grid=(2, 2)), dict(),
                dict(grid=(2, 2, 2), pos=torch.zeros(3, 4, device="cuda")), dict(pos=torch.zeros(2, 4, device="cuda")),
                dict(pos=torch.zeros(3, 4, device="cuda").double()), dict(grid=(2, 2, 2), q_weight=w),
                dict(grid=(2, 2, 2), q_weight=w, k_weight=torch.ones(128, device="cuda")),
                dict(grid=(2, 2, 2), q_weight=w[1:].repeat(3)[:64], k_weight=w.half()),
                dict(grid=(2, 2, 2), q_weight=w, k_weight=w, eps=-1.0), dict(grid=(2, 2, 2), q_out=q.float()),
                dict(grid=(2, 2, 2), q_out=q[:, :3]), dict(grid=(0, 2, 2))):
        with pytest.raises(ValueError):
            la.lite_qk_rope(q, q, plan, **bad)
    with pytest.raises(ValueError):
        la.lite_qk_rope(q, q.half(), plan, grid=(2, 2, 2))
    with pytest.raises(ValueError):
        la.lite_qk_rope(q, q, la.RopePlan((44, 42, 42)), grid=(2, 2, 2))
