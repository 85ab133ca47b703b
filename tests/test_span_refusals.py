"""What lite_qk_rope, lite_attn_span and lite_attn_prefix refuse, and the span tables (CPU only).

The C calls are rejected by argument validation before the library touches CUDA; the fake pointers are
never dereferenced. The Python checks raise before any C call.
"""

import ctypes

import pytest
import torch

from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import spans as sp
from temporal_block_sparse_b200.attention import AxisRope, ChunkedAttention

FAKE = 1 << 20
INVALID, UNSUPPORTED = la.LITE_ERR_INVALID_ARG, la.LITE_ERR_UNSUPPORTED

_SPAN = ("q k v k_prefix v_prefix o lse spans slopes q_pos k_pos prefix_pos q0 q1 q2 k0 k1 k2 v0 v1 v2 kp0 kp1 kp2 vp0 "
         "vp1 vp2 B Nq Nk Np H Hk d span_batches pos_batches scale cap").split()


def span(fn="lite_attn_span", **kw):
    d, H, Hk, Nq, Nk = 128, 4, 2, 100, 200
    a = dict.fromkeys(_SPAN, 0)
    a.update(q=FAKE, k=FAKE, v=FAKE, o=FAKE, q0=Nq * H * d, q1=H * d, q2=d, k0=Nk * Hk * d, k1=Hk * d, k2=d,
             v0=Nk * Hk * d, v1=Hk * d, v2=d, kp1=Hk * d, kp2=d, vp1=Hk * d, vp2=d, B=2, Nq=Nq, Nk=Nk, H=H, Hk=Hk, d=d,
             span_batches=1, pos_batches=1, scale=0.0, cap=0.0)
    a.update(kw)
    return getattr(la.load(), fn)(la._SPAN_ARGS.pack(*(a[x] for x in _SPAN)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INVALID), (dict(o=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID), (dict(Nq=0), INVALID), (dict(Nk=0), INVALID),
    (dict(Nk=-1), INVALID), (dict(Hk=3), INVALID), (dict(cap=-1.0), INVALID), (dict(cap=float("nan")), INVALID),
    (dict(cap=float("inf")), INVALID), (dict(q_pos=FAKE), INVALID), (dict(k_pos=FAKE), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(H=256, Hk=1), UNSUPPORTED), (dict(q=FAKE + 8), UNSUPPORTED),
    (dict(o=FAKE + 2), UNSUPPORTED), (dict(lse=FAKE + 2), UNSUPPORTED), (dict(spans=FAKE + 4), UNSUPPORTED),
    (dict(slopes=FAKE + 1), UNSUPPORTED), (dict(q1=4), UNSUPPORTED), (dict(q1=0), UNSUPPORTED), (dict(k2=12), UNSUPPORTED),
    (dict(v1=-256), UNSUPPORTED), (dict(k0=-8), UNSUPPORTED), (dict(k1=1 << 40), UNSUPPORTED),
    (dict(Nk=(1 << 30) + 1), UNSUPPORTED), (dict(B=1 << 16, Nq=1 << 16), UNSUPPORTED),
    (dict(slopes=FAKE, Nk=(1 << 24) + 1), UNSUPPORTED),
])
def test_span_argument_errors(kw, code):
    assert span(**kw) == code
    assert span("lite_attn_prefix", **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Np=-1), INVALID), (dict(Np=5), INVALID), (dict(Np=5, k_prefix=FAKE), INVALID),
    (dict(Np=5, k_prefix=FAKE + 8, v_prefix=FAKE), UNSUPPORTED),
    (dict(Np=5, k_prefix=FAKE, v_prefix=FAKE, kp1=4), UNSUPPORTED),
    (dict(Np=(1 << 30) + 1, k_prefix=FAKE, v_prefix=FAKE), UNSUPPORTED),
    (dict(prefix_pos=FAKE), INVALID),
])
def test_prefix_argument_errors(kw, code):
    assert span("lite_attn_prefix", **kw) == code


def test_null_arguments():
    lib = la.load()
    for fn in (lib.lite_attn_span, lib.lite_attn_prefix, lib.lite_qk_rope):
        assert fn(None, None) == INVALID


_ROPE = ("q k qo ko qs0 qs1 qs2 ks0 ks1 ks2 qos0 qos1 qos2 kos0 kos1 kos2 wq wk freq axis pos pos_b pos_a grid start "
         "dtype pos_dtype norm pairing n_axes B N H Hk d eps").split()


def rope(freq=None, axis=None, grid=(3, 5, 7), **kw):
    plan = la.RopePlan((44, 42, 42))
    f = (ctypes.c_double * 64)(*(freq or plan.freq))
    x = (ctypes.c_int32 * 64)(*(axis or plan.axis))
    g = (ctypes.c_int64 * 3)(*grid)
    H, Hk, d, N = 4, 2, 128, 50
    a = dict.fromkeys(_ROPE, 0)
    a.update(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, qs0=N * H * d, qs1=H * d, qs2=d, ks0=N * Hk * d, ks1=Hk * d, ks2=d,
             qos0=N * H * d, qos1=H * d, qos2=d, kos0=N * Hk * d, kos1=Hk * d, kos2=d, freq=ctypes.addressof(f),
             axis=ctypes.addressof(x), grid=ctypes.addressof(g), n_axes=3, B=2, N=N, H=H, Hk=Hk, d=d, eps=1e-6)
    a.update(kw)
    return la.load().lite_qk_rope(la._ROPE_ARGS.pack(*(a[x] for x in _ROPE)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INVALID), (dict(qo=0), INVALID), (dict(ko=0), INVALID), (dict(freq=[float("nan")] * 64), INVALID),
    (dict(axis=[3] * 64), INVALID), (dict(axis=[-1] * 64), INVALID), (dict(n_axes=0), INVALID), (dict(n_axes=5), INVALID),
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID), (dict(dtype=3), INVALID),
    (dict(pairing=2), INVALID), (dict(norm=3), INVALID), (dict(norm=1), INVALID),
    (dict(norm=1, wq=FAKE, wk=FAKE, eps=-1.0), INVALID), (dict(grid=(3, 0, 7)), INVALID), (dict(start=-1), INVALID),
    (dict(start=56), INVALID), (dict(start=(1 << 63) - 1), INVALID), (dict(pos=FAKE, pos_dtype=0), INVALID),
    (dict(pos=FAKE, pos_dtype=2, pos_a=-1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(q=FAKE + 4), UNSUPPORTED), (dict(ko=FAKE + 8), UNSUPPORTED),
    (dict(norm=1, wq=FAKE + 4, wk=FAKE), UNSUPPORTED), (dict(qs1=12), UNSUPPORTED), (dict(kos2=4), UNSUPPORTED),
    (dict(qs0=-8), UNSUPPORTED), (dict(H=129), UNSUPPORTED), (dict(B=1 << 15, N=1 << 16, pos=FAKE, pos_dtype=2), UNSUPPORTED),
])
def test_rope_argument_errors(kw, code):
    assert rope(**kw) == code


def test_python_checks_come_before_any_call():
    x = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)  # not on a GPU
    with pytest.raises(ValueError, match="CUDA"):
        la.lite_attn_span(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        la.lite_attn_prefix(x, x[0], x[0], x, x)
    with pytest.raises(ValueError, match="CUDA"):
        la.lite_qk_rope(x, x, la.RopePlan((24, 20, 20)), grid=(2, 2, 2))
    with pytest.raises(ValueError, match="bf16, fp16 or fp32"):
        la.lite_qk_rope(x.double(), None, la.RopePlan((24, 20, 20)), grid=(2, 2, 2))


@pytest.mark.parametrize("kw", [
    dict(dims=(44, 42, 41)), dict(dims=()), dict(dims=(16,) * 5), dict(dims=(44, 42, 40)), dict(dims=(64, 64, 64)),
    dict(dims=(64,), pairing="other"), dict(dims=(64,), theta=0.0), dict(dims=(64,), theta=float("inf")),
    dict(dims=(64,), freqs=[1.0] * 31), dict(dims=(64,), freqs=[float("nan")] * 32), dict(dims=(-2, 66)),
    dict(dims=(128,), head_dim=64)])
def test_rope_plan_refusals(kw):
    with pytest.raises(ValueError):
        la.RopePlan(**kw)


def test_rope_plan_frequencies():
    p = la.RopePlan((4, 2), theta=100.0, head_dim=64)
    assert p.axis[:4] == [0, 0, 1, 0] and p.freq[:4] == [1.0, 100.0 ** -0.5, 1.0, 0.0] and len(p.freq) == 32
    assert la.RopePlan((64,), freqs=range(32)).freq[5] == 5.0


def table(t):
    assert t.dtype == torch.int32 and t.is_contiguous()
    return t.tolist()


def test_span_tables():
    assert table(sp.document_spans([2, 0, 1], device="cpu")) == [[0, 2], [0, 2], [2, 3]]
    assert table(sp.document_spans([2, 2], causal=True, device="cpu")) == [[0, 1], [0, 2], [2, 3], [2, 4]]
    assert table(sp.prefix_spans(4, 2, device="cpu")) == [[0, 2], [0, 2], [0, 3], [0, 4]]
    assert table(sp.prefix_spans(2, 9, device="cpu")) == [[0, 2], [0, 2]]
    assert table(sp.frame_spans(2, 2, device="cpu")) == [[0, 2], [0, 2], [0, 4], [0, 4]]
    assert table(sp.frame_spans(2, 1, window=2, past=3, device="cpu")) == [[2, 4], [3, 5]]
    assert table(sp.padded_spans([3, 0], 2, device="cpu")) == [[[0, 3], [0, 3]], [[0, 0], [0, 0]]]
    assert table(sp.padded_spans([3, 1], 2, causal=True, device="cpu")) == [[[0, 2], [0, 3]], [[0, 0], [0, 1]]]
    for f in (lambda: sp.document_spans([]), lambda: sp.document_spans([-1]), lambda: sp.prefix_spans(0, 0),
              lambda: sp.prefix_spans(3, -1), lambda: sp.frame_spans(0, 1), lambda: sp.frame_spans(1, 1, window=0),
              lambda: sp.frame_spans(1, 1, past=-1), lambda: sp.padded_spans([1], 0), lambda: sp.padded_spans([-1], 1)):
        with pytest.raises(ValueError):
            f()


def test_chunked_attention_refusals():
    rope_ = AxisRope((24, 20, 20), (4, 2, 2))
    for kw in (dict(frames=0, frame_tokens=4), dict(frames=1, frame_tokens=0), dict(frames=1, frame_tokens=4, window=0)):
        with pytest.raises(ValueError):
            ChunkedAttention(rope_, **kw)
    a = ChunkedAttention(rope_, frames=2, frame_tokens=4)
    x = torch.zeros(1, 6, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="whole number of frames"):
        a(x, x, x)
    x = torch.zeros(1, 12, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="2 frames"):
        a(x, x, x)
    with pytest.raises(ValueError):
        a.set_history(x[0], x[0, :3])
