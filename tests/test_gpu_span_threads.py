"""lite_qk_rope and lite_attn_span called by several host threads at once (needs a B200).

ctypes releases the interpreter lock during a call, so the host code of such calls runs side by side.
"""

import threading

import pytest
import torch

from temporal_block_sparse_b200 import lite_attn as la
from temporal_block_sparse_b200 import spans as sp
from temporal_block_sparse_b200 import workload as wl

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(autouse=True)
def _clean_state():
    la.load()
    yield
    assert la.lite_get_device_status() == 0


def at_once(calls, times):
    """Runs every call `times` times in a thread of its own, on a stream of its own; their first results have to
    come out equal to those of a call by itself."""
    want = [call(None) for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    start, failed = threading.Barrier(len(calls)), []

    def work(call, stream, first):
        try:
            torch.cuda.set_device(0)
            start.wait(30)
            for i in range(times):
                got = call(stream)
                if i % 100 == 0:
                    stream.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, first))
        except Exception as e:  # noqa: BLE001 (told to the test below)
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(calls, streams, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert not failed, failed[0]


def test_rope_calls_of_different_head_counts(monkeypatch):
    # 128 heads take 109 KB of shared memory, 64 heads 55 KB, in the same kernel
    d, plan = 128, la.RopePlan(wl.axis_split(128))
    pos = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    calls = []
    for heads in (128, 64, 128, 60):
        q = torch.randn(1, 3, heads, d, device="cuda").to(torch.bfloat16)
        calls.append(lambda stream, q=q: la.lite_qk_rope(q, None, plan, pos=pos, stream=stream)[:1])
    at_once(calls, 500)
    # the C calls alone, one right after the other, so that they meet often (all that the packed arguments point to
    # is alive: plan, pos, q and outs)
    packed = []
    monkeypatch.setattr(la, "_call_on", lambda fn, args, index, stream: packed.append((args, stream)))
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [call(s) for call, s in zip(calls, streams)]
    codes, rope = set(), la.load().lite_qk_rope

    def work(args, stream):
        for _ in range(20000):
            codes.add(rope(args, stream.cuda_stream))

    threads = [threading.Thread(target=work, args=x) for x in packed]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert codes == {la.LITE_OK} and len(outs) == 4


def test_span_calls_of_every_kind():
    calls = []
    for d, cap, Nq in ((64, 0.0, 1), (128, 0.0, 1), (128, 5.0, 200), (64, 5.0, 200)):
        q, k = (torch.randn(2, n, 4, d, device="cuda").to(torch.bfloat16) for n in (Nq, 900))
        spans = sp.padded_spans([900, 301], Nq, causal=True)
        calls.append(lambda stream, a=(q, k, k, spans), cap=cap: la.lite_attn_span(*a, cap=cap, stream=stream))
    at_once(calls, 600)
