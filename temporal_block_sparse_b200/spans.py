"""Key spans of query rows for lite_attn_span and lite_attn_prefix.

A table holds, for every query row, the first key it sees and the one after the last: int32 [Nq, 2], or
[B, Nq, 2] where batch entries differ. Rows without keys have an empty span.
"""

from __future__ import annotations

from typing import Optional, Sequence

import torch


def _table(first: torch.Tensor, end: torch.Tensor, device) -> torch.Tensor:
    first, end = torch.broadcast_tensors(first, end)
    return torch.stack([first, end], -1).to(torch.int32).contiguous().to(device or "cuda")


def document_spans(lengths: Sequence[int], causal: bool = False, device=None) -> torch.Tensor:
    """Sequences of these lengths packed one after the other: a row sees its own sequence (causal: up
    to and with itself). [sum(lengths), 2]."""
    lengths = torch.as_tensor([int(x) for x in lengths], dtype=torch.int64)
    if lengths.numel() == 0 or (lengths < 0).any():
        raise ValueError("lengths: non-negative numbers, one at least")
    end = lengths.cumsum(0)
    first, last = torch.repeat_interleave(end - lengths, lengths), torch.repeat_interleave(end, lengths)
    return _table(first, torch.arange(first.numel()) + 1 if causal else last, device)


def prefix_spans(N: int, prefix: int, device=None) -> torch.Tensor:
    """The first `prefix` rows see each other, later rows see everything up to and with themselves. [N, 2]."""
    if N < 1 or prefix < 0:
        raise ValueError("N >= 1 and prefix >= 0")
    n = torch.arange(N)
    return _table(torch.zeros(N, dtype=torch.int64), torch.clamp(n + 1, min=min(prefix, N)), device)


def frame_spans(frames: int, frame_tokens: int, window: Optional[int] = None, past: int = 0, device=None) -> torch.Tensor:
    """Frame-causal rows: a token sees all tokens of its frame and of the frames before it (of the
    last `window` frames with its own, if given). `past` frames of keys precede the rows' frames.
    [frames * frame_tokens, 2]."""
    if frames < 1 or frame_tokens < 1 or past < 0 or (window is not None and window < 1):
        raise ValueError("frames, frame_tokens and window >= 1, past >= 0")
    f = torch.arange(frames).repeat_interleave(frame_tokens) + past
    first = torch.zeros_like(f) if window is None else torch.clamp(f + 1 - window, min=0)
    return _table(first * frame_tokens, (f + 1) * frame_tokens, device)


def padded_spans(key_lengths: Sequence[int], Nq: int, causal: bool = False, device=None) -> torch.Tensor:
    """A padded batch: entry b holds key_lengths[b] keys. causal: its Nq rows are the last of them, each sees up
    to and with itself (rows before its first key see none). [B, Nq, 2]."""
    lengths = torch.as_tensor([int(x) for x in key_lengths], dtype=torch.int64)
    if lengths.numel() == 0 or (lengths < 0).any() or Nq < 1:
        raise ValueError("key_lengths: non-negative numbers, one at least; Nq >= 1")
    end = lengths[:, None].expand(-1, Nq)
    if causal:
        end = torch.clamp(end - Nq + 1 + torch.arange(Nq), min=0)
    return _table(torch.zeros_like(end), end, device)
