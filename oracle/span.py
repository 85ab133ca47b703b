"""Span attention, shared-prefix attention and rotary positions in plain numpy, 64 bits.

Test infrastructure: written from the formulas of include/lite_attn.h, one head and one batch entry at
a time, without the library.
"""

from __future__ import annotations

import math
from typing import Optional

import numpy as np


def span_attention(q, k, v, spans=None, k_prefix=None, v_prefix=None, scale: Optional[float] = None, cap: float = 0.0,
                   slopes=None, q_pos=None, k_pos=None, prefix_pos=None):
    """(o [B, Nq, H, d], lse [B, H, Nq], weighted [B, Nq, H, d]): the last is sum p |v|, which error
    bounds are counted in."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, Nq, H, d = q.shape
    Nk, Hk = k.shape[1], k.shape[2]
    Np = 0 if k_prefix is None else k_prefix.shape[0]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, w = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((B, H, Nq), -np.inf)
    if spans is None:
        spans = np.broadcast_to(np.array([0, Nk]), (B, Nq, 2))
    spans = np.broadcast_to(np.asarray(spans, dtype=np.int64), (B, Nq, 2))
    own = np.arange(Nk)
    for b in range(B):
        seen = (own >= spans[b, :, :1]) & (own < spans[b, :, 1:])
        seen = np.concatenate([np.ones((Nq, Np), dtype=bool), seen], 1)
        for h in range(H):
            hk = h // (H // Hk)
            kk, vv = k[b, :, hk], v[b, :, hk]
            if Np:
                kk = np.concatenate([np.asarray(k_prefix, dtype=np.float64)[:, hk], kk])
                vv = np.concatenate([np.asarray(v_prefix, dtype=np.float64)[:, hk], vv])
            s = q[b, :, h] @ kk.T * scale
            if cap:
                s = cap * np.tanh(s / cap)
            if slopes is not None:
                qp = np.arange(Np + Nk - Nq, Np + Nk) if q_pos is None else np.broadcast_to(q_pos, (B, Nq))[b]
                kp = np.arange(Np, Np + Nk) if k_pos is None else np.broadcast_to(k_pos, (B, Nk))[b]
                pp = np.arange(Np) if prefix_pos is None else prefix_pos
                s = s - float(slopes[h]) * np.abs(qp[:, None].astype(np.float64) - np.concatenate([pp, kp])[None])
            for n in range(Nq):
                x, y = s[n, seen[n]], vv[seen[n]]
                if x.size == 0:
                    continue
                m = x.max()
                p = np.exp(x - m)
                t = p.sum()
                o[b, n, h] = p @ y / t
                w[b, n, h] = p @ np.abs(y) / t
                lse[b, h, n] = m + math.log(t)
    return o, lse, w


def rope(x, positions, freq, axis, pairing: str, weight=None, eps: float = 1e-6):
    """x [B, N, heads, d] normed (weight of d or heads * d elements, or None) and turned; positions [B, axes, N]."""
    x = np.array(x, dtype=np.float64)
    B, N, heads, d = x.shape
    if weight is not None:
        weight = np.asarray(weight, dtype=np.float64)
        if weight.size == d:
            x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * weight
        else:
            x = x / np.sqrt((x ** 2).mean((-2, -1), keepdims=True) + eps) * weight.reshape(heads, d)
    y = np.empty_like(x)
    for p in range(d // 2):
        i, j = (2 * p, 2 * p + 1) if pairing == "interleaved" else (p, p + d // 2)
        phi = (np.asarray(positions, dtype=np.float64)[:, axis[p]] * freq[p])[:, :, None]
        c, s = np.cos(phi), np.sin(phi)
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def grid_positions(grid, start: int, N: int):
    """[axes, N] coordinates of cells start .. start + N - 1 of a row-major grid."""
    out = []
    index = [start + n for n in range(N)]
    for size in reversed(grid):
        out.append([i % size for i in index])
        index = [i // size for i in index]
    return np.array(out[::-1], dtype=np.float64)
