"""Sliding-window attention with sinks: the plain definition, float64, from contiguous per-sequence K/V.

Test infrastructure only (see the package docstring).  The query at position p of its row sees the keys k <= p
with k > p - window, and the row's first ``sinks`` keys; everything else is ``attention_row``.
"""
from __future__ import annotations

import math

import numpy as np


def visible_keys(p: int, window: int, sinks: int) -> np.ndarray:
    """Positions the query at position p sees, ascending."""
    return np.array([k for k in range(p + 1) if k > p - window or k < sinks])


def window_attention_row(q: np.ndarray, k: np.ndarray, v: np.ndarray, window: int, sinks: int) -> np.ndarray:
    """q fp16 [q_len, Hq, d]; k, v [ctx, Hkv, d] in position order, this pass's included.  float64 [q_len, Hq, d].
    Keys and values that a query does not see are not touched (they may be anything)."""
    q_len, num_q_heads, d = q.shape
    ctx, num_kv_heads, _ = k.shape
    group = num_q_heads // num_kv_heads
    out = np.zeros((q_len, num_q_heads, d), dtype=np.float64)
    for i in range(q_len):
        keys = visible_keys(ctx - q_len + i, window, sinks)
        kk, vv = k[keys].astype(np.float64), v[keys].astype(np.float64)
        qi = q[i].astype(np.float64).reshape(num_kv_heads, group, d)
        scores = np.einsum("ghd,kgd->ghk", qi, kk) / math.sqrt(d)
        weights = np.exp(scores - scores.max(axis=-1, keepdims=True))
        weights /= weights.sum(axis=-1, keepdims=True)
        out[i] = np.einsum("ghk,kgd->ghd", weights, vv).reshape(num_q_heads, d)
    return out
