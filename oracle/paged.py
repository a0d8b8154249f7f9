"""Paged caches in fp64, stream by stream, with the pages already gathered: what a chunk's rows
attend to, the attention weight that every cached token gathers, and eviction by it.

The streams are plain arrays here: k, v [tokens, kv_heads, d] (the chunk's own tokens last), q
[rows, q_heads, d]; query head h reads KV head h // (q_heads // kv_heads).
"""
from __future__ import annotations

import numpy as np


def visible(n_kv: int, n_q: int, causal: bool) -> np.ndarray:
    """[n_q, n_kv] truth values: row i stands at place n_kv - n_q + i."""
    place = np.arange(n_kv)[None, :]
    last = (n_kv - n_q + np.arange(n_q))[:, None] if causal else np.full((n_q, 1), n_kv - 1)
    return place <= last


def attend(q, k, v, causal: bool):
    """(out [rows, q_heads, d], lse [rows, q_heads], weight [kv_heads, tokens], reach [rows, q_heads, d]):
    reach is sum_j p_j |v_j|, the size that rounding p is measured against."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n_q, heads, d = q.shape
    n_kv, kv_heads, _ = k.shape
    group = heads // kv_heads
    seen = visible(n_kv, n_q, causal)
    out, reach = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((n_q, heads), -np.inf)
    weight = np.zeros((kv_heads, n_kv))
    if n_kv == 0:
        return out, lse, weight, reach
    for h in range(heads):
        s = np.where(seen, q[:, h] @ k[:, h // group].T / np.sqrt(d), -np.inf)
        top = s.max(1, keepdims=True)
        e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        total = e.sum(1, keepdims=True)
        p = e / np.where(total > 0, total, 1.0)
        out[:, h] = p @ v[:, h // group]
        reach[:, h] = p @ np.abs(v[:, h // group])
        with np.errstate(divide="ignore"):
            lse[:, h] = (top + np.log(total))[:, 0]
        weight[h // group] += p.sum(0)
    return out, lse, weight, reach


def accumulate(old, got, n_q: int):
    """The weights after a chunk: the chunk's own tokens (the last n_q) start from zero."""
    base = np.array(old, np.float64)
    if n_q:
        base[:, max(0, base.shape[1] - n_q):] = 0.0
    return base + got


def kept(weight, keep: int, sinks: int, recent: int) -> list[int]:
    """Places that one KV head keeps of weight [tokens]: written as the definition reads, one token
    at a time. NaN ranks below everything, equal weights go to the earlier place."""
    n = len(weight)
    if n <= keep:
        return list(range(n))
    fixed = set(range(sinks)) | set(range(n - recent, n))
    rest = [j for j in range(n) if j not in fixed]
    rest.sort(key=lambda j: ((1, 0.0) if np.isnan(weight[j]) else (0, -float(weight[j])), j))
    return sorted(fixed | set(rest[:keep - len(fixed)]))
