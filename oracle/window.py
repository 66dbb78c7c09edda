"""Attention with a sliding window and sinks (oracle, test only).

The plain definition in fp64: the query at position p sees position p' iff
p' <= p and (window == 0 or p' > p - window or p' < sinks), and its output is
softmax(q . K^T * scale) V over what it sees (zero where it sees nothing).  K
and V are gathered through the block table (katajob Q&A, "The paging idea");
only blocks that hold a seen position are looked up.  The pages describe no
window.
"""
from __future__ import annotations

import numpy as np


def seen(first: int, n: int, window: int, sinks: int) -> np.ndarray:
    """[n, first + n] boolean: what the queries at positions first .. see."""
    q = first + np.arange(n)[:, None]
    p = np.arange(first + n)[None, :]
    m = p <= q
    if window:
        m &= (p > q - window) | (p < sinks)
    return m


def paged_attention_window(q, k_cache, v_cache, tables, ctx, n, softmax_scale, window=0, sinks=0):
    """q [sum n, Hq, D] fp64, the caches' values [num_blocks, N_kv, T, D] fp64.
    Returns (out, |w| . |V|, the largest sum_d |q_d K_d| * scale a query sees):
    the last two carry the error bounds of a finite-precision evaluation."""
    q = np.asarray(q, dtype=np.float64)
    total, hq, d = q.shape
    hkv, t = k_cache.shape[1], k_cache.shape[2]
    g = hq // hkv
    out, mag, top = np.zeros(q.shape), np.zeros(q.shape), np.zeros((total, hq))
    at = 0
    for s in range(len(ctx)):
        c, m = int(ctx[s]), int(n[s])
        if m == 0 or c == 0:
            at += m
            continue
        mask = seen(c - m, m, window, sinks)
        pos = np.flatnonzero(mask.any(axis=0))
        mask = mask[:, pos]
        blk = np.array([int(tables[s][p // t]) for p in pos])
        k, v = k_cache[blk, :, pos % t], v_cache[blk, :, pos % t]   # [keys, N_kv, D]
        for j in range(hq):
            x = q[at:at + m, j] @ k[:, j // g].T * softmax_scale
            x = np.where(mask, x, -np.inf)
            w = np.exp(x - x.max(axis=1, keepdims=True))
            w /= w.sum(axis=1, keepdims=True)
            out[at:at + m, j] = w @ v[:, j // g]
            mag[at:at + m, j] = w @ np.abs(v[:, j // g])
            a = np.abs(q[at:at + m, j]) @ np.abs(k[:, j // g]).T * abs(softmax_scale)
            top[at:at + m, j] = np.where(mask, a, 0.0).max(axis=1)
        at += m
    return out, mag, top
