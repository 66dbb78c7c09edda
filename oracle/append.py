"""Append with rotation and block-scaled E4M3 caches (oracle, test only).

Sources: the foundry page on paged block allocation, "In and out" (the step
writes the new tokens' K/V into reserved slots).  The pages describe neither a
rotation nor a scale per block; both are plain definitions here:

* rotation: with r = rotary_dim and angles a_i of a token's position (given as
  cosines and sines), pair (x0, x1) of index i becomes (x0 cos a_i - x1 sin a_i,
  x0 sin a_i + x1 cos a_i); pair i is elements (i, i + r/2), or (2i, 2i + 1).
  ``rotate`` works in the precision of its inputs, one rounding per operation;
* block scale: one per (block, KV head).  Appending x to a block sets
  s = max(s_before, 2^e), e the least integer in [-40, 40] with
  amax |x| <= 448 * 2^e over the finite x, s_before counting only where the
  block holds earlier rows; where s grew the earlier values are rounded to E4M3
  again at the new scale.

A cache is a dense array [num_blocks, N_kv, T, D] of E4M3 bytes (or of values
for 16/32-bit caches); a sequence's chunk is its last n positions.
"""
from __future__ import annotations

import math

import numpy as np

from . import e4m3

MIN_EXP, MAX_EXP = -40, 40


def rotate(x, cos_sin, positions, interleaved: bool):
    """x [n, heads, D] rotated by the table rows of its positions, in the
    table's dtype."""
    x = np.array(x, dtype=cos_sin.dtype)
    r = cos_sin.shape[1]
    c = cos_sin[positions][:, None, :r // 2]
    s = cos_sin[positions][:, None, r // 2:]
    i0 = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    i1 = i0 + 1 if interleaved else i0 + r // 2
    x0, x1 = x[..., i0], x[..., i1]
    y0 = x0 * c - x1 * s
    y1 = x0 * s + x1 * c
    x[..., i0], x[..., i1] = y0, y1
    return x


def scale_for(amax: float) -> float:
    """The least power of two s in [2^-40, 2^40] with amax <= 448 s (by search)."""
    for e in range(MIN_EXP, MAX_EXP):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** MAX_EXP


def append_block_scaled(cache, scales, which: int, x, tables, ctx, n):
    """Write x (fp32 rows [sum n, N_kv, D], sequence s's chunk at its rows in
    batch order) into the byte cache and scales [num_blocks, N_kv, 2]."""
    t = cache.shape[2]
    at = 0
    for s in range(len(ctx)):
        c, k = int(ctx[s]), int(n[s])
        for h in range(cache.shape[1]):
            for j in range((c - k) // t, -(-c // t) if k else 0):
                a, z = max(c - k, j * t), min(c, (j + 1) * t)
                blk = int(tables[s][j])
                rows = np.asarray(x[at + a - (c - k):at + z - (c - k), h], dtype=np.float32)
                mag = np.abs(rows[np.isfinite(rows)])
                new = scale_for(float(mag.max()) if mag.size else 0.0)
                if a > j * t:
                    old = float(scales[blk, h, which])
                    if new > old:
                        held = e4m3.decode(cache[blk, h, :a - j * t])
                        cache[blk, h, :a - j * t] = e4m3.encode(held * (old / new))
                    new = max(new, old)
                scales[blk, h, which] = new
                cache[blk, h, a - j * t:z - j * t] = e4m3.encode(rows.astype(np.float64) / new)
        at += k


def append_values(cache, x, tables, ctx, n):
    """Write rows x into a value cache, unscaled."""
    t = cache.shape[2]
    at = 0
    for s in range(len(ctx)):
        for p in range(int(ctx[s]) - int(n[s]), int(ctx[s])):
            cache[int(tables[s][p // t]), :, p % t] = x[at]
            at += 1


def angle_table(max_position: int, rotary_dim: int, base: float = 10000.0):
    """cosines, then sines, of p * base^(-2i / r), fp64 by the math module."""
    r = rotary_dim
    out = np.empty((max_position, r))
    for p in range(max_position):
        for i in range(r // 2):
            a = p * base ** (-2.0 * i / r)
            out[p, i], out[p, r // 2 + i] = math.cos(a), math.sin(a)
    return out
