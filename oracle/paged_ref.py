"""Rotary positions and the paged key-value cache in float64 NumPy: plain
definitions, one pair, one sequence and one head at a time, the oracle of
attn_paged.h.

Test infrastructure only; nothing here is shared with the CUDA path."""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, orig_len=0, low_turns=1.0, high_turns=32.0):
    """Radians per position of each pair."""
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    out = []
    for i in range(rot_dim // 2):
        w = base ** (-2 * i / rot_dim)
        if scaling == "linear":
            w /= factor
        if scaling == "by_parts":
            turns = orig_len * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low_turns) / (high_turns - low_turns)))
            w = keep * w + (1 - keep) * w / factor
        out.append(w)
    return np.array(out)


def rope(x, pos, inv_freq, interleaved=False, out_scale=1.0, inverse=False):
    """x [..., N, D] with N positions: pair (a, b) of frequency w at position
    p becomes out_scale (a cos - b sin, a sin + b cos) of the angle p w."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(inv_freq)
    for i, w in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = np.asarray(pos, dtype=np.float64) * w * (-1.0 if inverse else 1.0)
        c, s = np.cos(angle) * out_scale, np.sin(angle) * out_scale
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def decode(q, k_pool, v_pool, page_table, seq_lens, sm_scale=None):
    """q [B, Hq, Dqk]; pools [pages, Hkv, page, D].  Returns o, lse."""
    B, Hq, Dqk = q.shape
    Hkv, page = k_pool.shape[1], k_pool.shape[2]
    s = Dqk**-0.5 if sm_scale is None else sm_scale
    o = np.zeros((B, Hq, v_pool.shape[-1]))
    lse = np.full((B, Hq), -np.inf)
    for b in range(B):
        n = int(seq_lens[b])
        if n == 0:
            continue
        at = [(int(page_table[b, p // page]), p % page) for p in range(n)]
        pages, slots = [x[0] for x in at], [x[1] for x in at]
        for h in range(Hq):
            k = np.asarray(k_pool[pages, h // (Hq // Hkv), slots], dtype=np.float64)
            v = np.asarray(v_pool[pages, h // (Hq // Hkv), slots], dtype=np.float64)
            z = s * (k @ np.asarray(q[b, h], dtype=np.float64))
            top = z.max()
            w = np.exp(z - top)
            o[b, h] = w @ v / w.sum()
            lse[b, h] = top + math.log(w.sum())
    return o, lse
