"""The paged cache made smaller, in float64 NumPy: plain definitions, one
group, one key and one head at a time, the oracle of attn_cache.h.

Test infrastructure only; nothing here is shared with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

MOST = 65504.0


def group_of(d):
    """Elements that share a step and a least value in a row of d."""
    return min(d, 64)


def round4(x):
    """x [..., D] (values that fp32 holds) -> whole numbers [..., D], steps and
    least values [..., groups], by the definition's own fp32 differences and
    quotients and fp16 roundings."""
    x = np.asarray(x, dtype=np.float32)
    d = x.shape[-1]
    size = group_of(d)
    n = np.zeros(x.shape, dtype=np.int64)
    step = np.zeros((*x.shape[:-1], d // size), dtype=np.float16)
    least = np.zeros_like(step)
    for at in np.ndindex(*step.shape):
        g = x[at[:-1]][at[-1] * size:(at[-1] + 1) * size]
        if not np.isfinite(g).all():
            step[at] = least[at] = np.nan
            continue
        g = np.clip(g, np.float32(-MOST), np.float32(MOST))
        least[at] = np.float16(g.min())
        step[at] = np.float16((g.max() - np.float32(least[at])) / np.float32(15))
        if step[at] > 0:
            q = np.rint((g - np.float32(least[at])) / np.float32(step[at]))
            n[at[:-1]][at[-1] * size:(at[-1] + 1) * size] = np.clip(q, 0, 15).astype(np.int64)
    return n, step, least


def values4(n, step, least):
    """m + n s in float64."""
    size = group_of(n.shape[-1])
    s, m = (np.repeat(np.asarray(a, dtype=np.float64), size, axis=-1) for a in (step, least))
    return m + np.asarray(n, dtype=np.float64) * s


def pack4(n):
    """Bytes: element 2i in the low half of byte i."""
    return (n[..., 0::2] | n[..., 1::2] << 4).astype(np.uint8)


def unpack4(b):
    n = np.empty((*b.shape[:-1], 2 * b.shape[-1]), dtype=np.int64)
    n[..., 0::2], n[..., 1::2] = b & 15, b >> 4
    return n


def weights(q, lse, k_pool, page_table, seq_lens, w, sm_scale=None, decay=1.0):
    """q [B, Hq, D], lse [B, Hq], keys [pages, Hkv, page, D], w [B, Hkv, places]."""
    B, Hq, D = q.shape
    Hkv, page = k_pool.shape[1], k_pool.shape[2]
    s = D**-0.5 if sm_scale is None else sm_scale
    out = np.array(w, dtype=np.float64)
    for b in range(B):
        n = int(seq_lens[b])
        for h in range(Hkv if n else 0):
            at = [(int(page_table[b, p // page]), p % page) for p in range(n)]
            k = np.asarray(k_pool[[x[0] for x in at], h, [x[1] for x in at]], dtype=np.float64)
            total = np.zeros(n)
            for i in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                if lse[b, i] != -np.inf:
                    total += np.exp(s * (k @ np.asarray(q[b, i], dtype=np.float64)) - float(lse[b, i]))
            out[b, h, :n] = (decay * out[b, h, :n] if decay else 0.0) + total
    return out


def kept(w, n, keep, sinks=0, recent=0):
    """The places, in order, that a head of n keys with weights w keeps."""
    if n <= keep:
        return list(range(n))
    recent = min(recent, keep)
    sinks = min(sinks, keep - recent)
    others = sorted(range(sinks, n - recent), key=lambda j: (-(math.inf if math.isnan(w[j]) else float(w[j])),
                                                             not math.isnan(w[j]), j))
    return sorted([*range(sinks), *others[:keep - sinks - recent], *range(n - recent, n)])
