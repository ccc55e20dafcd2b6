"""The scored step from its definitions, in 64 bits (numpy).

Test infrastructure: written apart from the product, one loop per row and
head.  Inputs are float64 arrays (the values that bf16, e4m3 or 8-bit data
stand for) and integer arrays.
"""
from __future__ import annotations

import numpy as np


def normalise(x, weight, eps):
    """RMS norm of each head: x [..., d], weight [d]."""
    out = np.empty_like(x)
    for i in np.ndindex(x.shape[:-1]):
        out[i] = x[i] / np.sqrt(np.mean(x[i] * x[i]) + eps) * weight
    return out


def rows_in_8_bits(x):
    """Codes [..., d] and units [...] of rows x."""
    unit = np.abs(x).max(-1) / 127
    with np.errstate(invalid="ignore", divide="ignore"):
        codes = np.rint(x / unit[..., None])
    return np.where(unit[..., None] == 0, 0, codes), unit


def gather(cache, table, first, end):
    """Tokens first .. end - 1 of one sequence, [tokens, heads, d]; rows of
    blocks outside the pool are NaN."""
    nb, B = cache.shape[:2]
    out = np.full((max(0, end - first), *cache.shape[2:]), np.nan)
    for i, t in enumerate(range(first, end)):
        if 0 <= table[t // B] < nb:
            out[i] = cache[table[t // B], t % B]
    return out


def scores(q, k, scale, cap, slope, pos, at):
    """Changed scores of one query over keys at positions `at`."""
    s = (k @ q) * scale
    if cap:
        s = cap * np.tanh(s / cap)
    if slope is not None:
        s = s - slope * np.abs(pos - at)
    return s


def visible(pos, seq_len, window, prefix):
    """[first, end) of the keys that a query at `pos` sees."""
    end = pos + 1
    if pos < min(prefix, seq_len):
        end = min(prefix, seq_len)
    return (max(0, pos - window + 1) if window else 0), end


def attend(q, pos, seq_len, k_cache, v_cache, table, scale, cap=0.0, window=0, slopes=None,
           prefix=0):
    """One row at position `pos`: (out, sum of p |v| / sum of p, the largest
    sum of |q k scale|), the first two [heads, d].  Tokens of blocks outside
    the pool are passed over."""
    nb, B, hkv, d = k_cache.shape
    heads = q.shape[0]
    out, mag, most = np.zeros((heads, d)), np.zeros((heads, d)), 0.0
    first, end = visible(pos, seq_len, window, prefix)
    at = np.array([t for t in range(first, end) if 0 <= table[t // B] < nb], np.int64)
    if seq_len <= 0 or not len(at):
        return out, mag, most
    block = np.asarray(table)[at // B]
    for h in range(heads):
        g = h // (heads // hkv)
        k, v = k_cache[block, at % B, g], v_cache[block, at % B, g]
        s = scores(q[h], k, scale, cap, None if slopes is None else slopes[h], pos, at)
        p = np.exp(s - s.max())
        out[h], mag[h] = p @ v / p.sum(), p @ np.abs(v) / p.sum()
        most = max(most, float((np.abs(k) @ np.abs(q[h])).max() * abs(scale)))
    return out, mag, most
