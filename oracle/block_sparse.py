"""The block-sparse decode step from its definitions, in 64 bits (numpy).

Test infrastructure: written apart from the product, one loop per row, head
and block.  Inputs are float64 arrays (the values that bf16 or e4m3 data
stand for) and integer arrays.
"""
from __future__ import annotations

import numpy as np

LIMIT = 2.0 ** 50


def axes_of_pairs(pairs: int, sections, in_turn: bool):
    """The position axis of each pair: sections in a row, or axes in turn
    while they have pairs left (else axis 0)."""
    if not in_turn:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    for i in range(pairs):
        a = i % len(sections)
        if a and left[a] > 0:
            left[a] -= 1
        else:
            a = 0
        out.append(a)
    return out


def rotate(x, cos, sin, adjacent: bool):
    """[heads, d] of one token; cos, sin: [pairs].  Returns the rotated
    channels and, per channel, the sum of the two products' magnitudes."""
    y, mag = x.copy(), np.abs(x)
    p = len(cos)
    for i in range(p):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + p)
        y[:, a] = x[:, a] * cos[i] - x[:, b] * sin[i]
        y[:, b] = x[:, b] * cos[i] + x[:, a] * sin[i]
        mag[:, a] = np.abs(x[:, a] * cos[i]) + np.abs(x[:, b] * sin[i])
        mag[:, b] = np.abs(x[:, b] * cos[i]) + np.abs(x[:, a] * sin[i])
    return y, mag


def rope_rows(x, positions, table, sections, in_turn, adjacent):
    """[N, heads, d] rotated by [axes, N] positions (rows of `table`)."""
    pairs = table.shape[1] // 2
    axis = axes_of_pairs(pairs, sections, in_turn) if len(sections) > 1 else [0] * pairs
    out, mag = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[0]):
        rows = [table[positions[axis[i], t]] for i in range(pairs)]
        cos = np.array([r[i] for i, r in enumerate(rows)])
        sin = np.array([r[pairs + i] for i, r in enumerate(rows)])
        out[t], mag[t] = rotate(x[t], cos, sin, adjacent)
    return out, mag


def power_above(amax: float) -> float:
    """The smallest power of two u >= 2^-50 with amax / u <= 127."""
    u = 2.0 ** -50
    while amax > 127 * u:
        u *= 2
    return u


def block_range(k):
    """Codes [heads, 2, d] and powers [heads] of one block's keys
    [block_size, heads, d] (may hold NaN and infinities)."""
    heads, d = k.shape[1:]
    codes, scales = np.zeros((heads, 2, d), np.int64), np.zeros(heads)
    for h in range(heads):
        hi, lo = np.zeros(d), np.zeros(d)
        for c in range(d):
            v = [min(max(x, -LIMIT), LIMIT) for x in k[:, h, c] if x == x]
            if v:
                hi[c], lo[c] = max(v), min(v)
        u = power_above(max(np.abs(hi).max(), np.abs(lo).max()))
        codes[h, 0], codes[h, 1], scales[h] = np.ceil(hi / u), np.floor(lo / u), u
    return codes, scales


def query_codes(q):
    """8-bit codes and power of one query head."""
    q = np.where(np.isnan(q), 0.0, np.clip(q, -LIMIT, LIMIT))
    u = power_above(np.abs(q).max())
    return np.rint(q / u), u


def select(q, codes, scales, table, n, block_size, top, sink, recent):
    """The selection of one row, [kv_heads, top]; q: [heads, d]; table: the
    row's block table."""
    hkv = codes.shape[1]
    group = q.shape[0] // hkv
    nb = min(-(-max(n, 0) // block_size), len(table))
    out = np.full((hkv, top), -1, np.int64)
    for h in range(hkv):
        if nb <= top:
            out[h, :nb] = np.arange(nb)
            continue
        heads = [query_codes(q[h * group + i]) for i in range(group)]
        score = []
        for j in range(sink, nb - recent):
            if not 0 <= table[j] < codes.shape[0]:
                score.append(-np.inf)
                continue
            hi, lo = codes[table[j], h].astype(np.float64)
            score.append(max(np.maximum(c * hi, c * lo).sum() * u for c, u in heads)
                         * scales[table[j], h])
        best = sorted(range(len(score)), key=lambda i: (-score[i], i))[:top - sink - recent]
        out[h] = np.sort(np.concatenate([np.arange(sink), sink + np.array(best, np.int64),
                                         np.arange(nb - recent, nb)]))
    return out


def decode_selected(q, k_cache, v_cache, table, n, listed, scale):
    """Attention of one row over its listed blocks: (out, sum of p |v| / sum
    of p), both [heads, d].  k_cache, v_cache: float64 [NB, B, Hkv, d]."""
    num_blocks, B, hkv, d = k_cache.shape
    group = q.shape[0] // hkv
    out, mag = np.zeros((q.shape[0], d)), np.zeros((q.shape[0], d))
    for h in range(hkv):
        ks, vs = [], []
        for j in listed[h]:
            if j < 0 or j >= len(table) or not 0 <= table[j] < num_blocks:
                continue
            m = min(B, n - j * B)
            if m > 0:
                ks.append(k_cache[table[j], :m, h])
                vs.append(v_cache[table[j], :m, h])
        if not ks:
            continue
        k, v = np.concatenate(ks), np.concatenate(vs)
        for i in range(h * group, (h + 1) * group):
            x = (k @ q[i]) * scale
            p = np.exp(x - x.max())
            out[i], mag[i] = p @ v / p.sum(), p @ np.abs(v) / p.sum()
    return out, mag
