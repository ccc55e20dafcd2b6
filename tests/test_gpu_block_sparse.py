"""GPU parity of the block-sparse decode step (rotating cache write, block
key ranges, block selection, attention over listed blocks) against the
64-bit oracle.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
* rotation: two products and a sum in fp32, each off by at most u times its
  magnitude, so 3 u (|x c| + |y s|) <= 2^-22 (|x c| + |y s|); then half a
  step of bf16 (2^-8 relative) or e4m3 (2^-4 relative, 2^-10 absolute among
  its subnormals; the quotient by the scale adds u).
* ranges and selections: whole numbers and powers of two, equal.
* attention: a logit is a sum of d <= 128 exact products, off by at most
  (d + 2) u sum |q k| scale; with the tests' N(0, 1) inputs sum |q k| scale
  stays under 16 (where a test scales the keys it says so), so a weight's
  relative error is at most 130 * 16 * 2^-24 < 2^-12.9, plus 2^-16 for its
  two-part rounding and 2^-21 for exp2.  Numerator and denominator both:
  under 2^-11 sum p |v| / sum p in all; then half a step of bf16.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import block_sparse as bs
from oracle import core as ocore
from paged_kv_cache_108_gb300 import ops, synth
from tests import harness

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).to(DEV)


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(DEV).to(torch.bfloat16)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _codes_np(t):
    """float64 values of an e4m3 cache held as uint8 or float8."""
    return t.view(torch.uint8).view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)


def _table(max_position, rot, base=10000.0):
    ang = np.arange(max_position)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _junk_cache(rng, kv, *shape):
    """A pool of random bits (NaN and infinities among them)."""
    if kv == "bf16":
        return _dev(rng.integers(-2 ** 15, 2 ** 15, shape), torch.int16).view(torch.bfloat16)
    return _dev(rng.integers(0, 256, shape), torch.uint8)


# ------------------------------------------------------------ rope_and_cache

ROPE = [
    # tokens, H, Hkv, d, rot, sections, in turn, adjacent, kv
    (1, 32, 8, 128, 128, None, False, False, "bf16"),
    (1, 1, 1, 64, 16, None, False, True, "fp8"),
    (3, 4, 2, 64, 64, None, False, True, "bf16"),
    (37, 4, 2, 64, 32, [4, 6, 6], False, False, "fp8"),
    (37, 4, 2, 64, 32, [6, 5, 5], True, True, "bf16"),
    (65, 32, 8, 128, 128, [16, 24, 24], False, False, "fp8"),
    (65, 8, 8, 128, 112, [20, 18, 18], True, False, "bf16"),
    (130, 7, 3, 128, 48, [7, 9, 5, 3], False, True, "bf16"),
    (130, 5, 1, 64, 64, [32, 0], False, False, "fp8"),
    (301, 2, 2, 64, 48, [0, 24], False, False, "bf16"),
    (41, 96, 16, 128, 128, None, False, False, "fp8"),
]


def _rope_case(tokens, H, Hkv, d, rot, sections, in_turn, adjacent, kv, seed=0, max_position=5000):
    rng = np.random.default_rng(seed)
    B, NB = 16, tokens // 16 + 3
    axes = 1 if sections is None else len(sections)
    qkv = _bf16(rng, tokens, (H + 2 * Hkv) * d)
    c = dict(q=qkv[:, :H * d].view(tokens, H, d), k=qkv[:, H * d:(H + Hkv) * d].view(tokens, Hkv, d),
             v=qkv[:, (H + Hkv) * d:].view(tokens, Hkv, d))
    slots = rng.permutation(NB * B)[:tokens]
    if tokens > 8:
        slots[[2, 5]] = [-1, NB * B]  # padding and a slot past the pool
    pos = rng.integers(0, max_position, (axes, tokens))
    pos[:, 0] = max_position - 1
    c.update(slots=slots, pos=pos, table=_table(max_position, rot), sections=sections or [rot // 2],
             kc=_junk_cache(rng, kv, NB, B, Hkv, d), vc=_junk_cache(rng, kv, NB, B, Hkv, d),
             in_turn=in_turn, adjacent=adjacent, kv=kv, ks=None, vs=None)
    if kv == "fp8":
        c.update(ks=_dev([0.0117], torch.float32), vs=_dev([0.5 / 448], torch.float32))  # v saturates
    return c


def _rope_run(c, out=None, q=None, stream=None):
    out = torch.full_like(c["q"], 7.0, memory_format=torch.contiguous_format) if out is None else out
    pos = _dev(c["pos"] if c["pos"].shape[0] > 1 else c["pos"][0])
    ops.rope_and_cache(out, c["q"] if q is None else q, c["k"], c["v"], c["kc"], c["vc"],
                       _dev(c["slots"]), pos, _dev(c["table"], torch.float32), c["ks"], c["vs"],
                       sections=c["sections"], sections_in_turn=c["in_turn"],
                       adjacent_pairs=c["adjacent"], stream=stream)
    return out


def _check_rope(c, out, kc0, vc0, skipped=()):
    N = c["q"].shape[0]
    pos = c["pos"].copy()
    pos[:, list(skipped)] = 0
    args = (pos, c["table"].astype(np.float64), c["sections"], c["in_turn"], c["adjacent"])
    want, mag = bs.rope_rows(_np(c["q"]), *args)
    keep = [t for t in range(N) if t not in skipped]
    err = np.abs(_np(out) - want)[keep]
    assert (err <= 2 ** -8 * np.abs(want[keep]) + 2 ** -22 * mag[keep]).all()
    assert (_np(out)[list(skipped)] == 7.0).all()
    want, mag = bs.rope_rows(_np(c["k"]), *args)
    slots = c["slots"]
    hit = [t for t in keep if 0 <= slots[t] < kc0.shape[0] * kc0.shape[1]]
    flat = lambda t: t.view(-1, *t.shape[2:])  # noqa: E731
    if c["kv"] == "bf16":
        err = np.abs(_np(flat(c["kc"]))[slots[hit]] - want[hit])
        assert (err <= 2 ** -8 * np.abs(want[hit]) + 2 ** -22 * mag[hit]).all()
    else:
        s = float(c["ks"].item())
        w = np.clip(want[hit] / s, -448, 448)
        err = np.abs(_codes_np(flat(c["kc"]))[slots[hit]] - w)
        assert (err <= np.maximum(2 ** -4 * np.abs(w), 2 ** -10) + 2 ** -21 * mag[hit] / s).all()
    # values: the plain write's bits; slots not named: as they were
    rk, rv = harness.bits_from_dev(kc0).copy(), harness.bits_from_dev(vc0).copy()
    masked = np.full(N, -1, np.int32)
    masked[hit] = slots[hit]
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    ocore.reshape_and_cache(bits(c["k"]), bits(c["v"]), rk, rv, masked,
                            1.0 if c["ks"] is None else float(c["ks"].item()),
                            1.0 if c["vs"] is None else float(c["vs"].item()))
    assert np.array_equal(harness.bits_from_dev(c["vc"]), rv)
    untouched = np.ones(kc0.shape[0] * kc0.shape[1], bool)
    untouched[slots[hit]] = False
    assert np.array_equal(harness.bits_from_dev(flat(c["kc"]))[untouched],
                          harness.bits_from_dev(flat(kc0))[untouched])


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_rope_and_cache(case):
    c = _rope_case(*case)
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    out = _rope_run(c)
    _check_rope(c, out, kc0, vc0)


@pytest.mark.parametrize("tokens,H,Hkv,rot", [(2501, 45, 3, 16), (2500, 6, 1, 16), (700, 3, 1, 32)])
def test_rope_long_calls(tokens, H, Hkv, rot):
    # two tokens a CTA, the last one alone; several of few heads
    c = _rope_case(tokens, H, Hkv, 64, rot, None, False, False, "bf16", seed=6)
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    _check_rope(c, _rope_run(c), kc0, vc0)


def test_rope_skips_tokens_with_a_position_outside_the_table():
    c = _rope_case(20, 4, 2, 64, 32, [4, 6, 6], False, False, "bf16", seed=3)
    c["pos"][1, 4], c["pos"][0, 9], c["pos"][2, 19] = -1, 5000, 2 ** 31 - 1
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    out = _rope_run(c)
    _check_rope(c, out, kc0, vc0, skipped=(4, 9, 19))


def test_rope_in_place_equals_out_of_place_and_no_query_heads():
    c = _rope_case(77, 8, 2, 128, 64, None, False, False, "bf16", seed=4)
    kc, vc = c["kc"].clone(), c["vc"].clone()
    want = _rope_run(c)
    k_bits = c["kc"].view(torch.int16).clone()
    c["kc"], c["vc"] = kc, vc
    q = c["q"].contiguous()
    _rope_run(c, out=q, q=q)
    assert torch.equal(q, want) and torch.equal(kc.view(torch.int16), k_bits)
    c["kc"] = kc.clone()
    none = torch.empty(77, 0, 128, device=DEV, dtype=torch.bfloat16)
    _rope_run(c, out=none, q=none)
    assert torch.equal(c["kc"].view(torch.int16), k_bits)


def test_rope_far_positions_and_no_tokens():
    # rows past 2^31 bytes of the table: 2^25 + 9 positions of 16 channels
    c = _rope_case(5, 2, 1, 64, 16, None, False, False, "bf16", seed=5, max_position=50)
    rows = 2 ** 25 + 9
    table = torch.zeros(rows, 16, device=DEV)
    tail = _table(50, 16)
    table[-50:] = _dev(tail, torch.float32)
    out = torch.empty(5, 2, 64, device=DEV, dtype=torch.bfloat16)
    ops.rope_and_cache(out, c["q"], c["k"], c["v"], c["kc"], c["vc"], _dev(c["slots"]),
                       _dev(c["pos"][0] + rows - 50), table)
    want, mag = bs.rope_rows(_np(c["q"]), c["pos"], tail.astype(np.float64), [8], False, False)
    assert (np.abs(_np(out) - want) <= 2 ** -8 * np.abs(want) + 2 ** -22 * mag).all()
    z = lambda *s: torch.empty(*s, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    ops.rope_and_cache(z(0, 2, 64), z(0, 2, 64), z(0, 1, 64), z(0, 1, 64), c["kc"], c["vc"],
                       _dev([]), _dev([]), table)


# --------------------------------------------------------- summarize_blocks

@pytest.mark.parametrize("B", [1, 2, 8, 16, 32, 128, 1024])
@pytest.mark.parametrize("Hkv,d,kv", [(1, 64, "fp8"), (3, 64, "bf16"), (8, 128, "bf16"), (5, 128, "fp8")])
def test_summarize_blocks(B, Hkv, d, kv):
    rng = np.random.default_rng(B + Hkv)
    NB = 7 if B < 1024 else 3
    if kv == "bf16":
        k = (rng.standard_normal((NB, B, Hkv, d)) * 10.0 ** rng.integers(-8, 8, (NB, 1, Hkv, 1))).astype(np.float32)
        kc = torch.from_numpy(k).to(DEV).to(torch.bfloat16)
        kc[0, :, 0, 3] = float("nan")          # a channel without a number
        kc[0, B // 2, 0, 5] = float("nan")
        kc[1, 0, -1, 1] = float("inf")
        kc[1, B - 1, 0, 2] = float("-inf")
        kc[2, :, 0] = 0.0                      # a head of zeros
        kc[2, 0, -1] = 1e-30 if B > 1 else 0.0  # far below the least power
        values = _np(kc)
    else:
        kc = _junk_cache(rng, "fp8", NB, B, Hkv, d)  # every code, NaN among them
        values = _codes_np(kc)
    full = [0, 1, 2][:NB] + ([5] if NB > 5 else [])
    slots = [b * B + B - 1 for b in full] + [-1, -B, NB * B + B - 1, full[0] * B + B - 1]
    if B > 1:
        slots += [4 % NB * B + B - 2] if NB > 4 else []
        slots += [B // 2]
    codes, scales = ops.alloc_block_ranges(kc)
    codes.fill_(55)
    scales.fill_(-3.0)
    ops.summarize_blocks(kc, _dev(rng.permutation(slots)), codes, scales)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    for b in range(NB):
        if b in full:
            want, u = bs.block_range(values[b])
            assert np.array_equal(scales[b], u), b
            assert np.array_equal(codes[b], want), b
        else:
            assert (codes[b] == 55).all() and (scales[b] == -3.0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,tokens", [(4, 2049), (16, 5000), (64, 1500)])
def test_summarize_a_prompt(B, tokens, kv):
    rng = np.random.default_rng(tokens)
    NB, Hkv, d = -(-tokens // B), 2, 64
    kc = _bf16(rng, NB, B, Hkv, d) if kv == "bf16" else _junk_cache(rng, kv, NB, B, Hkv, d)
    order = rng.permutation(NB)
    slots = order[np.arange(tokens) // B] * B + np.arange(tokens) % B
    codes, scales = ops.alloc_block_ranges(kc)
    ops.summarize_blocks(kc, _dev(slots), codes, scales)
    values = _np(kc) if kv == "bf16" else _codes_np(kc)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    for b in range(NB):
        if b == order[-1] and tokens % B:
            assert (scales[b] == 0).all() and (codes[b] == 0).all()
        elif b % max(1, NB // 40) == 0:
            want, u = bs.block_range(values[b])
            assert np.array_equal(codes[b], want) and np.array_equal(scales[b], u)


# ------------------------------------------------------------ select_blocks

def _ranges(rng, NB, Hkv, d):
    a, b = rng.integers(-127, 128, (2, NB, Hkv, d))
    codes = np.stack([np.maximum(a, b), np.minimum(a, b)], 2).astype(np.int8)
    scales = 2.0 ** rng.integers(-7, -4, (NB, Hkv))
    return codes, scales.astype(np.float32)


def _tables(rng, lens, B, NB, width=None):
    width = width or max(1, max(-(-max(n, 0) // B) for n in lens))
    t = np.zeros((len(lens), width), np.int32)
    for i in range(len(lens)):
        t[i] = rng.integers(0, NB, width)
    return t


def _check_select(rng, lens, G, Hkv, d, B, top, sink=1, recent=1, row_seqs=None, NB=97, q=None,
                  codes=None, tables=None, seqs=None):
    H = G * Hkv
    rows = len(lens)
    c, s = _ranges(rng, NB, Hkv, d) if codes is None else codes
    if tables is None:
        need = max(1, max(-(-max(n, 0) // B) for n in lens))
        tables = rng.integers(0, NB, (seqs or rows, need)).astype(np.int32)
    q = _bf16(rng, rows, H, d) if q is None else q
    sel = torch.full((rows, Hkv, top), 12345, device=DEV, dtype=torch.int32)
    ops.select_blocks(sel, q, _dev(c, torch.int8), _dev(s, torch.float32), _dev(tables), _dev(lens), B,
                      sink=sink, recent=recent, row_seqs=None if row_seqs is None else _dev(row_seqs))
    got, qv = sel.cpu().numpy(), _np(q)
    for r in range(rows):
        sq = r if row_seqs is None else row_seqs[r]
        if not 0 <= sq < len(tables):
            assert (got[r] == -1).all()
            continue
        want = bs.select(qv[r], c, s.astype(np.float64), tables[sq], int(lens[r]), B, top, sink, recent)
        assert np.array_equal(got[r], want), (r, lens[r])
    return got


@pytest.mark.parametrize("G,Hkv,d", [(1, 3, 64), (2, 2, 128), (4, 2, 128), (8, 1, 64), (8, 2, 128), (4, 1, 64)])
@pytest.mark.parametrize("B,top", [(1, 5), (8, 7), (16, 16), (64, 33)])
def test_select_blocks(G, Hkv, d, B, top):
    rng = np.random.default_rng(G * 1000 + d + B)
    lens = [0, -3, 1, B, B * top, B * top + 1, B * (top + 1), B * 90 - 1, B * 91, B * 200 + B // 2]
    _check_select(rng, lens, G, Hkv, d, B, top)
    _check_select(rng, lens, G, Hkv, d, B, top, sink=0, recent=top)
    _check_select(rng, lens, G, Hkv, d, B, top, sink=2, recent=2)


@pytest.mark.parametrize("rows,blocks,top", [(1, 8192, 256), (1, 4000, 3999), (3, 1025, 3), (2, 20001, 1000),
                                             (40, 700, 64)])
def test_select_among_many(rows, blocks, top):
    rng = np.random.default_rng(blocks)
    lens = [blocks * 16 - 7 * r for r in range(rows)]
    _check_select(rng, lens, 4, 2, 128, 16, top, NB=500)


@pytest.mark.parametrize("G,rows,Hkv,blocks", [(1, 310, 4, 40), (2, 310, 4, 33), (4, 310, 4, 20),
                                               (2, 160, 4, 45), (8, 160, 4, 25), (4, 90, 4, 50),
                                               (1, 40, 8, 60), (4, 30, 2, 1100), (2, 70, 4, 530)])
def test_select_launch_shapes(G, rows, Hkv, blocks):
    # from a warp a unit up to several CTAs a unit
    rng = np.random.default_rng(rows + G)
    lens = [max(1, (blocks - r % 7) * 16 - r) for r in range(rows)]
    if blocks > 500:  # the oracle's time goes by the long rows
        lens = [n if r % 9 == 0 else n % 300 for r, n in enumerate(lens)]
    _check_select(rng, lens, G, Hkv, 64, 16, 11, NB=211)


def test_select_from_the_widest_table():
    rng = np.random.default_rng(41)
    _check_select(rng, [196608 * 16 - 5], 1, 1, 64, 16, 300, NB=500)
    # a wide table of short rows, enough rows that a CTA is two warps
    tables = rng.integers(0, 97, (700, 4000)).astype(np.int32)
    _check_select(rng, [16 * (r % 30) + 3 for r in range(700)], 1, 1, 64, 16, 9, tables=tables)


@pytest.mark.parametrize("rows,blocks", [(1, 4096), (70, 150)])
def test_select_ties_go_to_the_lowest_index(rows, blocks):
    rng = np.random.default_rng(7)
    lens = [blocks * 16] * rows
    c = np.zeros((40, 2, 2, 64), np.int8)
    s = np.ones((40, 2), np.float32)
    # every score 0
    got = _check_select(rng, lens, 2, 2, 64, 16, 20, codes=(c, s), NB=40)
    assert got[0, 0].tolist() == list(range(19)) + [blocks - 1]
    # three values, most of them equal
    c[::3, :, 0] = 1
    c[7, :, 0] = 2
    _check_select(rng, lens, 2, 2, 64, 16, 33, codes=(c, s), NB=40)


def test_select_odd_values():
    rng = np.random.default_rng(8)
    lens = [16 * 50] * 8
    q = _bf16(rng, 8, 4, 64)
    q[0] = 0.0
    q[1, 0] = float("nan")
    q[2, 1, 3] = float("inf")
    q[3, 2, 9] = float("-inf")
    q[4] *= 1e30
    q[5] *= 1e-38
    q[6, :, 1:] = 0.0
    tables = rng.integers(0, 97, (8, 50)).astype(np.int32)
    tables[7, 5:40:3] = [-1, 97, 2 ** 31 - 1, -2 ** 31] * 3  # blocks outside the pool
    c, s = _ranges(rng, 97, 2, 64)
    s[::5] = 2.0 ** 44
    s[1::5] = 2.0 ** -50
    _check_select(rng, lens, 2, 2, 64, 16, 11, q=q, codes=(c, s), tables=tables)
    _check_select(rng, lens, 2, 2, 64, 16, 45, q=q, codes=(c, s), tables=tables)


@pytest.mark.parametrize("G,d", [(1, 128), (4, 128), (8, 128), (8, 64)])
def test_select_largest_codes(G, d):
    # sums at the ends of their range, a unit apart: no rounding may show
    rng = np.random.default_rng(40)
    lens = [16 * 60] * 3
    q = torch.full((3, 2 * G, d), 127.0, device=DEV, dtype=torch.bfloat16)
    q[1] = -127.0
    q[2, :, ::2] = -127.0
    c = np.empty((90, 2, 2, d), np.int8)
    c[:, :, 0], c[:, :, 1] = 127, 126
    c[30:60, :, 0], c[30:60, :, 1] = -126, -127
    for b in range(90):  # each block a unit or two from the next
        c[b, :, :, rng.integers(0, d, b % 7)] -= 1 if b < 30 or b >= 60 else -1
    c[:, :, 1] = np.minimum(c[:, :, 0], c[:, :, 1])
    s = np.ones((90, 2), np.float32)
    _check_select(rng, lens, G, 2, d, 16, 13, q=q, codes=(c, s), NB=90)


def test_select_rows_of_one_sequence_and_cut_lengths():
    rng = np.random.default_rng(9)
    lens = [700, 701, 702, 33, 34, 10 ** 9, 2 ** 31 - 1, 50, 60]
    _check_select(rng, lens, 4, 2, 128, 16, 12, row_seqs=[0, 0, 0, 2, 2, 1, 1, -1, 3], seqs=3,
                  tables=rng.integers(0, 97, (3, 60)).astype(np.int32))
    z = lambda *s: torch.empty(*s, device=DEV, dtype=torch.int32)  # noqa: E731
    ops.select_blocks(z(0, 2, 4), torch.empty(0, 4, 64, device=DEV, dtype=torch.bfloat16),
                      torch.zeros(5, 2, 2, 64, device=DEV, dtype=torch.int8),
                      torch.zeros(5, 2, device=DEV), z(0, 3), z(0), 16)


# ---------------------------------------------------------- decode_selected

def _check_attend(rng, lens, listed, G, Hkv, d, B, kv, tables=None, row_seqs=None, NB=None, key=1.0,
                  scale=None):
    """listed: [rows][Hkv][top].  Every slot that no row may see holds random
    bits, NaN and infinities among them."""
    rows, H = len(lens), G * Hkv
    width = max(1, max(-(-max(n, 0) // B) for n in lens)) if tables is None else tables.shape[1]
    if tables is None:
        NB = rows * width + 3
        tables = rng.permutation(NB)[:rows * width].reshape(rows, width).astype(np.int32)
    kc, vc = _junk_cache(rng, kv, NB, B, Hkv, d), _junk_cache(rng, kv, NB, B, Hkv, d)
    ks = vs = None
    kscale = vscale = 1.0
    if kv == "fp8":
        kscale, vscale = 0.0117, 0.0093
        ks, vs = _dev([kscale], torch.float32), _dev([vscale], torch.float32)
    for r in range(rows):
        sq = r if row_seqs is None else row_seqs[r]
        if not 0 <= sq < len(tables):
            continue
        n = min(max(int(lens[r]), 0), width * B)
        for j in range(-(-n // B)):
            b, m = tables[sq, j], min(B, n - j * B)
            if not 0 <= b < NB:
                continue
            for cache, f, sc in ((kc, key, kscale), (vc, 1.0, vscale)):
                x = torch.from_numpy((rng.standard_normal((m, Hkv, d)) * f).astype(np.float32)).to(DEV)
                cache[b, :m] = x.to(torch.bfloat16) if kv == "bf16" else \
                    (x / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    q = _bf16(rng, rows, H, d)
    out = torch.full_like(q, 9.0)
    scale = d ** -0.5 if scale is None else scale
    args = (q, kc, vc, _dev(tables), _dev(lens), _dev(listed), scale, ks, vs)
    ops.decode_selected(out, *args, row_seqs=None if row_seqs is None else _dev(row_seqs))
    kv_np = [(_np(x) if kv == "bf16" else _codes_np(x) * s) for x, s in ((kc, np.float32(kscale)), (vc, np.float32(vscale)))]
    got, qv = _np(out), _np(q)
    for r in range(rows):
        sq = r if row_seqs is None else row_seqs[r]
        if not 0 <= sq < len(tables):
            assert (got[r] == 0).all()
            continue
        want, mag = bs.decode_selected(qv[r], *kv_np, tables[sq], int(lens[r]), listed[r], scale)
        err = np.abs(got[r] - want)
        assert (err <= 2 ** -8 * np.abs(want) + 2 ** -11 * mag).all(), (r, err.max())
    return out, args


def _lists(rng, lens, Hkv, B, top, width=None):
    out = np.full((len(lens), Hkv, top), -1, np.int64)
    for r, n in enumerate(lens):
        nb = -(-max(int(n), 0) // B)
        if width:
            nb = min(nb, width)
        for h in range(Hkv):
            k = min(top, nb)
            out[r, h, :k] = np.sort(rng.permutation(nb)[:k])
            if nb > top:
                out[r, h, top - 1] = nb - 1
    return out


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("G,Hkv,d", [(1, 3, 128), (2, 2, 64), (4, 2, 128), (8, 1, 128), (8, 2, 64), (4, 3, 64),
                                     (1, 2, 64), (2, 1, 128)])
@pytest.mark.parametrize("B,top", [(1, 40), (8, 9), (16, 20), (128, 3), (1024, 2)])
def test_decode_selected(B, top, G, Hkv, d, kv):
    rng = np.random.default_rng(B + G + d)
    lens = [0, 1, B, B + 1, 15, 16, 17, 3 * B - 1, 5 * B + B // 2, -4]
    _check_attend(rng, lens, _lists(rng, lens, Hkv, B, top), G, Hkv, d, B, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("rows,blocks,top", [(1, 300, 200), (1, 70, 64), (2, 130, 90), (9, 60, 31),
                                             (50, 40, 33), (30, 50, 48), (25, 60, 56), (21, 64, 60),
                                             (1, 430, 400)])
def test_decode_selected_shared_by_a_cluster(rows, blocks, top, kv):
    rng = np.random.default_rng(blocks)
    lens = [blocks * 16 - 5 - 9 * r for r in range(rows)]
    _check_attend(rng, lens, _lists(rng, lens, 2, 16, top), 4, 2, 128, 16, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,rows,G", [(1, 2, 4), (4, 1, 8), (2, 7, 1)])
def test_decode_selected_longest_lists(B, rows, G, kv):
    rng = np.random.default_rng(42)
    lens = [4500 * B - 3 * r for r in range(rows)]
    _check_attend(rng, lens, _lists(rng, lens, 1, B, 4096), G, 1, 64, B, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decode_selected_any_order_gaps_repeats_and_strangers(kv):
    rng = np.random.default_rng(11)
    lens = [16 * 6 - 3] * 7
    tables = rng.permutation(60)[:7 * 6].reshape(7, 6).astype(np.int32)
    tables[6, [1, 4]] = [-1, 60]  # outside the pool
    lists = np.full((7, 2, 9), -1)
    lists[0, :, :4] = [5, 0, 3, 2]                  # the partial block first
    lists[1, :, 2:8] = [4, -1, -7, 1, 5, -1]        # gaps
    lists[2, :, :5] = [2, 2, 5, 5, 5]               # listed twice, thrice
    lists[3, :, :6] = [6, 7, 2 ** 31 - 1, 2 ** 27, 1, -2 ** 31]  # past the end
    lists[4, 0, 8] = 3                              # one head has one entry, the last
    lists[6, :, :6] = [0, 1, 2, 3, 4, 5]
    out, _ = _check_attend(rng, lens, lists, 4, 2, 128, 16, kv, tables=tables, NB=60)
    assert (out[5] == 0).all() and (out[4, 4:] == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decode_selected_several_rows_of_a_sequence(kv):
    rng = np.random.default_rng(12)
    tables = rng.permutation(40)[:20].reshape(2, 10).astype(np.int32)
    rows = [0, 0, 0, 1, 1, -1, 2]
    lens = [150, 150, 150, 77, 77, 80, 80]
    lists = _lists(rng, lens, 3, 16, 6)
    _check_attend(rng, lens, lists, 2, 3, 64, 16, kv, tables=tables, NB=40, row_seqs=rows)
    # a row that ends inside a block that its sequence has filled further
    lens2 = np.array(lens) - [40, 17, 0, 30, 0, 0, 0]
    q = _bf16(rng, 7, 6, 64)
    kc, vc = _bf16(rng, 40, 16, 3, 64), _bf16(rng, 40, 16, 3, 64)
    out = torch.empty_like(q)
    ops.decode_selected(out, q, kc, vc, _dev(tables), _dev(lens2), _dev(lists), 0.125, row_seqs=_dev(rows))
    for r in range(5):
        want, mag = bs.decode_selected(_np(q)[r], _np(kc), _np(vc), tables[rows[r]], int(lens2[r]), lists[r], 0.125)
        assert (np.abs(_np(out)[r] - want) <= 2 ** -8 * np.abs(want) + 2 ** -11 * mag).all()


def test_decode_selected_steep_and_flat_logits():
    rng = np.random.default_rng(13)
    lens = [16 * 20 - 1] * 3
    lists = _lists(rng, lens, 2, 16, 20)
    _check_attend(rng, lens, lists, 4, 2, 128, 16, "bf16", scale=0.0)    # the mean
    _check_attend(rng, lens, lists, 8, 2, 128, 16, "bf16", scale=-0.05)
    # keys 2^6 larger at 2^-6 the scale: the same logits
    _check_attend(rng, lens, lists, 4, 2, 64, 16, "bf16", key=64.0, scale=0.125 / 64)


def test_decode_selected_of_every_block_is_decode():
    rng = np.random.default_rng(14)
    S, H, Hkv, d, B, width = 5, 32, 8, 128, 16, 21
    lens = np.array([1, 16, 17, 200, 336], np.int32)
    tables = rng.permutation(S * width).reshape(S, width).astype(np.int32)
    kc, vc = _bf16(rng, S * width, B, Hkv, d), _bf16(rng, S * width, B, Hkv, d)
    q = _bf16(rng, S, H, d)
    a, b = torch.empty_like(q), torch.empty_like(q)
    ws = ops.alloc_workspace(S, H, d, width, B)
    ops.decode(a, q, kc, vc, _dev(tables), _dev(lens), d ** -0.5, workspace=ws)
    every = np.broadcast_to(np.arange(width), (S, Hkv, width))
    ops.decode_selected(b, q, kc, vc, _dev(tables), _dev(lens), _dev(every), d ** -0.5)
    # each within the bf16 decode tolerance of the true value
    assert ((a.float() - b.float()).abs() <= 2 * (1e-2 + 2e-2 * a.float().abs())).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_cache_beyond_32_bit_offsets(kv):
    # K and V of over 2^32 bytes each; the blocks in use are at both ends
    Hkv, d, B = 8, 128, 16
    NB = 2 ** 32 // (B * Hkv * d * (2 if kv == "bf16" else 1)) + 5
    rng = np.random.default_rng(30)
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    kc, vc = (torch.zeros(NB, B, Hkv, d, device=DEV, dtype=dt) for _ in range(2))
    ks, vs = (None, None) if kv == "bf16" else (_dev([0.02], torch.float32), _dev([0.02], torch.float32))
    table = np.array([[NB - 1, 0, NB - 2, NB // 2 + 1]], np.int32)
    n = 61
    p = np.arange(n)
    slots = _dev(table[0, p // B] * B + p % B)
    x = _bf16(rng, n, 16 + 2 * Hkv, d)
    q_out = torch.empty(n, 16, d, device=DEV, dtype=torch.bfloat16)
    tab = _table(100, d)
    ops.rope_and_cache(q_out, x[:, :16], x[:, 16:16 + Hkv], x[:, 16 + Hkv:], kc, vc, slots, _dev(p),
                       _dev(tab, torch.float32), ks, vs)
    codes, scales = ops.alloc_block_ranges(kc)
    ops.summarize_blocks(kc, slots, codes, scales)
    used = [int(b) for b in table[0]]
    small = lambda t: torch.stack([t[b] for b in used])  # noqa: E731
    k, v = ((_np(small(t)) if kv == "bf16" else _codes_np(small(t))) for t in (kc, vc))
    want, mag = bs.rope_rows(_np(x[:, 16:16 + Hkv]), p[None], tab.astype(np.float64), [64], False, False)
    got = k.reshape(-1, Hkv, d)[:n] * (1.0 if kv == "bf16" else float(ks.item()))
    step = 2 ** -8 * np.abs(want) if kv == "bf16" else np.maximum(2 ** -4 * np.abs(want), 2 ** -10 * 0.02)
    assert (np.abs(got - want) <= step + 2 ** -21 * mag).all()
    for i, b in enumerate(used[:3]):
        c, u = bs.block_range(k[i])
        assert np.array_equal(codes[b].cpu().numpy(), c) and np.array_equal(scales[b].cpu().numpy(), u)
    q, sel = q_out[-1:].contiguous(), torch.empty(1, Hkv, 3, device=DEV, dtype=torch.int32)
    ops.select_blocks(sel, q, codes, scales, _dev(table), _dev([n]), B)
    cs = np.stack([codes[b].cpu().numpy() for b in used])
    us = np.stack([scales[b].cpu().numpy() for b in used]).astype(np.float64)
    assert np.array_equal(sel[0].cpu().numpy(), bs.select(_np(q)[0], cs, us, [0, 1, 2, 3], n, B, 3, 1, 1))
    out = torch.empty_like(q)
    ops.decode_selected(out, q, kc, vc, _dev(table), _dev([n]), sel, d ** -0.5, ks, vs)
    if kv == "fp8":
        k, v = k * float(ks.item()), v * float(vs.item())
    want, mag = bs.decode_selected(_np(q)[0], k, v, [0, 1, 2, 3], n, sel[0].cpu().numpy(), d ** -0.5)
    assert (np.abs(_np(out)[0] - want) <= 2 ** -8 * np.abs(want) + 2 ** -11 * mag).all()


# ------------------------------------------------------------- the whole step

class _Step:
    """Several decode steps of a small batch on one cache: the product's four
    calls, and the oracle on the product's own cache, ranges and queries (each
    call's inputs are what the call before it wrote)."""

    def __init__(self, kv, seed=0, S=3, start=(255, 100, 30)):
        rng = self.rng = np.random.default_rng(seed)
        self.S, self.H, self.Hkv, self.d, self.B, self.top = S, 8, 2, 128, 16, 5
        self.kv = kv
        width, NB = 20, 70
        self.tables = rng.permutation(NB)[:S * width].reshape(S, width).astype(np.int32)
        self.lens = np.array(start, np.int32)
        self.kc = _junk_cache(rng, kv, NB, self.B, self.Hkv, self.d)
        self.vc = _junk_cache(rng, kv, NB, self.B, self.Hkv, self.d)
        self.ks = self.vs = None
        if kv == "fp8":
            self.ks, self.vs = _dev([0.02], torch.float32), _dev([0.02], torch.float32)
        self.codes, self.scales = ops.alloc_block_ranges(self.kc)
        self.table = _dev(_table(400, self.d), torch.float32)
        # the step's buffers
        self.bt = _dev(self.tables)
        self.cl = _dev(self.lens)
        self.slots = _dev(np.zeros(S))
        self.pos = _dev(np.zeros(S))
        self.qkv = torch.empty(S, (self.H + 2 * self.Hkv) * self.d, device=DEV, dtype=torch.bfloat16)
        self.q = torch.empty(S, self.H, self.d, device=DEV, dtype=torch.bfloat16)
        self.sel = torch.empty(S, self.Hkv, self.top, device=DEV, dtype=torch.int32)
        self.out = torch.empty_like(self.q)
        self._prefill()

    def _prefill(self):
        for i, n in enumerate(self.lens):
            p = np.arange(n)
            slots = self.tables[i, p // self.B] * self.B + p % self.B
            x = _bf16(self.rng, int(n), self.H + 2 * self.Hkv, self.d)
            self._append(torch.empty(int(n), self.H, self.d, device=DEV, dtype=torch.bfloat16), x,
                         _dev(slots), _dev(p))

    def _append(self, q_out, x, slots, pos):
        H, K = self.H, self.Hkv
        ops.rope_and_cache(q_out, x[:, :H], x[:, H:H + K], x[:, H + K:], self.kc, self.vc, slots, pos,
                           self.table, self.ks, self.vs)
        ops.summarize_blocks(self.kc, slots, self.codes, self.scales)

    def stage(self):
        """The next token of every sequence."""
        self.lens = self.lens + 1
        p = self.lens - 1
        self.cl.copy_(_dev(self.lens))
        self.pos.copy_(_dev(p))
        self.slots.copy_(_dev(self.tables[np.arange(self.S), p // self.B] * self.B + p % self.B))
        self.qkv.copy_(_bf16(self.rng, *self.qkv.shape))

    def run(self):
        x = self.qkv.view(self.S, -1, self.d)
        self._append(self.q, x, self.slots, self.pos)
        ops.select_blocks(self.sel, self.q, self.codes, self.scales, self.bt, self.cl, self.B)
        ops.decode_selected(self.out, self.q, self.kc, self.vc, self.bt, self.cl, self.sel,
                            self.d ** -0.5, self.ks, self.vs)

    def check(self):
        torch.cuda.synchronize()
        k, v = ((_np(x) if self.kv == "bf16" else _codes_np(x)) for x in (self.kc, self.vc))
        codes, scales = self.codes.cpu().numpy(), self.scales.cpu().numpy().astype(np.float64)
        for i in range(self.S):
            for j in range(self.lens[i] // self.B):
                want, u = bs.block_range(k[self.tables[i, j]])
                assert np.array_equal(codes[self.tables[i, j]], want)
                assert np.array_equal(scales[self.tables[i, j]], u)
        x = _np(self.qkv).reshape(self.S, -1, self.d)[:, :self.H]
        want, mag = bs.rope_rows(x, self.lens[None] - 1, self.table.double().cpu().numpy(), [64], False, False)
        assert (np.abs(_np(self.q) - want) <= 2 ** -8 * np.abs(want) + 2 ** -22 * mag).all()
        if self.kv == "fp8":
            k, v = k * float(self.ks.item()), v * float(self.vs.item())
        sel, q, out = self.sel.cpu().numpy(), _np(self.q), _np(self.out)
        for i in range(self.S):
            want = bs.select(q[i], codes, scales, self.tables[i], int(self.lens[i]), self.B, self.top, 1, 1)
            assert np.array_equal(sel[i], want)
            want, mag = bs.decode_selected(q[i], k, v, self.tables[i], int(self.lens[i]), sel[i], self.d ** -0.5)
            assert (np.abs(out[i] - want) <= 2 ** -8 * np.abs(want) + 2 ** -11 * mag).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_steps_eager(kv):
    s = _Step(kv)
    for _ in range(4):  # the first fills a block of the first sequence
        s.stage()
        s.run()
        s.check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_steps_captured_and_replayed(kv):
    s = _Step(kv, seed=1, start=(79, 47, 14))
    s.stage()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    s.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for _ in range(3):
        s.stage()
        g.replay()
        s.check()


def test_first_use_inside_a_capture():
    # a fresh process whose first call of each kernel is captured: the rows are
    # few and the context long, so that the clustered variants are among them
    code = """
import torch
from tests.test_gpu_block_sparse import _Step
s = _Step.__new__(_Step)
_Step._prefill = lambda self: None
_Step.__init__(s, "bf16", 5)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s.run()
s.lens = s.lens * 0
for _ in range(20):
    s.stage()
    g.replay()
s.check()
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert "captured first" in r.stdout, r.stderr[-2000:]


def test_two_batches_on_two_streams():
    a, b = _Step("bf16", seed=2), _Step("fp8", seed=3)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.stage(), b.stage()
        torch.cuda.synchronize()
        for s, st in ((a, sa), (b, sb)):
            with torch.cuda.stream(st):
                s.run()
        torch.cuda.synchronize()
        a.check(), b.check()


def test_two_host_threads():
    steps = [_Step("bf16", seed=6), _Step("fp8", seed=7)]
    for s in steps:
        s.stage()
        s.run()
    torch.cuda.synchronize()
    want = [(s.q.clone(), s.sel.clone(), s.out.clone()) for s in steps]
    failed = []

    def work(s, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    s.run()
                torch.cuda.current_stream().synchronize()
            for got, ref in zip((s.q, s.sel, s.out), w):
                assert torch.equal(got, ref)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(steps, want)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed, failed
    for s in steps:
        s.check()


def test_selection_finds_the_block_that_matters():
    # one key per sequence answers the query; the selection's answer is the
    # whole context's
    rng = np.random.default_rng(20)
    S, H, Hkv, d, B, nb, top = 2, 4, 1, 64, 16, 120, 8
    tables = rng.permutation(S * nb).reshape(S, nb).astype(np.int32)
    k = rng.standard_normal((S * nb, B, Hkv, d)).astype(np.float32)
    q = _bf16(rng, S, H, d)
    for i, j in enumerate((37, 101)):
        k[tables[i, j], 5, 0] = _np(q)[i].sum(0) * 3
    kc = torch.from_numpy(k).to(DEV).to(torch.bfloat16)
    vc = _bf16(rng, S * nb, B, Hkv, d)
    codes, scales = ops.alloc_block_ranges(kc)
    ops.summarize_blocks(kc, _dev(np.arange(S * nb) * B + B - 1), codes, scales)
    lens, sel = _dev([nb * B - 2] * S), torch.empty(S, Hkv, top, device=DEV, dtype=torch.int32)
    ops.select_blocks(sel, q, codes, scales, _dev(tables), lens, B)
    assert 37 in sel[0, 0].tolist() and 101 in sel[1, 0].tolist()
