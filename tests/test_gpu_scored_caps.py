"""The scored step's attention under caps far above the scores: the cap must
leave small scores as they are, whatever its size and whatever other rows of
a tile hold.

A capped score is off by at most 2^-20 of the score itself: up to 5/8 of the
cap an odd polynomial with leading coefficient 1 (2^-22 relative, with its
roundings), above that 1 - 2 / (1 + e^2u), off by 2^-21.5 of the cap
(exponential, reciprocal and sum) where the score is at least 0.55 of it.  The
tiles do so for caps above 64.  The other terms are those of `weight_error` in
the parity tests, but for e4m3 tiles: q and the weights enter the products in
f16 there, so a weight is off by half a step of f16, 2^-11, and an element of q
below 2^-14 of its row's largest by 2^-25 of that one."""
import numpy as np
import pytest
import torch

from oracle import scored
from paged_kv_cache_108_gb300 import ops
from tests.test_gpu_scored import _attn_case, _bf16, _dev, _mod, _np, _slopes, _values
from tests.test_gpu_scored_edges import _rows, _step, _varlen

pytestmark = pytest.mark.gpu


def _check(c, got, q, rows, cap, tiles, window=0, bias=False, prefix=None):
    """rows: (row of q, sequence, position)."""
    k, v = _values(c["kc"], c["ks"]), _values(c["vc"], c["vs"])
    got, q = _np(got), _np(q)
    most_v = np.nanmax(np.abs(v))
    slopes = _slopes(c["H"]).astype(np.float64) if bias else None
    for r, i, pos in rows:
        n = c["lens"][i]
        want, mag, most = scored.attend(q[r], pos, n, k, v, c["tables"][i], c["scale"], cap, window,
                                        slopes, prefix[i] if prefix else 0)
        e = (c["d"] + 6) * 2 ** -24 * most + 2 ** -21 + 2 ** -20 * most
        if bias:
            e += 3 * 2 ** -24 * n * slopes.max()
        if c["kv"] == "bf16":
            e += 2 ** -9 if tiles else 2 ** -16
            floor = 0.0
        else:
            e += 2 ** -11
            # f16 weights end at 2^-24, raised by 2^14 (tiles: 2^7)
            floor = n * 2.0 ** (-32 if tiles else -39) * most_v
            if tiles:
                e += 2 ** -25 * np.abs(q[r]).max() * np.nansum(np.abs(k), -1).max() * abs(c["scale"])
        tol = 2 ** -8 * np.abs(want) + 2 * e * (mag + np.abs(want)) + floor + 1e-30
        bad = ~(np.abs(got[r] - want) <= tol)
        assert not bad.any(), (r, i, pos, float(np.abs(got[r] - want).max()), float(e))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (4, 4, 64), (8, 1, 128)])
@pytest.mark.parametrize("cap", [50.0, 65.0, 1e3, 3e4, 1e6])
def test_decode_under_large_caps(kv, H, Hkv, d, cap):
    lens = [700, 33, 1]
    c = _attn_case(101, kv, lens, H, Hkv, d, 16)
    q = _bf16(c["rng"], 3, H, d, scale=3.0)
    q[:, 1] *= 2.0 ** 6  # a head whose scores pass small caps
    out = torch.empty_like(q)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"],
                      **_mod(c, cap, 0, False))
    _check(c, out, q, [(i, i, n - 1) for i, n in enumerate(lens)], cap, False)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (4, 4), (8, 1)])
@pytest.mark.parametrize("cap", [65.0, 1e3, 3e4, 1e6])
@pytest.mark.parametrize("loud", [False, True])
def test_prompts_under_large_caps(kv, H, Hkv, cap, loud):
    """`loud`: every fifth token's scores reach the cap, in the tiles' rows
    beside others whose scores are small."""
    new, lens = [40, 33], [300, 33]
    c = _attn_case(102, kv, lens, H, Hkv, 128, 16)
    q, starts = _step(c, new)
    if loud:
        q[::5] *= 2.0 ** np.ceil(np.log2(cap / 10))
    out = _varlen(c, q, starts, cap=cap)
    _check(c, out, q, _rows(c, starts, 4), cap, kv != "int8")


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_large_cap_and_scales_of_any_size(kv):
    new, lens = [40, 33], [300, 33]
    for scale in (-0.09, 1e-30, 0.0, 0.5):
        c = _attn_case(103, kv, lens, 8, 2, 128, 16)
        c["scale"] = scale
        q, starts = _step(c, new)
        out = _varlen(c, q, starts, cap=1e5, window=200)
        _check(c, out, q, _rows(c, starts, 8), 1e5, True, 200)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_capped_rows_do_not_depend_on_loud_neighbours(kv):
    """Under a large cap a row's scores are those that it has alone: rows
    beside it that reach the cap choose no formula for it."""
    c = _attn_case(104, kv, [700], 8, 2, 128, 16)
    q, starts = _step(c, [64])
    want = _varlen(c, q, starts, cap=200.0)
    q[1::2] *= 256.0
    got = _varlen(c, q, starts, cap=200.0)
    assert torch.equal(got[::2], want[::2])


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_large_caps_with_biases_windows_and_prefixes(kv):
    new, lens, prefix = [70, 129, 40], [900, 513, 60], [850, 0, 60]
    c = _attn_case(105, kv, lens, 8, 2, 128, 16)
    q, starts = _step(c, new)
    q[::7] *= 64.0
    for cap, window in ((100.0, 0), (1e4, 300)):
        out = _varlen(c, q, starts, cap=cap, window=window, bias=True, prefix=prefix)
        _check(c, out, q, _rows(c, starts, 17), cap, kv != "int8", window, True, prefix)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_queries_that_are_not_finite_under_a_large_cap(kv):
    c = _attn_case(106, kv, [200, 77], 8, 2, 128, 16)
    q, starts = _step(c, [40, 30])
    clean = _varlen(c, q, starts, cap=1e3)
    q[3, 2, 5] = float("nan")
    q[50, 7, 1] = float("inf")
    got = _varlen(c, q, starts, cap=1e3)
    assert torch.isnan(got[3, 2]).all()
    same = torch.ones(got.shape[:2], dtype=torch.bool)
    same[3, 2] = same[50, 7] = False
    assert torch.equal(got[same.cuda()], clean[same.cuda()])
