"""The scored step's prompt tiles: e4m3 tiles against the bound that their
arithmetic gives, and steps of more than 65535 new tokens.

Over e4m3 the tiles hold keys and values in f16 (exact), q in f16 under a power
of two that puts its row's largest element in [1, 2) (bf16's 8 bits fit but for
elements below 2^-14 of the largest, off by up to 2^-25 of it), and weights in
f16: half a step, 2^-11.  Weights are at most 2^8 relative to their reference,
raised by 2^7, and end at 2^-24: each is off by up to 2^-32 of the largest
besides.  The cap: 3.7e-6 of itself up to 64 (and 2^-22 of the score for its
roundings).  Logits, exponentials and biases as `weight_error` in the parity
tests."""
import numpy as np
import pytest
import torch

from oracle import scored
from tests.test_gpu_scored import PROMPTS, _attn_case, _check_rows, _dev, _np, _slopes, _values
from tests.test_gpu_scored_edges import _rows, _step, _varlen

pytestmark = pytest.mark.gpu


def _check_e4m3(c, got, q, rows, cap, window, bias, prefix=None):
    k, v = _values(c["kc"], c["ks"]), _values(c["vc"], c["vs"])
    slopes = _slopes(c["H"]).astype(np.float64) if bias else None
    got, q = _np(got), _np(q)
    key = np.nansum(np.abs(k), -1).max() * abs(c["scale"])
    most_v = np.nanmax(np.abs(v))
    for r, i, pos in rows:
        n = c["lens"][i]
        want, mag, most = scored.attend(q[r], pos, n, k, v, c["tables"][i], c["scale"], cap, window,
                                        slopes, prefix[i] if prefix else 0)
        e = (c["d"] + 6) * 2 ** -24 * most + 2 ** -21 + 2 ** -11 + 2 ** -25 * np.abs(q[r]).max() * key
        if cap:
            e += 3.7e-6 * cap + 2 ** -22 * min(most, cap)
        if bias:
            e += 3 * 2 ** -24 * n * slopes.max()
        tol = 2 ** -8 * np.abs(want) + 2 * e * (mag + np.abs(want)) + n * 2 ** -32 * most_v + 1e-30
        bad = ~(np.abs(got[r] - want) <= tol)
        assert not bad.any(), (r, i, pos, n, float(np.abs(got[r] - want).max()), float(e))


@pytest.mark.parametrize("case", [p for p in PROMPTS if p[4] == 128 and sum(p[1]) > 40],
                         ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_e4m3_prompts_within_their_arithmetic(case):
    lens, new, H, Hkv, d, B, cap, window, bias, prefix = case
    c = _attn_case(131, "fp8", lens, H, Hkv, d, B)
    q, starts = _step(c, new)
    out = _varlen(c, q, starts, cap=cap, window=window, bias=bias, prefix=prefix)
    _check_e4m3(c, out, q, _rows(c, starts, 7), cap, window, bias, prefix)


@pytest.mark.parametrize("scale", [-0.09, 0.09, 0.5])
@pytest.mark.parametrize("cap", [0.0, 1.5, 20.0, 50.0, 64.0])
def test_e4m3_scales_and_caps_within_their_arithmetic(scale, cap):
    new, lens = [40, 33], [1300, 33]
    c = _attn_case(132, "fp8", lens, 8, 2, 128, 16)
    c["scale"] = scale
    q, starts = _step(c, new)
    q[::3] *= _dev(2.0 ** np.random.default_rng(1).uniform(-20, 0, (q[::3].shape[0], 8, 128)),
                   torch.float32)  # elements far below their row's largest
    out = _varlen(c, q, starts, cap=cap)
    _check_e4m3(c, out, q, _rows(c, starts, 8), cap, 0, False)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_more_than_65535_new_tokens_take_the_tiles(kv):
    """A small window keeps it cheap.  The tiles alone report a block outside the
    pool: here one that a second request's first block names."""
    new, lens = [66_000, 40], [66_100, 60]
    c = _attn_case(133, kv, lens, 2, 1, 128, 64)
    c["scale"] = 0.05
    q, starts = _step(c, new)
    out = _varlen(c, q, starts, cap=30.0, window=150)
    _check_rows(c, out, q, _rows(c, starts, 4001), 30.0, 150, False, None, True)
    ws = _workspace_after_a_bad_block(c, q, starts)
    assert int(ws[:4].view(torch.int32).item()) == 3


def _workspace_after_a_bad_block(c, q, starts):
    from paged_kv_cache_108_gb300 import ops
    from tests.test_gpu_scored import _mod
    tables = np.array(c["tables"])
    tables[1, 0] = 10 ** 6
    ws = ops.alloc_scored_workspace(q.shape[0], c["H"], c["Hkv"], c["d"])
    ws[:4] = 0
    ops.varlen_scored(torch.empty_like(q), q, c["kc"], c["vc"], _dev(tables), _dev(c["lens"]),
                      _dev(starts), c["scale"], workspace=ws, **_mod(c, 30.0, 150, False))
    return ws
