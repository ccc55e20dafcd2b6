"""Decoding over 8-bit rows whose units differ by any factor: tokens with
nearly all the weight keep their values beside others whose values are larger
by up to 2^100 but hardly count.

A weight times its row's unit enters the products in f16, relative to the
largest such product of its head up to then: off by half a step, 2^-11, or by
half of f16's last, 2^-25, under a raise of 2^12: 2^-37 of the largest
product.  (The reference is at most the largest product; 2^-36 allows for its
own roundings.)  A code is at most 127."""
import numpy as np
import pytest
import torch

from paged_kv_cache_108_gb300 import ops
from tests.test_gpu_scored import DEV, _attn_case, _bf16, _dev, _mod, _np, _values

pytestmark = pytest.mark.gpu


def _check(c, got, q, rows):
    k, v = _values(c["kc"], c["ks"]), _values(c["vc"], c["vs"])
    units, codes = _np(c["vs"]), c["vc"].cpu().numpy().astype(np.float64)
    got, q, B = _np(got), _np(q), c["B"]
    for r, i, n in rows:
        at = np.arange(n)
        block = np.asarray(c["tables"][i])[at // B]
        for h in range(c["H"]):
            g = h // (c["H"] // c["Hkv"])
            s = k[block, at % B, g] @ q[r, h] * c["scale"]
            most = (np.abs(k[block, at % B, g]) @ np.abs(q[r, h])).max() * abs(c["scale"])
            p = np.exp(s - s.max())
            p /= p.sum()
            u = units[block, at % B, g]
            val = codes[block, at % B, g] * u[:, None]
            want, mag = p @ val, p @ np.abs(val)
            e = (c["d"] + 6) * 2 ** -24 * most + 2 ** -21 + 2 ** -11
            floor = n * 2 ** -36 * 127 * (p * u).max()
            tol = 2 ** -8 * np.abs(want) + 2 * e * (mag + np.abs(want)) + floor + 1e-38
            bad = ~(np.abs(got[r, h] - want) <= tol)
            assert not bad.any(), (r, h, float((np.abs(got[r, h] - want) / (np.abs(want) + 1e-38)).max()))


def _pointed(c, q, i, heads, tokens, strength):
    """Makes sequence i's tokens' keys point along the first of their head's
    queries; the others' keys get a hundredth of their size."""
    B = c["B"]
    c["ks"].mul_(0.01)
    for t in tokens:
        b, o = int(c["tables"][i, t // B]), t % B
        for g in range(c["Hkv"]):
            x = q[i, g * heads].float()
            c["kc"][b, o, g] = torch.round(x / x.abs().max() * 127).to(torch.int8)
            c["ks"][b, o, g] = strength / 127


@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (4, 4, 64), (8, 1, 128), (2, 1, 64)])
@pytest.mark.parametrize("power", [20, 34, 40, 60, 100])
@pytest.mark.parametrize("place", ["first", "last", "middle", "both"])
def test_small_units_keep_their_values(H, Hkv, d, power, place):
    """Tokens with nearly all the weight of the first head of each group, whose
    values' units are 2^power below the others'."""
    n = 900
    c = _attn_case(111, "int8", [n, 40], H, Hkv, d, 16)
    q = _bf16(c["rng"], 2, H, d, scale=1.0)
    tokens = {"first": [0], "last": [n - 1], "middle": [n // 2 + 3], "both": [0, n - 2]}[place]
    # scores of the tokens: some d scale strength = (power + 30) ln 2
    strength = (power + 30) * 0.6931 * 3.0 / (d * c["scale"]) * 0.7
    _pointed(c, q, 0, H // Hkv, tokens, strength * 2)
    c["vs"].copy_(torch.full_like(c["vs"], 2.0 ** (power // 2)))
    for t in tokens:
        c["vs"][int(c["tables"][0, t // 16]), t % 16] = 2.0 ** (power // 2 - power)
    out = torch.empty_like(q)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(c["lens"]), c["scale"],
                      **_mod(c, 0.0, 0, False))
    _check(c, out, q, [(0, 0, n), (1, 1, 40)])


def test_units_over_every_size_split_over_ctas():
    """Long rows cut into parts, units over 2^200, zeros among them."""
    lens = [9000, 1200, 70]
    c = _attn_case(112, "int8", lens, 4, 1, 128, 16)
    c["vs"].copy_(_dev(2.0 ** c["rng"].uniform(-100, 100, tuple(c["vs"].shape)), torch.float32))
    c["vs"][c["rng"].random(tuple(c["vs"].shape)) < 0.1] = 0.0
    q = _bf16(c["rng"], 3, 4, 128, scale=20.0)
    outs = []
    for _ in range(2):
        out = torch.empty_like(q)
        ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"],
                          **_mod(c, 0.0, 0, False))
        outs.append(out)
    assert torch.equal(*outs)
    _check(c, outs[0], q, [(i, i, n) for i, n in enumerate(lens)])


def test_units_in_prompts_and_of_growing_weights():
    """New tokens over 8-bit rows; weights that grow along the context while the
    units fall, so that the reference follows them down."""
    n, d, B = 1500, 128, 16
    c = _attn_case(113, "int8", [n], 4, 1, d, B)
    q = _bf16(c["rng"], 3, 4, d, scale=1.0)
    flat = np.asarray(c["tables"][0])
    t = np.arange(n)
    # keys along one direction of growing length: scores rise by some 80 nats
    x = q[2, 0].float()
    code = torch.round(x / x.abs().max() * 127).to(torch.int8)
    c["kc"].copy_(code.expand_as(c["kc"]))
    at = (_dev(flat[t // B], torch.long), _dev(t % B, torch.long))
    c["ks"][at] = _dev(np.linspace(0, 30.0 / 127, n), torch.float32)[:, None]
    c["vs"][at] = _dev(2.0 ** -np.linspace(-30, 70, n), torch.float32)[:, None]
    out = torch.empty_like(q)
    ops.varlen_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev([n]), _dev([0, 3]), c["scale"],
                      **_mod(c, 0.0, 0, False))
    _check(c, out, q, [(r, 0, n - 2 + r) for r in range(3)])


@pytest.mark.parametrize("unit", [float("inf"), float("nan")])
@pytest.mark.parametrize("token", [0, 100, 899])
def test_rows_that_are_not_finite_reach_their_heads_alone(unit, token):
    c = _attn_case(114, "int8", [900, 40], 8, 2, 128, 16)
    b, o = int(c["tables"][0, token // 16]), token % 16
    c["vs"][b, o, 1] = unit
    c["vc"][b, o, 1] = 0
    q = _bf16(c["rng"], 2, 8, 128)
    out = torch.empty_like(q)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(c["lens"]), c["scale"],
                      **_mod(c, 30.0, 0, False))
    assert torch.isnan(out[0, 4:]).all()
    assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1]).all()
