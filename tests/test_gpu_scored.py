"""GPU parity of the scored step (normalised, rotated write into any cache,
reading back, decode and prompt attention with changed scores) against the
64-bit oracle.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
* norm: a sum of d squares, a root, a quotient and two products in fp32, each
  off by u relative or (the sum, of positive terms) by at most d u: under
  2^-16 relative in all; then the rotation's 3 u (|x c| + |y s|), then half a
  step of bf16 (2^-8), e4m3 (2^-4, 2^-10 among its subnormals) or of the
  8-bit row (half a unit, and the unit's own error times 127).
* reading back: one product in fp32 and half a step of bf16; bf16 bits equal.
* attention: see `weight_error`.
"""
import numpy as np
import pytest
import torch

from oracle import block_sparse as bs
from oracle import scored
from paged_kv_cache_108_gb300 import ops

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).to(DEV)


def _bf16(rng, *shape, scale=1.0):
    return _dev(rng.standard_normal(shape) * scale, torch.float32).to(torch.bfloat16)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _values(cache, scale):
    """What a cache holds, float64."""
    if cache.dtype == torch.uint8:
        return _np(cache.view(torch.float8_e4m3fn)) * float(scale.item())
    if cache.dtype == torch.int8:
        return cache.cpu().numpy().astype(np.float64) * _np(scale)[..., None]
    return _np(cache)


def _cache(rng, kv, *shape, junk=False):
    """(cache, scale): N(0, 1) rows, or random bits (NaNs among them)."""
    if junk:
        if kv == "bf16":
            return _dev(rng.integers(-2 ** 15, 2 ** 15, shape), torch.int16).view(torch.bfloat16), None
        if kv == "fp8":
            return _dev(rng.integers(0, 256, shape), torch.uint8), _dev([0.0117], torch.float32)
        units = _dev(rng.standard_normal(shape[:3]), torch.float32)
        units[rng.random(shape[:3]) < 0.2] = float("nan")
        return _dev(rng.integers(-128, 128, shape), torch.int8), units
    x = rng.standard_normal(shape).astype(np.float32)
    if kv == "bf16":
        return _dev(x, torch.float32).to(torch.bfloat16), None
    if kv == "fp8":
        s = 5.0 / 448
        return (_dev(x / s, torch.float32).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8),
                _dev([s], torch.float32))
    codes, units = scored.rows_in_8_bits(x.astype(np.float64))
    return (_dev(codes, torch.int8),
            _dev(units * 2.0 ** rng.uniform(-2, 2, units.shape), torch.float32))


# ------------------------------------------------------- norm_rope_and_cache

WRITES = [
    # tokens, H, Hkv, d, rot, sections, in turn, adjacent, norm, kv
    (1, 32, 8, 128, 128, None, False, False, True, "bf16"),
    (1, 1, 1, 64, 16, None, False, True, True, "int8"),
    (3, 4, 2, 64, 64, None, False, True, True, "fp8"),
    (37, 4, 2, 64, 0, None, False, False, True, "int8"),
    (37, 4, 2, 64, 0, None, False, False, False, "int8"),
    (37, 4, 2, 64, 32, [6, 5, 5], True, True, True, "bf16"),
    (65, 32, 8, 128, 128, [16, 24, 24], False, False, True, "int8"),
    (65, 8, 8, 128, 112, None, False, False, False, "int8"),
    (130, 7, 3, 128, 48, [7, 9, 5, 3], False, True, True, "int8"),
    (301, 2, 2, 64, 48, None, False, False, True, "fp8"),
    (301, 0, 2, 64, 64, None, False, False, True, "int8"),
    (2500, 5, 1, 128, 128, None, False, False, True, "bf16"),
]


def _table(max_position, rot, base=10000.0):
    ang = np.arange(max_position)[:, None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _write_case(tokens, H, Hkv, d, rot, sections, in_turn, adjacent, norm, kv, seed=0):
    rng = np.random.default_rng(seed)
    B, NB, last = 16, tokens // 16 + 3, 5000
    axes = 1 if sections is None else len(sections)
    qkv = _bf16(rng, tokens, (H + 2 * Hkv) * d, scale=3.0)
    c = dict(q=qkv[:, :H * d].view(tokens, H, d), k=qkv[:, H * d:(H + Hkv) * d].view(tokens, Hkv, d),
             v=qkv[:, (H + Hkv) * d:].view(tokens, Hkv, d))
    slots = rng.permutation(NB * B)[:tokens]
    if tokens > 8:
        slots[[2, 5]] = [-1, NB * B]  # padding and a slot past the pool
    pos = rng.integers(0, last, (axes, tokens))
    pos[:, 0] = last - 1
    kc, ks = _cache(rng, kv, NB, B, Hkv, d, junk=True)
    vc, vs = _cache(rng, kv, NB, B, Hkv, d, junk=True)
    w = rng.standard_normal((2, d)).astype(np.float32) if norm else None
    return dict(c, slots=slots, pos=pos, table=_table(last, rot), sections=sections or [rot // 2],
                kc=kc, ks=ks, vc=vc, vs=vs, w=w, in_turn=in_turn, adjacent=adjacent, rot=rot, kv=kv)


def _write(c, out=None, q=None, stream=None):
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    rotates = c["rot"] > 0
    w = [None if c["w"] is None else _dev(x, torch.float32) for x in (c["w"] if c["w"] is not None else (0, 0))]
    ops.norm_rope_and_cache(out, c["q"] if q is None else q, c["k"], c["v"], c["kc"], c["vc"],
                            _dev(c["slots"]),
                            _dev(c["pos"] if c["pos"].shape[0] > 1 else c["pos"][0]) if rotates else None,
                            _dev(c["table"], torch.float32) if rotates else None, *w, 1e-5, c["ks"],
                            c["vs"], sections=c["sections"] if rotates else None,
                            sections_in_turn=c["in_turn"], adjacent_pairs=c["adjacent"],
                            stream=stream)
    return out


def _written(c, x, which):
    """(normalised and rotated rows, the magnitudes their errors go by)."""
    x = _np(x)
    if c["w"] is not None:
        x = scored.normalise(x, c["w"][which].astype(np.float64), 1e-5)
    if not c["rot"]:
        return x, np.abs(x)
    return bs.rope_rows(x, c["pos"], c["table"].astype(np.float64), c["sections"], c["in_turn"],
                        c["adjacent"])


def _bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("case", WRITES, ids=lambda c: "-".join(map(str, c)))
def test_write_matches_oracle(case):
    c = _write_case(*case)
    before = [None if t is None else t.clone() for t in (c["kc"], c["vc"], c["ks"], c["vs"])]
    out = _write(c)
    torch.cuda.synchronize()
    want, mag = _written(c, c["q"], 0)
    err = np.abs(_np(out) - want)
    assert (err <= 2 ** -8 * np.abs(want) + 2 ** -15.9 * mag).all()
    N, slots = c["q"].shape[0], c["slots"]
    room = c["kc"].shape[0] * c["kc"].shape[1]
    hit = [t for t in range(N) if 0 <= slots[t] < room]
    flat = lambda t: t.view(-1, *t.shape[2:])  # noqa: E731
    for x, which, cache, scale, old, old_scale in (
            (c["k"], 1, c["kc"], c["ks"], before[0], before[2]),
            (c["v"], None, c["vc"], c["vs"], before[1], before[3])):
        want, mag = _written(c, x, which) if which else (_np(x), np.abs(_np(x)))
        want, mag = want[hit], mag[hit]
        fp32 = 2 ** -15.9 * mag if which else 0
        if c["kv"] == "bf16":
            got = _np(flat(cache)[_dev(slots[hit], torch.long)])
            if which:
                assert (np.abs(got - want) <= 2 ** -8 * np.abs(want) + fp32).all()
            else:
                assert np.array_equal(got, want)
        elif c["kv"] == "fp8":
            s = float(scale.item())
            got = _np(flat(cache)[_dev(slots[hit], torch.long)].view(torch.float8_e4m3fn))
            w = np.clip(want / s, -448, 448)
            slack = fp32 / s + 2 ** -23 * np.abs(w)
            assert (np.abs(got - w) <= np.maximum(2 ** -4 * np.abs(w), 2 ** -10) + slack).all()
        else:
            codes, units = scored.rows_in_8_bits(want)
            u = _np(flat(scale))[slots[hit]]
            most = mag.max(-1)
            assert (np.abs(u - units) <= 2 ** -15.9 * most / 127 + 2 ** -23 * units).all()
            held = flat(cache).cpu().numpy()[slots[hit]].astype(np.float64) * u[..., None]
            # half a unit, the fp32 errors, and a code's 127 times the unit's
            slack = 2 * 2 ** -15.9 * most[..., None] if which else 2 ** -21 * most[..., None]
            assert (np.abs(held - want) <= 0.5 * units[..., None] + slack).all()
            if not which:  # no arithmetic before the row's: its codes and units are exact
                unit32 = (np.abs(want).max(-1).astype(np.float32) / np.float32(127))
                code32 = np.rint(want.astype(np.float32) / unit32[..., None])
                assert np.array_equal(u, unit32)
                assert np.array_equal(flat(cache).cpu().numpy()[slots[hit]], code32)
        # slots not named: as they were
        rest = np.setdiff1d(np.arange(room), slots[hit])
        assert np.array_equal(_bits(flat(cache)[_dev(rest, torch.long)]),
                              _bits(flat(old)[_dev(rest, torch.long)]))
        if c["kv"] == "int8":
            assert np.array_equal(_bits(flat(scale)[_dev(rest, torch.long)]),
                                  _bits(flat(old_scale)[_dev(rest, torch.long)]))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_write_without_norm_is_rope_and_cache(kv):
    c = _write_case(70, 8, 2, 128, 64, None, False, True, False, kv)
    d = _write_case(70, 8, 2, 128, 64, None, False, True, False, kv)
    out = _write(c)
    want = torch.full_like(out, 7.0)
    ops.rope_and_cache(want, d["q"], d["k"], d["v"], d["kc"], d["vc"], _dev(d["slots"]),
                       _dev(d["pos"][0]), _dev(d["table"], torch.float32), d["ks"], d["vs"],
                       adjacent_pairs=True)
    for a, b in ((out, want), (c["kc"], d["kc"]), (c["vc"], d["vc"])):
        assert np.array_equal(_bits(a), _bits(b))


def test_write_in_place_and_skipped_positions():
    c = _write_case(20, 4, 2, 64, 64, None, False, False, True, "int8")
    c["pos"][0, [1, 7]] = [-1, 5000]  # neither query nor rows are written
    q = c["q"].contiguous()
    first = q.clone()
    before = [t.clone() for t in (c["kc"], c["vc"], c["ks"], c["vs"])]
    _write(c, out=q, q=q)
    assert torch.equal(q[[1, 7]], first[[1, 7]])
    for t, old in zip((c["kc"], c["vc"], c["ks"], c["vs"]), before):
        at = c["slots"][[1, 7]]
        flat, was = t.view(-1, *t.shape[2:]), old.view(-1, *old.shape[2:])
        assert np.array_equal(_bits(flat[_dev(at, torch.long)]), _bits(was[_dev(at, torch.long)]))
    c["pos"][0, [1, 7]] = 0
    want, mag = _written(c, first, 0)
    keep = [t for t in range(20) if t not in (1, 7)]
    assert (np.abs(_np(q) - want) <= 2 ** -8 * np.abs(want) + 2 ** -15.9 * mag)[keep].all()


def test_int8_rows_of_zeros_infinities_and_nans():
    d = 64
    x = torch.zeros(5, 1, d, dtype=torch.bfloat16, device=DEV)
    x[1, 0, 3] = float("inf")
    x[2, 0, 5] = float("nan")
    x[3, 0, 7] = 1e-38
    x[4, 0] = torch.arange(-32, 32, device=DEV).to(torch.bfloat16)
    kc, vc = (torch.full((1, 8, 1, d), 9, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = ops.alloc_cache_units(kc)
    none = torch.empty(5, 0, d, dtype=torch.bfloat16, device=DEV)
    ops.norm_rope_and_cache(none, none, x, x, kc, vc, _dev([0, 1, 2, 3, 4]), k_scale=ks, v_scale=vs)
    rows = [torch.full((5, 1, d), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ops.gather_cache(*rows, kc, vc, _dev([[0]]), _dev([5]), _dev([0, 5]), None, ks, vs)
    for got in rows:
        got = _np(got)
        assert (got[0] == 0).all() and np.isnan(got[1]).all() and np.isnan(got[2]).all()
        assert abs(got[3, 0, 7] / _np(x)[3, 0, 7] - 1) < 2 ** -7 and (np.delete(got[3, 0], 7) == 0).all()
        assert (np.abs(got[4, 0] - np.arange(-32, 32)) <= 0.5 * 32 / 127 + 2 ** -8 * 32).all()


# -------------------------------------------------------------- gather_cache

@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B,Hkv,d,lens,first", [
    (16, 8, 128, [5, 0, 33, 16, 1], [0, 0, 0, 0, 0]),
    (1, 1, 64, [40], [7]),
    (64, 3, 64, [200, 64, 129, 3], [63, 64, 1, -2]),
    (16, 32, 128, [700], None),
    (8, 2, 128, list(range(1, 71)), None),
])
def test_gather_matches_oracle(kv, B, Hkv, d, lens, first):
    rng = np.random.default_rng(3)
    width = -(-max(lens) // B)
    NB = len(lens) * width + 2
    tables = rng.permutation(NB)[:len(lens) * width].reshape(len(lens), width)
    if len(lens) > 3:
        tables[2, 0] = NB + 5  # outside the pool
    kc, ks = _cache(rng, kv, NB, B, Hkv, d)
    vc, vs = _cache(rng, kv, NB, B, Hkv, d)
    f = first or [0] * len(lens)
    # room: exact, one row short or two rows over
    room = [max(0, n - max(s, 0) + (-1 if i % 3 == 1 else 2 * (i % 2))) for i, (n, s) in enumerate(zip(lens, f))]
    starts = np.cumsum([3] + room)
    rows = starts[-1] + 4
    ko, vo = (torch.full((rows, Hkv, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ops.gather_cache(ko, vo, kc, vc, _dev(tables), _dev(lens), _dev(starts),
                     None if first is None else _dev(first), ks, vs)
    for got, cache, scale in ((ko, kc, ks), (vo, vc, vs)):
        want = np.full((rows, Hkv, d), 7.0)
        vals = _values(cache, scale)
        for i, (n, s) in enumerate(zip(lens, f)):
            if s < 0:
                continue
            x = scored.gather(vals, tables[i], s, min(n, s + room[i]))
            keep = ~np.isnan(x)
            part = want[starts[i]:starts[i] + len(x)]
            part[keep] = x[keep]
        tol = 0 if kv == "bf16" else (2 ** -8 + 2 ** -23) * np.abs(want)
        assert (np.abs(_np(got) - want) <= tol).all()


# ------------------------------------------------------------------ attention

def weight_error(kv, d, most, cap, bias, tiles):
    """A bound on the relative error of a softmax weight.  A logit sums d
    products of at most `most` in all (fp32: (d + 2) u of that, and four more
    roundings of u: q's and the row's units, the scale), e4m3 tiles hold q in
    three e4m3 parts (2^-12).  The cap adds 2^-20 of itself (one exponential,
    one sum, one reciprocal, each off by 2^-22 relative in a quotient of at
    most 2; on the tiles a polynomial within 3.7e-6 < 2^-18 and six roundings of
    u) and 4 u of the score; a bias three u of itself.  exp2 and its
    argument: 2^-21.  Weights enter P V in two bf16 parts (2^-16), one f16 part
    over 8-bit elements (half a step: 2^-11), or on the tiles in one bf16 part
    (2^-9) or two e4m3 parts (2^-8)."""
    e = (d + 6) * 2 ** -24 * most + 2 ** -21
    if tiles and kv == "fp8":
        e += 2 ** -12 * most + 2 ** -8
    else:
        e += 2 ** -9 if tiles else 2 ** -16 if kv == "bf16" else 2 ** -11
    if cap:
        e += (2 ** -18 if tiles else 2 ** -20) * cap + 2 ** -22 * min(most, cap)
    return e + 3 * 2 ** -24 * bias


def _attn_case(seed, kv, lens, H, Hkv, d, B, scale_q=3.0, junk_rest=True):
    rng = np.random.default_rng(seed)
    width = max(1, -(-max(lens + [1]) // B))
    need = [-(-n // B) for n in lens]
    NB = sum(need) + 3
    order, tables, at = rng.permutation(NB), np.full((len(lens), width), -1, np.int64), 0
    for i, m in enumerate(need):
        tables[i, :m] = order[at:at + m]
        at += m
    kc, ks = _cache(rng, kv, NB, B, Hkv, d)
    vc, vs = _cache(rng, kv, NB, B, Hkv, d)
    if junk_rest:  # tokens behind a context's end hold anything
        for i, n in enumerate(lens):
            if n % B:
                for c, s in ((kc, ks), (vc, vs)):
                    b = int(tables[i, n // B])
                    if kv == "int8":
                        s[b, n % B:] = float("nan")
                    else:
                        c[b, n % B:] = float("nan") if kv == "bf16" else 0x7F
    return dict(rng=rng, kv=kv, tables=tables, lens=lens, kc=kc, ks=ks, vc=vc, vs=vs, H=H, Hkv=Hkv,
                d=d, B=B, scale=d ** -0.5, scale_q=scale_q)


def _slopes(H):
    return (2.0 ** (-8 * np.arange(1, H + 1) / H)).astype(np.float32)


def _mod(c, cap, window, bias):
    return dict(cap=cap, window=window,
                slopes=_dev(_slopes(c["H"]), torch.float32) if bias else None, k_scale=c["ks"],
                v_scale=c["vs"])


def _check_rows(c, got, q, rows, cap, window, bias, prefix=None, tiles=False):
    """rows: (row of q, sequence, position)."""
    k, v = _values(c["kc"], c["ks"]), _values(c["vc"], c["vs"])
    slopes = _slopes(c["H"]).astype(np.float64) if bias else None
    got, q = _np(got), _np(q)
    for r, i, pos in rows:
        n = c["lens"][i]
        want, mag, most = scored.attend(q[r], pos, n, k, v, c["tables"][i], c["scale"], cap, window,
                                        slopes, prefix[i] if prefix else 0)
        dist = float(n) * (slopes.max() if bias else 0.0)
        e = weight_error(c["kv"], c["d"], most, cap, dist, tiles)
        # Numerator and denominator both, then half a step of bf16.  f16 weights
        # (8-bit elements, not on the tiles) are raised by 2^14 and end at 2^-24:
        # each is off by up to 2^-25 2^-14 of the largest besides, and the sum of
        # the weights is at least the largest.
        floor = 0.0 if c["kv"] == "bf16" or tiles else n * 2 ** -39 * np.nanmax(np.abs(v))
        tol = 2 ** -8 * np.abs(want) + 2 * e * (mag + np.abs(want)) + floor + 1e-30
        bad = ~(np.abs(got[r] - want) <= tol)
        assert not bad.any(), (r, i, pos, n, float(np.abs(got[r] - want).max()), float(e))


DECODES = [
    # lens, H, Hkv, d, B, cap, window, bias
    ([1], 32, 8, 128, 16, 50.0, 0, False),
    ([5, 16, 17, 40, 0, 1], 4, 2, 64, 16, 30.0, 0, False),
    ([5, 16, 17, 40, 0, 1], 4, 2, 64, 16, 0.0, 7, True),
    ([300, 31, 129], 8, 8, 128, 16, 30.0, 0, True),
    ([300, 31, 129], 8, 1, 128, 1, 30.0, 100, False),
    ([1000, 64, 65], 16, 2, 64, 64, 0.0, 1, False),
    ([700, 2, 333, 128], 8, 4, 128, 128, 50.0, 256, True),
    ([2000], 32, 8, 128, 16, 0.0, 0, True),
    ([1900, 0, 3], 8, 2, 64, 8, 20.0, 1024, False),
    ([1024], 2, 2, 64, 1024, 50.0, 1000, False),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("case", DECODES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_decode_matches_oracle(kv, case):
    lens, H, Hkv, d, B, cap, window, bias = case
    c = _attn_case(11, kv, lens, H, Hkv, d, B)
    if window:  # blocks that the window has left behind: freed
        for i, n in enumerate(lens):
            c["tables"][i, :max(0, n - window) // B] = -7
    q = _bf16(c["rng"], len(lens), H, d, scale=c["scale_q"])
    ws = ops.alloc_scored_workspace(len(lens), H, Hkv, d).random_(0, 256)
    out = torch.full_like(q, 7.0)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"],
                      workspace=ws, **_mod(c, cap, window, bias))
    _check_rows(c, out, q, [(i, i, n - 1) for i, n in enumerate(lens)], cap, window, bias)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_decode_passes_over_blocks_outside_the_pool(kv):
    c = _attn_case(12, kv, [100, 64], 4, 2, 128, 16)
    c["tables"][0, [1, 4]] = [-1, 10 ** 6]
    q = _bf16(c["rng"], 2, 4, 128)
    out = torch.empty_like(q)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(c["lens"]), c["scale"],
                      **_mod(c, 50.0, 0, False))
    _check_rows(c, out, q, [(0, 0, 99), (1, 1, 63)], 50.0, 0, False)


@pytest.mark.parametrize("kv,H,Hkv,d", [("bf16", 8, 2, 128), ("fp8", 8, 1, 64), ("int8", 4, 4, 128),
                                        ("int8", 8, 1, 128)])
def test_decode_ragged_batches_are_split_evenly(kv, H, Hkv, d):
    """One long sequence among short and empty ones: units shared by many
    CTAs, CTAs that hold many units."""
    lens = [7000, 0, 1, 130, 0, 2048] + [17] * 40 + [900]
    c = _attn_case(13, kv, lens, H, Hkv, d, 16)
    q = _bf16(c["rng"], len(lens), H, d, scale=3.0)
    ws = ops.alloc_scored_workspace(len(lens), H, Hkv, d)
    args = (c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"])
    outs = []
    for _ in range(3):
        ws.random_(0, 256)
        out = torch.full_like(q, 7.0)
        ops.decode_scored(out, q, *args, workspace=ws, **_mod(c, 30.0, 0, False))
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    _check_rows(c, outs[0], q, [(i, i, n - 1) for i, n in enumerate(lens)], 30.0, 0, False)


def test_decode_many_units_without_splits():
    """As many units as make every CTA take a whole one."""
    H = Hkv = 4
    n = 6 * 2 * 160 // 4 + 3
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 40, n)]
    for kv in ("bf16", "int8"):
        c = _attn_case(14, kv, lens, H, Hkv, 64, 16)
        q = _bf16(c["rng"], n, H, 64)
        out = torch.full_like(q, 7.0)
        ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"],
                          **_mod(c, 0.0, 0, True))
        _check_rows(c, out, q, [(i, i, m - 1) for i, m in enumerate(lens)][::7], 0.0, 0, True)


def test_int8_units_of_any_size():
    """Values' units that differ by up to 2^80, and zeros among them."""
    c = _attn_case(15, "int8", [400, 33], 8, 2, 128, 16)
    c["vs"].copy_(_dev(2.0 ** c["rng"].uniform(-60, 20, tuple(c["vs"].shape)), torch.float32))
    c["vs"][c["rng"].random(tuple(c["vs"].shape)) < 0.1] = 0.0
    q = _bf16(c["rng"], 2, 8, 128)
    out = torch.empty_like(q)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(c["lens"]), c["scale"],
                      **_mod(c, 0.0, 0, False))
    _check_rows(c, out, q, [(0, 0, 399), (1, 1, 32)], 0.0, 0, False)


PROMPTS = [
    # seq_lens, new tokens, H, Hkv, d, B, cap, window, bias, prefix
    ([300, 37, 129], [100, 37, 1], 8, 2, 128, 16, 50.0, 0, False, None),
    ([300, 37, 129], [100, 37, 40], 8, 2, 128, 16, 30.0, 33, True, None),
    ([200, 150, 5], [200, 90, 5], 4, 4, 128, 16, 30.0, 0, False, [130, 100, 9]),
    ([700], [300], 8, 1, 128, 128, 0.0, 200, False, [450]),
    ([515, 260], [129, 255], 4, 2, 128, 8, 50.0, 128, True, [400, 0]),
    ([3, 0, 9], [4, 0, 9], 8, 8, 128, 16, 50.0, 0, False, None),        # more new than there are
    ([40, 17, 200], [3, 2, 5], 4, 2, 64, 16, 30.0, 0, True, [39, 0, 3]),
    ([40, 17, 200, 9], [3, 1, 2, 1], 8, 1, 128, 16, 30.0, 50, False, None),
    ([90, 40], [60, 40], 4, 2, 64, 4, 50.0, 21, True, [70, 10]),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_prompts_match_oracle(kv, case):
    lens, new, H, Hkv, d, B, cap, window, bias, prefix = case
    c = _attn_case(21, kv, lens, H, Hkv, d, B)
    if window:
        for i, (n, t) in enumerate(zip(lens, new)):
            c["tables"][i, :max(0, n - t + 1 - window) // B] = -7
    starts = np.cumsum([0] + new)
    q = _bf16(c["rng"], int(starts[-1]) + 3, H, d, scale=c["scale_q"])
    ws = ops.alloc_scored_workspace(q.shape[0], H, Hkv, d).random_(0, 256)
    ws[:4] = 0
    out = torch.full_like(q, 7.0)
    ops.varlen_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), _dev(starts),
                      c["scale"], prefix_lens=None if prefix is None else _dev(prefix),
                      workspace=ws, **_mod(c, cap, window, bias))
    n = q.shape[0]
    tiles = (kv != "int8" and d == 128 and B >= 8
             and (n > 8 and n > 2 * len(lens) if kv == "bf16" else n > 16 and n > 4 * len(lens)))
    if tiles:
        assert int(ws[:4].view(torch.int32).item()) == 0
    assert (out[int(starts[-1]):] == 7.0).all()  # rows behind the last request
    rows, zero = [], []
    for i, (n, t) in enumerate(zip(lens, new)):
        if t > n:
            zero += range(starts[i], starts[i + 1])
        else:
            rows += [(int(starts[i]) + j, i, n - t + j) for j in range(t)]
    assert (out[zero] == 0).all()
    some = rows if len(rows) < 120 else [rows[k] for k in sorted(set(
        list(range(0, len(rows), 7)) + [0, 1, len(rows) - 1, len(rows) - 2]))]
    _check_rows(c, out, q, some, cap, window, bias, prefix, tiles)


def test_prompt_over_gathered_rows():
    """Contexts of 8-bit rows, read back to block starts, as a bf16 cache of
    the prompt's tiles: what the row-by-row form over the 8-bit cache gives."""
    lens, new, H, Hkv, d, B = [300, 77], [64, 77], 8, 2, 128, 16
    c = _attn_case(31, "int8", lens, H, Hkv, d, B)
    starts = np.cumsum([0] + new)
    q = _bf16(c["rng"], int(starts[-1]), H, d, scale=2.0)
    blocks = [-(-n // B) for n in lens]
    at = np.cumsum([0] + blocks)
    rows = [torch.zeros(int(at[-1]) * B, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ops.gather_cache(*rows, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), _dev(at * B), None,
                     c["ks"], c["vs"])
    tables = np.zeros((2, max(blocks)), np.int64)
    for i, m in enumerate(blocks):
        tables[i, :m] = np.arange(at[i], at[i] + m)
    flat = dict(c, kv="bf16", kc=rows[0].view(-1, B, Hkv, d), vc=rows[1].view(-1, B, Hkv, d), ks=None,
                vs=None, tables=tables)
    out = torch.empty_like(q)
    ops.varlen_scored(out, q, flat["kc"], flat["vc"], _dev(tables), _dev(lens), _dev(starts),
                      c["scale"], **_mod(flat, 30.0, 0, False))
    picked = [(int(starts[i]) + j, i, n - t + j) for i, (n, t) in enumerate(zip(lens, new))
              for j in range(0, t, 9)]
    _check_rows(flat, out, q, picked, 30.0, 0, False, None, True)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_step_as_a_layer_runs_it(kv):
    """A prompt written and attended to, then single tokens: normalised and
    rotated keys in any cache, attention over what was written."""
    H, Hkv, d, B, n, steps = 8, 2, 128, 16, 45, 4
    rng = np.random.default_rng(41)
    width = -(-(n + steps) // B)
    tables = rng.permutation(width + 2)[:width][None]
    kc, ks = _cache(rng, kv, width + 2, B, Hkv, d, junk=True)
    vc, vs = _cache(rng, kv, width + 2, B, Hkv, d, junk=True)
    cs = _dev(_table(n + steps, d), torch.float32)
    w = [_dev(1 + 0.1 * rng.standard_normal(d), torch.float32) for _ in range(2)]
    ws = ops.alloc_scored_workspace(n, H, Hkv, d)
    mod = dict(cap=20.0, k_scale=ks, v_scale=vs)
    for lo, hi in [(0, n)] + [(n + i, n + i + 1) for i in range(steps)]:
        t = np.arange(lo, hi)
        x = _bf16(rng, hi - lo, H + 2 * Hkv, d)
        q = torch.empty(hi - lo, H, d, dtype=torch.bfloat16, device=DEV)
        ops.norm_rope_and_cache(q, x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc,
                                _dev(tables[0, t // B] * B + t % B), _dev(t), cs, *w, 1e-6, ks, vs)
        out = torch.empty_like(q)
        if hi - lo > 1:
            ops.varlen_scored(out, q, kc, vc, _dev(tables), _dev([hi]), _dev([0, hi - lo]), d ** -0.5,
                              workspace=ws, **mod)
        else:
            ops.decode_scored(out, q, kc, vc, _dev(tables), _dev([hi]), d ** -0.5, workspace=ws, **mod)
        c = dict(kv=kv, kc=kc, vc=vc, ks=ks, vs=vs, tables=tables, lens=[hi], H=H, d=d,
                 scale=d ** -0.5)
        _check_rows(c, out, q, [(r, 0, lo + r) for r in range(hi - lo)], 20.0, 0, False, None,
                    kv != "int8" and hi - lo > 1)


# ------------------------------------------------------- streams and graphs

def test_replayed_graphs_share_a_workspace_and_follow_their_inputs():
    lens = [900, 17, 2500]
    H, Hkv, d, B = 8, 2, 128, 16
    c = _attn_case(51, "int8", lens, H, Hkv, d, B)
    q = [_bf16(c["rng"], 3, H, d, scale=2.0) for _ in range(2)]
    out = [torch.zeros_like(q[0]) for _ in range(2)]
    tables, dev_lens = _dev(c["tables"]), _dev(lens)
    ws = ops.alloc_scored_workspace(3, H, Hkv, d)

    def step(i):
        ops.decode_scored(out[i], q[i], c["kc"], c["vc"], tables, dev_lens, c["scale"], workspace=ws,
                          **_mod_kept)

    _mod_kept = _mod(c, 30.0, 0, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)
        step(1)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            step(i)
    for turn in range(3):
        for i in range(2):
            q[i].copy_(_bf16(c["rng"], 3, H, d, scale=2.0))
            graphs[i].replay()
        step(0)  # an eager call between replays
        graphs[0].replay()
    for i in range(2):
        _check_rows(c, out[i], q[i], [(r, r, n - 1) for r, n in enumerate(lens)], 30.0, 0, False)


def test_calls_on_another_stream_without_a_workspace():
    c = _attn_case(52, "bf16", [500, 40], 8, 2, 128, 16)
    q = _bf16(c["rng"], 2, 8, 128)
    side = torch.cuda.Stream()
    args = (c["kc"], c["vc"], _dev(c["tables"]), _dev(c["lens"]), c["scale"])
    mod = _mod(c, 50.0, 0, True)
    torch.cuda.synchronize()
    outs = [torch.zeros_like(q) for _ in range(4)]
    torch.cuda.synchronize()
    for k, out in enumerate(outs):
        ops.decode_scored(out, q, *args, stream=side if k % 2 else side.cuda_stream, **mod)
    side.synchronize()
    for out in outs:
        assert torch.equal(out, outs[0])
    _check_rows(c, outs[0], q, [(0, 0, 499), (1, 1, 39)], 50.0, 0, True)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_caches_beyond_32_bit_offsets(kv):
    """Slots whose element offsets pass 2^32 (int8) and bytes 2^33 (bf16)."""
    H = Hkv = 32
    d, B = 128, 16
    NB = (1 << 32) // (Hkv * d * B) + 40
    dt = torch.bfloat16 if kv == "bf16" else torch.int8
    kc, vc = (torch.zeros(NB, B, Hkv, d, dtype=dt, device=DEV) for _ in range(2))
    ks, vs = ops.alloc_cache_units(kc) if kv == "int8" else (None, None)
    rng = np.random.default_rng(61)
    table = np.array([[NB - 1, 0, NB - 30, NB - 7]])
    n = 50
    t = np.arange(n)
    x = _bf16(rng, n, 3 * H, d)
    q = torch.empty(n, H, d, dtype=torch.bfloat16, device=DEV)
    ops.norm_rope_and_cache(q, x[:, :H], x[:, H:2 * H], x[:, 2 * H:], kc, vc,
                            _dev(table[0, t // B] * B + t % B), k_scale=ks, v_scale=vs)
    rows = [torch.empty(n, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ops.gather_cache(*rows, kc, vc, _dev(table), _dev([n]), _dev([0, n]), None, ks, vs)
    tol = 0.5 / 127 if kv == "int8" else 0.0
    for got, src in zip(rows, (x[:, H:2 * H], x[:, 2 * H:])):
        src = _np(src)
        slack = tol * np.abs(src).max(-1, keepdims=True) + (2 ** -8 * np.abs(_np(got)) if tol else 0)
        assert (np.abs(_np(got) - src) <= slack * (1 + 2 ** -20)).all()
    out = torch.empty(1, H, d, dtype=torch.bfloat16, device=DEV)
    ops.decode_scored(out, q[-1:].contiguous(), kc, vc, _dev(table), _dev([n]), d ** -0.5, cap=30.0,
                      k_scale=ks, v_scale=vs)
    # the oracle over the few blocks in use
    used = _dev(np.unique(table), torch.long)
    small = dict(kv=kv, kc=kc[used], vc=vc[used], ks=None if ks is None else ks[used],
                 vs=None if vs is None else vs[used], H=H, d=d, scale=d ** -0.5, lens=[n],
                 tables=np.searchsorted(np.unique(table), table))
    _check_rows(small, out, q[-1:], [(0, 0, n - 1)], 30.0, 0, False)
