"""Block-sparse decode step on a GPU: values at the ends of their range, sizes
at the ends of theirs, and how tensors' memory is written.

Tolerances are those derived in test_gpu_block_sparse.py; where bits have to
be equal the test says so.
"""
import numpy as np
import pytest
import torch

from oracle import block_sparse as bs
from paged_kv_cache_108_gb300 import ops
from tests.test_gpu_block_sparse import DEV, _bf16, _dev, _np, _rope_case, _rope_run

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------- summarize_blocks

def test_ranges_bound_tiny_keys_beside_huge_ones():
    # k / u below the smallest float must still round outward
    rng = np.random.default_rng(50)
    B, Hkv, d = 16, 2, 128
    k = torch.zeros(4, B, Hkv, d, dtype=torch.float32)
    k[:, :, :, 0] = torch.tensor([2.0 ** 23, 2.0 ** 30, 2.0 ** 50, 2.0 ** 60])[:, None, None]
    tiny = 2.0 ** rng.integers(-133, -100, (4, B, Hkv, 40)) * rng.choice([-1.0, 1.0], (4, 1, Hkv, 40))
    k[:, :, :, 1:41] = torch.from_numpy(tiny).float()
    kc = k.to(DEV).to(torch.bfloat16)
    values = _np(kc)
    assert (values[:, :, :, 1:41] == tiny).all()  # bf16 holds them
    codes, scales = ops.alloc_block_ranges(kc)
    ops.summarize_blocks(kc, _dev(np.arange(4) * B + B - 1), codes, scales)
    for b in range(4):
        want, u = bs.block_range(values[b])
        assert np.array_equal(scales[b].cpu().numpy(), u)
        assert np.array_equal(codes[b].cpu().numpy(), want)
        assert set(np.abs(want[:, :, 1:41]).max(1).ravel()) == {1}


@pytest.mark.parametrize("heads", [32767, 32768])
def test_ranges_of_the_most_heads_and_the_smallest_blocks(heads):
    rng = np.random.default_rng(51)
    kc = _bf16(rng, 3, 1, heads, 128)
    slots = np.full(1025, -1)
    slots[[7, 1000, 1024]] = [2, 0, 1]
    codes, scales = ops.alloc_block_ranges(kc)
    ops.summarize_blocks(kc, _dev(slots), codes, scales)
    some = [0, 1, 255, 256, 8191, heads // 2, heads - 257, heads - 2, heads - 1]
    values = _np(kc[:, :, some])
    for b in range(3):
        want, u = bs.block_range(values[b])
        assert np.array_equal(scales[b, some].cpu().numpy(), u)
        assert np.array_equal(codes[b, some].cpu().numpy(), want)
    assert (scales > 0).all()


# ----------------------------------------------------------- decode_selected

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("G,top", [(1, 70), (4, 70), (8, 70), (4, 3)])
def test_weights_far_below_the_largest_count(G, top, kv):
    # The first token outweighs each of the others by up to 2^26 and has a zero
    # value, so that the output is what the others add up to.
    B, d, n = 16, 64, 16 * top - 5
    q = torch.zeros(1, G, d, device=DEV, dtype=torch.bfloat16)
    q[0, :, 0] = torch.linspace(0.75, 1.0, G, device=DEV).to(torch.bfloat16)
    k = torch.zeros(top, B, 1, d, device=DEV)
    k[0, 0, 0, 0] = 1.0
    v = torch.ones(top, B, 1, d, device=DEV)
    v[:, :, 0, 1::2] = 0.5
    v[0, 0] = 0.0
    kc, vc = ((x.to(torch.bfloat16) if kv == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8))
              for x in (k, v))
    one = None if kv == "bf16" else _dev([1.0], torch.float32)
    table, sel = _dev(np.arange(top)[None]), _dev(np.arange(top)[None, None])
    scale = 26 * float(np.log(2.0))
    out = torch.empty_like(q)
    ops.decode_selected(out, q, kc, vc, table, _dev([n]), sel, scale, one, one)
    want, mag = bs.decode_selected(_np(q)[0], _np(k), _np(v), np.arange(top), n, sel[0].cpu().numpy(), scale)
    assert want.min() > 0.4 * (n - 1) * 2.0 ** -26
    assert (np.abs(_np(out)[0] - want) <= 2 ** -8 * np.abs(want) + 2 ** -11 * mag).all()


@pytest.mark.parametrize("rows", [1, 80])
def test_value_scales_near_the_ends_of_fp32(rows):
    # the result is in range although the sum of the values under the scale is not
    B, d, top = 16, 64, 64
    rng = np.random.default_rng(53)
    q = _bf16(rng, rows, 4, d)
    codes = torch.full((top, B, 2, d), 448.0, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    table, sel = _dev(np.tile(np.arange(top), (rows, 1))), _dev(np.tile(np.arange(top), (rows, 2, 1)))
    for e in (112, -120):
        out = torch.empty_like(q)
        ops.decode_selected(out, q, codes, codes, table, _dev([B * top] * rows), sel, 1e-3,
                            _dev([1e-3], torch.float32), _dev([2.0 ** e], torch.float32))
        want = 448.0 * 2.0 ** e  # the mean of equal values; the weights' errors cancel but for 2^-11
        assert (np.abs(_np(out) - want) <= (2 ** -8 + 2 ** -11) * want).all()


# ------------------------------------------------------------ rope_and_cache

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("tokens,H,Hkv,d,rot,adjacent", [(41, 4, 2, 64, 32, False), (41, 8, 2, 128, 48, True),
                                                        (2500, 16, 4, 128, 64, False), (2501, 6, 3, 64, 16, True)])
def test_what_is_not_rotated_keeps_its_bits(tokens, H, Hkv, d, rot, adjacent, kv):
    # values, and the channels from rot_dim on, NaN of every kind among them
    c = _rope_case(tokens, H, Hkv, d, rot, None, False, adjacent, kv, seed=54)
    rng = np.random.default_rng(55)
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    for name, first in (("q", rot), ("k", rot), ("v", 0)):
        t = c[name] = c[name].contiguous()
        odd = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, t[..., first:].shape).astype(np.int16)).to(DEV)
        odd[:, :, ::5] = torch.from_numpy(rng.choice(np.array([0x7f81, 0x7fff, -1, -127, 0x7f80, -128, -32768, 1], np.int16),
                                                     tuple(odd[:, :, ::5].shape))).to(DEV)
        bits(t)[..., first:] = odd
    kc, vc = c["kc"].clone(), c["vc"].clone()
    out = _rope_run(c)
    assert torch.equal(bits(out)[..., rot:], bits(c["q"])[..., rot:])
    ops.reshape_and_cache(c["k"], c["v"], kc, vc, _dev(c["slots"]), c["ks"], c["vs"])  # the plain write
    raw = lambda t: t.view(torch.uint8)  # noqa: E731
    w = kc.element_size()
    assert torch.equal(raw(c["vc"]), raw(vc))
    assert torch.equal(raw(c["kc"])[..., rot * w:], raw(kc)[..., rot * w:])


# ----------------------------------------------------------- tensors' memory

def test_outputs_that_are_lazy_clones_are_written_alone():
    # a tensor that shares its memory until it is written: the other keeps what it held
    rng = np.random.default_rng(56)
    c = _rope_case(40, 4, 2, 64, 32, None, False, False, "bf16", seed=57)
    shared = {x: c[x].clone() for x in ("kc", "vc")}
    kept = {x: t.clone() for x, t in shared.items()}
    want_q = _rope_run(c)
    k_want, v_want = c["kc"], c["vc"]
    c["kc"], c["vc"] = (torch._lazy_clone(shared[x]) for x in ("kc", "vc"))
    base = torch.full_like(want_q, 3.0)
    out = torch._lazy_clone(base)
    _rope_run(c, out=out)
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert same(out, want_q) and same(c["kc"], k_want) and same(c["vc"], v_want)
    assert (base == 3.0).all() and all(same(shared[x], kept[x]) for x in shared)
    # in place on a lazy clone: the queries are its own
    q0 = c["q"].contiguous()
    q = torch._lazy_clone(q0)
    before = q0.clone()
    _rope_run(c, out=q, q=q)
    assert same(q, want_q) and same(q0, before)

    NB, B, top = 12, 16, 5
    kc, vc = _bf16(rng, NB, B, 2, 64), _bf16(rng, NB, B, 2, 64)
    codes0, scales0 = ops.alloc_block_ranges(kc)
    codes, scales = torch._lazy_clone(codes0), torch._lazy_clone(scales0)
    ops.summarize_blocks(kc, _dev(np.arange(NB) * B + B - 1), codes, scales)
    assert (codes0 == 0).all() and (scales0 == 0).all() and (scales > 0).all()
    q = _bf16(rng, 1, 4, 64)
    table, lens = _dev(np.arange(NB)[None]), _dev([NB * B])
    sel0 = torch.full((1, 2, top), -5, device=DEV, dtype=torch.int32)
    sel = torch._lazy_clone(sel0)
    ops.select_blocks(sel, q, codes, scales, table, lens, B)
    assert (sel0 == -5).all() and (sel >= 0).all()
    out0 = torch.full_like(q, 9.0)
    out = torch._lazy_clone(out0)
    ops.decode_selected(out, q, kc, vc, table, lens, sel, 0.125)
    want, mag = bs.decode_selected(_np(q)[0], _np(kc), _np(vc), np.arange(NB), NB * B, sel[0].cpu().numpy(), 0.125)
    assert (out0 == 9.0).all()
    assert (np.abs(_np(out)[0] - want) <= 2 ** -8 * np.abs(want) + 2 ** -11 * mag).all()
