"""What the block-sparse step's calls refuse, before any device work: the C
entry points by status, the binding by ValueError."""
import ctypes

import pytest
import torch

from paged_kv_cache_108_gb300 import _lib, ops

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: validation fails first
OTHER = ctypes.c_void_p(0x900000)
ODD = ctypes.c_void_p(0x100002)
OK, INVALID, UNSUPPORTED = _lib.PA_OK, _lib.PA_ERR_INVALID, _lib.PA_ERR_UNSUPPORTED


def _desc(**kw):
    d = dict(num_blocks=32, block_size=16, num_kv_heads=2, head_dim=64, dtype=0)
    d.update(kw)
    return _lib.CacheDesc(**d)


def _rope(**kw):
    d = dict(rot_dim=64, max_position=100, num_axes=1, sections=(32, 0, 0, 0), turn=0, adj=0)
    d.update(kw)
    return _lib.RopeDesc(d["rot_dim"], d["max_position"], d["num_axes"],
                         (ctypes.c_int32 * 4)(*d["sections"]), d["turn"], d["adj"])


def _rope_call(desc=None, rope=None, q_out=OTHER, q=FAKE, qs=256, heads=4, key=FAKE, ks_=128,
               vs_=128, n=5, slots=FAKE, pos=FAKE, table=FAKE, kscale=None, vscale=None):
    return _lib.lib().pa_rope_and_cache(q_out, q, qs, heads, key, ks_, FAKE, vs_, FAKE, FAKE,
                                        desc or _desc(), slots, pos, table, rope or _rope(), n,
                                        kscale, vscale, None)


@pytest.mark.parametrize("kw,want", [
    (dict(desc=_desc(head_dim=96)), UNSUPPORTED),
    (dict(desc=_desc(dtype=1)), INVALID),                       # e4m3 without scales
    (dict(kscale=FAKE, vscale=FAKE), INVALID),                  # bf16 with scales
    (dict(n=-1), INVALID),
    (dict(heads=-1), INVALID),
    (dict(rope=_rope(rot_dim=24)), UNSUPPORTED),
    (dict(rope=_rope(rot_dim=80)), UNSUPPORTED),
    (dict(rope=_rope(rot_dim=0)), UNSUPPORTED),
    (dict(rope=_rope(max_position=0)), INVALID),
    (dict(rope=_rope(num_axes=0)), INVALID),
    (dict(rope=_rope(num_axes=5)), UNSUPPORTED),
    (dict(rope=_rope(num_axes=3, sections=(8, 12, 11, 0))), INVALID),   # sum 31
    (dict(rope=_rope(num_axes=3, sections=(-4, 18, 18, 0))), INVALID),
    (dict(rope=_rope(num_axes=3, sections=(8, 12, 12, 0), turn=1)), INVALID),  # 1 + 3 * 11 > 31
    (dict(qs=248), INVALID),
    (dict(qs=260), INVALID),
    (dict(ks_=120), INVALID),
    (dict(vs_=132), INVALID),
    (dict(q_out=None), INVALID),
    (dict(key=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(pos=None), INVALID),
    (dict(table=None), INVALID),
    (dict(key=ODD), INVALID),
    (dict(q_out=FAKE, qs=512), INVALID),                        # in place, rows apart
    (dict(q_out=ctypes.c_void_p(0x100000 + 512)), INVALID),     # overlaps by a row
    (dict(heads=32768 - 3, qs=1 << 26), UNSUPPORTED),
    (dict(n=0, q_out=None, key=None), OK),
])
def test_rope_and_cache_refuses(kw, want):
    assert _rope_call(**kw) == want
    if want != OK:
        assert "pa_rope_and_cache" in _lib.lib().pa_last_error().decode()


@pytest.mark.parametrize("kw,want", [
    (dict(desc=_desc(block_size=24)), UNSUPPORTED),
    (dict(n=-1), INVALID),
    (dict(codes=None), INVALID),
    (dict(codes=ODD), INVALID),
    (dict(scales=ODD), INVALID),
    (dict(k=None), INVALID),
    (dict(desc=_desc(num_kv_heads=32769)), UNSUPPORTED),
    (dict(n=0, k=None), OK),
])
def test_summarize_blocks_refuses(kw, want):
    a = dict(desc=_desc(), n=3, k=FAKE, codes=FAKE, scales=FAKE)
    a.update(kw)
    assert _lib.lib().pa_summarize_blocks(a["k"], a["desc"], FAKE, a["n"], a["codes"], a["scales"],
                                          None) == want


ROWS = [
    (dict(desc=_desc(num_blocks=0)), INVALID),
    (dict(heads=5), INVALID),
    (dict(heads=6), UNSUPPORTED),                  # GQA group 3
    (dict(heads=32), UNSUPPORTED),                 # GQA group 16
    (dict(max_blocks=0), INVALID),
    (dict(rows=-1), INVALID),
    (dict(rows=4, seqs=3), INVALID),               # no row_seqs
    (dict(rows=1 << 30, seqs=3, row_seqs=FAKE), UNSUPPORTED),
    (dict(top=0), INVALID),
    (dict(q=None), INVALID),
    (dict(q=ODD), INVALID),
    (dict(selected=ODD), INVALID),
    (dict(lens=None), INVALID),
    (dict(rows=0, seqs=0, q=None), OK),
]


def _row_args(kw):
    a = dict(desc=_desc(), heads=4, max_blocks=7, rows=3, seqs=3, row_seqs=None, top=4, sink=1,
             recent=1, q=FAKE, selected=FAKE, lens=FAKE, scale=0.1, out=FAKE, ks=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,want", ROWS + [
    (dict(sink=-1), INVALID), (dict(recent=0), INVALID), (dict(sink=3, recent=2), INVALID),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID),
    (dict(max_blocks=196609), UNSUPPORTED),
])
def test_select_blocks_refuses(kw, want):
    a = _row_args(kw)
    assert _lib.lib().pa_select_blocks(a["selected"], a["q"], FAKE, FAKE, a["desc"], FAKE,
                                       a["max_blocks"], a["lens"], a["row_seqs"], a["rows"],
                                       a["seqs"], a["heads"], a["top"], a["sink"], a["recent"],
                                       None) == want


@pytest.mark.parametrize("kw,want", ROWS + [
    (dict(top=4097), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(out=None), INVALID),
    (dict(desc=_desc(dtype=1)), INVALID), (dict(ks=FAKE), INVALID),
])
def test_decode_selected_refuses(kw, want):
    a = _row_args(kw)
    assert _lib.lib().pa_decode_selected(a["out"], a["q"], FAKE, FAKE, a["desc"], FAKE,
                                         a["max_blocks"], a["lens"], a["row_seqs"], a["selected"],
                                         a["rows"], a["seqs"], a["heads"], a["top"],
                                         ctypes.c_float(a["scale"]), a["ks"], a["ks"],
                                         None) == want


# ---------------------------------------------------------------- binding

H, HKV, D, B, NB = 8, 2, 64, 16, 10
BF = torch.bfloat16


def _z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_checks_the_rotating_write():
    kc = _z(NB, B, HKV, D)
    good = dict(q_out=_z(3, H, D), query=_z(3, H, D), key=_z(3, HKV, D), value=_z(3, HKV, D),
                k_cache=kc, v_cache=kc.clone(), slot_mapping=_z(3, dtype=torch.int32),
                positions=_z(3, dtype=torch.int32), cos_sin=_z(9, D, dtype=torch.float32))
    for kw, match in [
            (dict(key=_z(4, HKV, D)), "one row per slot"),
            (dict(query=_z(2, H, D), q_out=_z(2, H, D)), "query and q_out"),
            (dict(q_out=_z(3, H + 1, D)), "query and q_out"),
            (dict(positions=_z(4, dtype=torch.int32)), "positions"),
            (dict(positions=_z(2, 4, dtype=torch.int32)), "positions"),
            (dict(positions=_z(3, 3, dtype=torch.int32)), "sections"),
            (dict(positions=_z(3, 3, dtype=torch.int32), sections=[16, 16]), "sections"),
            (dict(positions=_z(5, 3, dtype=torch.int32), sections=[8, 8, 8, 8, 0]), "at most 4"),
            (dict(cos_sin=_z(9, dtype=torch.float32)), "cos_sin"),
            (dict(k_scale=_z(1, dtype=torch.float32)), "only for fp8"),
            (dict(), "CUDA tensor")]:
        with pytest.raises(ValueError, match=match):
            ops.rope_and_cache(**{**good, **kw})


def test_binding_refuses_what_is_no_tensor_or_number():
    kc = _z(NB, B, HKV, D)
    codes, scales = ops.alloc_block_ranges(kc)
    slots = _z(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="slot_mapping must be a CUDA tensor"):
        ops.summarize_blocks(kc, [0, 1], codes, scales)
    with pytest.raises(ValueError, match="cache must be"):
        ops.summarize_blocks(kc[0], slots, codes, scales)
    with pytest.raises(ValueError, match="cache dtype"):
        ops.summarize_blocks(kc.float(), slots, codes, scales)
    i32 = torch.int32
    sel = dict(selected=_z(3, HKV, 4, dtype=i32), q=_z(3, H, D), codes=codes, scales=scales,
               block_tables=_z(3, 7, dtype=i32), context_lens=_z(3, dtype=i32))
    with pytest.raises(ValueError, match="block_size must be an integer"):
        ops.select_blocks(block_size=None, **sel)
    with pytest.raises(ValueError, match="recent does not fit"):
        ops.select_blocks(block_size=B, recent=2 ** 40, **sel)
    with pytest.raises(ValueError, match="scale must be a number"):
        ops.decode_selected(out=_z(3, H, D), q=_z(3, H, D), k_cache=kc, v_cache=kc.clone(),
                            block_tables=sel["block_tables"], context_lens=sel["context_lens"],
                            selected=sel["selected"], scale="0.1")
    rope = dict(q_out=_z(3, H, D), query=_z(3, H, D), key=_z(3, HKV, D), value=_z(3, HKV, D),
                k_cache=kc, v_cache=kc.clone(), slot_mapping=slots,
                positions=_z(2, 3, dtype=i32), cos_sin=_z(9, D, dtype=torch.float32))
    with pytest.raises(ValueError, match="sections"):
        ops.rope_and_cache(sections=[16, "16"], **rope)
    with pytest.raises(ValueError, match="sections"):
        ops.rope_and_cache(sections=32, **rope)
    with pytest.raises(ValueError, match="sections_in_turn"):
        ops.rope_and_cache(sections=[16, 16], sections_in_turn=torch.zeros(2), **rope)


def test_binding_checks_ranges_and_selections():
    kc = _z(NB, B, HKV, D)
    codes, scales = ops.alloc_block_ranges(kc)
    assert codes.shape == (NB, HKV, 2, D) and scales.shape == (NB, HKV)
    slots = _z(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="codes"):
        ops.summarize_blocks(kc, slots, codes[:-1], scales)
    with pytest.raises(ValueError, match="scales"):
        ops.summarize_blocks(kc, slots, codes, scales[:, :1])
    i32 = torch.int32
    good = dict(selected=_z(3, HKV, 4, dtype=i32), q=_z(3, H, D), block_tables=_z(3, 7, dtype=i32),
                context_lens=_z(3, dtype=i32))
    bad = [(dict(selected=_z(3, 1, 4, dtype=i32)), "selected"),
           (dict(selected=_z(2, HKV, 4, dtype=i32)), "selected"),
           (dict(block_tables=_z(2, 7, dtype=i32)), "block_tables"),
           (dict(context_lens=_z(2, dtype=i32)), "context_lens needs 3"),
           (dict(row_seqs=_z(2, dtype=i32)), "row_seqs needs 3"),
           (dict(q=_z(3, H, 128)), "head_dim"),
           (dict(), "CUDA tensor")]
    for kw, match in bad:
        with pytest.raises(ValueError, match=match):
            ops.select_blocks(codes=codes, scales=scales, block_size=B, **{**good, **kw})
        q = kw.get("q", good["q"])
        with pytest.raises(ValueError, match=match):
            ops.decode_selected(out=torch.empty_like(q), k_cache=kc, v_cache=kc.clone(), scale=0.1,
                                **{**good, **kw})
