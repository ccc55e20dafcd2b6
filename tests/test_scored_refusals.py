"""What the scored step's calls refuse, before any device work: the C entry
points by status, the binding by ValueError."""
import ctypes

import pytest
import torch

from paged_kv_cache_108_gb300 import _lib, ops

FAKE = ctypes.c_void_p(0x10000000)  # never dereferenced: validation fails first
OTHER = ctypes.c_void_p(0x90000000)
ODD = ctypes.c_void_p(0x10000002)
OK, INVALID, UNSUPPORTED = _lib.PA_OK, _lib.PA_ERR_INVALID, _lib.PA_ERR_UNSUPPORTED
BIG = 1 << 40  # bytes of a workspace that is large enough


def _desc(**kw):
    d = dict(num_blocks=32, block_size=16, num_kv_heads=2, head_dim=64, dtype=0)
    d.update(kw)
    return _lib.CacheDesc(**d)


def _rope(**kw):
    d = dict(rot_dim=64, max_position=100, num_axes=1, sections=(32, 0, 0, 0), turn=0, adj=0)
    d.update(kw)
    return _lib.RopeDesc(d["rot_dim"], d["max_position"], d["num_axes"],
                         (ctypes.c_int32 * 4)(*d["sections"]), d["turn"], d["adj"])


@pytest.mark.parametrize("kw,want", [
    (dict(desc=_desc(head_dim=96)), UNSUPPORTED),
    (dict(desc=_desc(dtype=3)), INVALID),
    (dict(desc=_desc(dtype=1)), INVALID),                       # e4m3 without scales
    (dict(desc=_desc(dtype=2)), INVALID),                       # int8 without units
    (dict(desc=_desc(dtype=2), ks=ODD, vs=FAKE), INVALID),
    (dict(ks=FAKE, vs=FAKE), INVALID),                          # bf16 with scales
    (dict(n=-1), INVALID),
    (dict(heads=-1), INVALID),
    (dict(rope=_rope(rot_dim=24)), UNSUPPORTED),
    (dict(rope=_rope(rot_dim=-16)), UNSUPPORTED),
    (dict(rope=_rope(rot_dim=80)), UNSUPPORTED),
    (dict(rope=_rope(max_position=0)), INVALID),
    (dict(rope=_rope(num_axes=5)), UNSUPPORTED),
    (dict(rope=_rope(num_axes=3, sections=(8, 12, 11, 0))), INVALID),
    (dict(pos=None), INVALID),
    (dict(table=None), INVALID),
    (dict(qw=FAKE), INVALID),                                   # one weight alone
    (dict(kw=FAKE), INVALID),
    (dict(qw=ODD, kw=FAKE), INVALID),
    (dict(qw=FAKE, kw=FAKE, eps=-1e-6), INVALID),
    (dict(qw=FAKE, kw=FAKE, eps=float("nan")), INVALID),
    (dict(qw=FAKE, kw=FAKE, eps=float("inf")), INVALID),
    (dict(qs=248), INVALID),
    (dict(k_stride=120), INVALID),
    (dict(key=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(q_out=FAKE, qs=512), INVALID),                        # in place, rows apart
    (dict(desc=_desc(dtype=2), ks=OTHER, vs=FAKE), INVALID),    # q_out over the units
    (dict(heads=32768 - 3, qs=1 << 26), UNSUPPORTED),
    (dict(n=0, q_out=None, key=None), OK),
    (dict(n=0, rope=_rope(rot_dim=0, max_position=0, num_axes=0), pos=None, table=None), OK),
])
def test_norm_rope_and_cache_refuses(kw, want):
    a = dict(desc=_desc(), rope=_rope(), q_out=OTHER, q=FAKE, qs=256, heads=4, key=FAKE,
             k_stride=128, n=5, slots=FAKE, pos=FAKE, table=FAKE, qw=None, kw=None, eps=1e-6,
             ks=None, vs=None)
    a.update(kw)
    assert _lib.lib().pa_norm_rope_and_cache(
        a["q_out"], a["q"], a["qs"], a["heads"], a["key"], a["k_stride"], FAKE, 128, FAKE, FAKE,
        a["desc"], a["slots"], a["pos"], a["table"], a["rope"], a["qw"], a["kw"],
        ctypes.c_float(a["eps"]), a["n"], a["ks"], a["vs"], None) == want
    if want != OK:
        assert "pa_norm_rope_and_cache" in _lib.lib().pa_last_error().decode()


@pytest.mark.parametrize("kw,want", [
    (dict(desc=_desc(block_size=24)), UNSUPPORTED),
    (dict(desc=_desc(dtype=2)), INVALID),
    (dict(desc=_desc(dtype=1)), INVALID),
    (dict(desc=_desc(num_kv_heads=32769)), UNSUPPORTED),
    (dict(ks=FAKE, vs=FAKE), INVALID),
    (dict(rows=-1), INVALID),
    (dict(seqs=-1), INVALID),
    (dict(max_blocks=0), INVALID),
    (dict(ko=None), INVALID),
    (dict(ko=ODD), INVALID),
    (dict(starts=None), INVALID),
    (dict(first=ODD), INVALID),
    (dict(ko=FAKE), INVALID),                                    # over the cache
    (dict(vo=ctypes.c_void_p(0x10000000 - 512)), INVALID),       # its last rows over the cache
    (dict(vo=ctypes.c_void_p(0x90000000 + 256)), INVALID),       # the outputs over each other
    (dict(rows=0, ko=None), OK),
    (dict(seqs=0, ko=None), OK),
])
def test_gather_cache_refuses(kw, want):
    a = dict(desc=_desc(), ko=OTHER, vo=ctypes.c_void_p(0xA0000000), seqs=2, rows=7, max_blocks=3,
             starts=FAKE, first=None, ks=None, vs=None)
    a.update(kw)
    assert _lib.lib().pa_gather_cache(a["ko"], a["vo"], FAKE, FAKE, a["desc"], FAKE, a["max_blocks"],
                                      FAKE, a["first"], a["starts"], a["seqs"], a["rows"], a["ks"],
                                      a["vs"], None) == want


SCORED = [
    (dict(desc=_desc(num_blocks=0)), INVALID),
    (dict(desc=_desc(dtype=1)), INVALID),
    (dict(desc=_desc(dtype=2)), INVALID),
    (dict(ks=FAKE), INVALID),
    (dict(heads=5), INVALID),
    (dict(heads=6), UNSUPPORTED),                  # GQA group 3
    (dict(heads=32), UNSUPPORTED),                 # GQA group 16
    (dict(max_blocks=0), INVALID),
    (dict(max_blocks=1 << 27), UNSUPPORTED),       # 2^31 tokens a sequence
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(cap=-1.0), INVALID),
    (dict(cap=float("nan")), INVALID),
    (dict(cap=float("inf")), INVALID),
    (dict(cap=1e-7), UNSUPPORTED),
    (dict(cap=1e7), UNSUPPORTED),
    (dict(window=-1), INVALID),
    (dict(slopes=ctypes.c_void_p(0x10000002)), INVALID),
    (dict(q=None), INVALID),
    (dict(q=ODD), INVALID),
    (dict(out=None), INVALID),
    (dict(lens=None), INVALID),
    (dict(lens=ODD), INVALID),
    (dict(ws=None), INVALID),
    (dict(ws=ctypes.c_void_p(0x10000080)), INVALID),
    (dict(bytes=255), INVALID),
]


def _scored(kw):
    a = dict(desc=_desc(), heads=4, max_blocks=7, rows=3, seqs=3, q=FAKE, out=FAKE, lens=FAKE,
             scale=0.1, cap=50.0, window=0, slopes=None, ks=None, ws=FAKE, bytes=BIG, starts=FAKE,
             prefix=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,want", SCORED + [
    (dict(seqs=-1), INVALID),
    (dict(desc=_desc(num_kv_heads=32769), heads=32769), UNSUPPORTED),
    (dict(seqs=1 << 27), UNSUPPORTED),
    (dict(seqs=0, q=None), OK),
])
def test_decode_scored_refuses(kw, want):
    a = _scored(kw)
    assert _lib.lib().pa_decode_scored(
        a["out"], a["q"], FAKE, FAKE, a["desc"], FAKE, a["max_blocks"], a["lens"], a["seqs"],
        a["heads"], ctypes.c_float(a["scale"]), _lib.ScoreDesc(a["cap"], a["window"], a["slopes"]),
        a["ks"], a["ks"], a["ws"], a["bytes"], None) == want
    if want != OK:
        assert "pa_decode_scored" in _lib.lib().pa_last_error().decode()


@pytest.mark.parametrize("kw,want", SCORED + [
    (dict(rows=-1), INVALID),
    (dict(seqs=0), INVALID),                       # tokens without requests
    (dict(starts=None), INVALID),
    (dict(starts=ODD), INVALID),
    (dict(prefix=ODD), INVALID),
    (dict(desc=_desc(head_dim=128), rows=40, bytes=1 << 18), INVALID),  # below tiles and rows alike
    (dict(rows=0, q=None), OK),
])
def test_varlen_scored_refuses(kw, want):
    a = _scored(kw)
    assert _lib.lib().pa_varlen_scored(
        a["out"], a["q"], FAKE, FAKE, a["desc"], FAKE, a["max_blocks"], a["lens"], a["starts"],
        a["seqs"], a["rows"], a["heads"], ctypes.c_float(a["scale"]),
        _lib.ScoreDesc(a["cap"], a["window"], a["slopes"]), a["prefix"], a["ks"], a["ks"], a["ws"],
        a["bytes"], None) == want
    if want != OK:
        assert "pa_varlen_scored" in _lib.lib().pa_last_error().decode()


def test_workspace_sizes():
    size = _lib.lib().pa_scored_workspace_size
    assert size(-1, 4, 2, 64) == size(3, 5, 2, 64) == size(3, 4, 0, 64) == size(3, 4, 2, 0) == 0
    assert size(3, 4, 2, 64) > 256
    assert size(100000, 4, 2, 64) == 256           # nothing is split
    assert size(64, 32, 8, 128) >= size(8, 32, 8, 128) > 256


@pytest.mark.parametrize("call", ["pa_decode", "pa_copy_blocks", "pa_summarize_blocks"])
def test_other_calls_refuse_8_bit_rows(call):
    lib, d = _lib.lib(), _desc(dtype=2)
    if call == "pa_decode":
        st = lib.pa_decode(FAKE, FAKE, FAKE, FAKE, d, FAKE, 7, FAKE, 3, 4, ctypes.c_float(0.1), FAKE,
                           FAKE, FAKE, BIG, None)
    elif call == "pa_copy_blocks":
        st = lib.pa_copy_blocks(FAKE, FAKE, d, FAKE, 3, None)
    else:
        st = lib.pa_summarize_blocks(FAKE, d, FAKE, 3, FAKE, FAKE, None)
    assert st == INVALID


# ---------------------------------------------------------------- binding

H, HKV, D, B, NB = 8, 2, 64, 16, 10
BF, F32, I32, I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def _z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def _write_args(**kw):
    a = dict(q_out=_z(5, H, D), query=_z(5, H, D), key=_z(5, HKV, D), value=_z(5, HKV, D),
             k_cache=_z(NB, B, HKV, D), v_cache=_z(NB, B, HKV, D), slot_mapping=_z(5, dtype=I32),
             positions=_z(5, dtype=I32), cos_sin=_z(100, D, dtype=F32))
    a.update(kw)
    return a


INT8 = dict(k_cache=_z(NB, B, HKV, D, dtype=I8), v_cache=_z(NB, B, HKV, D, dtype=I8))


@pytest.mark.parametrize("kw,match", [
    (dict(key=_z(4, HKV, D)), "one row per slot"),
    (dict(q_out=_z(5, H + 1, D)), "query and q_out"),
    (dict(positions=None), "together"),
    (dict(cos_sin=None), "together"),
    (dict(cos_sin=_z(100, 0, dtype=F32)), "columns"),
    (dict(positions=_z(4, dtype=I32)), "positions must be"),
    (dict(q_weight=_z(D - 1, dtype=F32), k_weight=_z(D, dtype=F32)), "q_weight and k_weight must be"),
    (dict(eps="x"), "eps must be a number"),
    (INT8, "need k_scale"),
    (dict(INT8, k_scale=_z(1, dtype=F32), v_scale=_z(1, dtype=F32)), "must be .10, 16, 2."),
    (dict(INT8, v_cache=_z(NB, B, HKV, D)), "same shape and dtype"),
    (dict(k_scale=_z(1, dtype=F32), v_scale=_z(1, dtype=F32)), "only for fp8"),
    ({}, "CUDA"),
])
def test_binding_refuses_writes(kw, match):
    with pytest.raises(ValueError, match=match):
        ops.norm_rope_and_cache(**_write_args(**kw))


@pytest.mark.parametrize("kw,match", [
    (dict(k_out=_z(7, HKV + 1, D)), "k_out and v_out"),
    (dict(v_out=_z(6, HKV, D)), "k_out and v_out"),
    (dict(block_tables=_z(3, dtype=I32)), "block_tables"),
    (dict(context_lens=_z(2, dtype=I32)), "context_lens needs 3"),
    (dict(out_start_loc=_z(3, dtype=I32)), "out_start_loc needs num_seqs . 1 = 4"),
    (dict(first_tokens=_z(2, dtype=I32)), "first_tokens needs 3"),
    (dict(k_cache=_z(NB, B, HKV, D, dtype=torch.uint8), v_cache=_z(NB, B, HKV, D, dtype=torch.uint8),
          k_scale=_z(2, dtype=F32), v_scale=_z(1, dtype=F32)), "one element"),
    ({}, "CUDA"),
])
def test_binding_refuses_gathers(kw, match):
    a = dict(k_out=_z(7, HKV, D), v_out=_z(7, HKV, D), k_cache=_z(NB, B, HKV, D),
             v_cache=_z(NB, B, HKV, D), block_tables=_z(3, 4, dtype=I32),
             context_lens=_z(3, dtype=I32), out_start_loc=_z(4, dtype=I32))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        ops.gather_cache(**a)


@pytest.mark.parametrize("kw,match", [
    (dict(out=_z(2, H, D)), "q and out"),
    (dict(q=_z(3, H, 128), out=_z(3, H, 128)), "head_dim"),
    (dict(block_tables=_z(2, 4, dtype=I32)), "block_tables must be .3"),
    (dict(context_lens=_z(2, dtype=I32)), "context_lens needs 3"),
    (dict(slopes=_z(H - 1, dtype=F32)), "slopes must be"),
    (dict(cap=None), "cap must be a number"),
    (dict(window=1.5), "window must be an integer"),
    (dict(scale="x"), "scale must be a number"),
    (dict(workspace=None), "workspace must be"),
    ({}, "CUDA"),
])
def test_binding_refuses_decodes(kw, match):
    a = dict(out=_z(3, H, D), q=_z(3, H, D), k_cache=_z(NB, B, HKV, D), v_cache=_z(NB, B, HKV, D),
             block_tables=_z(3, 4, dtype=I32), context_lens=_z(3, dtype=I32), scale=0.1,
             workspace=_z(1 << 12, dtype=torch.uint8))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        ops.decode_scored(**a)


@pytest.mark.parametrize("kw,match", [
    (dict(block_tables=_z(2, 4, dtype=I32)), "block_tables must be .3"),
    (dict(query_start_loc=_z(3, dtype=I32)), "query_start_loc needs num_seqs . 1 = 4"),
    (dict(prefix_lens=_z(2, dtype=I32)), "prefix_lens needs 3"),
    (dict(slopes=_z(H, 1, dtype=F32)), "slopes must be"),
    ({}, "CUDA"),
])
def test_binding_refuses_prompts(kw, match):
    a = dict(out=_z(9, H, D), q=_z(9, H, D), k_cache=_z(NB, B, HKV, D), v_cache=_z(NB, B, HKV, D),
             block_tables=_z(3, 4, dtype=I32), seq_lens=_z(3, dtype=I32),
             query_start_loc=_z(4, dtype=I32), scale=0.1, workspace=_z(1 << 12, dtype=torch.uint8))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        ops.varlen_scored(**a)
