"""What the normalising write writes must lie apart: the two caches, and the
units of 8-bit rows.  By the C entry point, before any device work."""
import ctypes

import pytest

from paged_kv_cache_108_gb300 import _lib

OK, INVALID = _lib.PA_OK, _lib.PA_ERR_INVALID
P = ctypes.c_void_p
SLOTS, ROW = 32 * 16, 2 * 64  # of the cache below; elements a slot
POOL = {0: SLOTS * ROW * 2, 1: SLOTS * ROW, 2: SLOTS * ROW}  # bytes by dtype
UNITS = SLOTS * 2 * 4
K, V, KS, VS = 0x10000000, 0x20000000, 0x30000000, 0x40000000  # never dereferenced


def _write(dtype, k=K, v=V, ks=KS, vs=VS, n=5):
    desc = _lib.CacheDesc(32, 16, 2, 64, dtype)
    rope = _lib.RopeDesc(0, 0, 0, (ctypes.c_int32 * 4)(), 0, 0)
    src = P(0x70000000)
    status = _lib.lib().pa_norm_rope_and_cache(
        P(0x80000000), src, 256, 4, src, 128, src, 128, P(k), P(v), desc, P(0x90000000), None, None,
        rope, None, None, ctypes.c_float(1e-6), n, P(ks) if dtype else None, P(vs) if dtype else None,
        None)
    return status, _lib.lib().pa_last_error().decode()


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("by", ["same", "first", "last"])
def test_the_caches_must_not_overlap(dtype, by):
    v = {"same": K, "first": K - POOL[dtype] + 16, "last": K + POOL[dtype] - 16}[by]
    status, why = _write(dtype, v=v)
    assert status == INVALID and "pa_norm_rope_and_cache: k_cache and v_cache overlap" in why


@pytest.mark.parametrize("at,what", [
    (dict(vs=KS), "k_scale and v_scale"),
    (dict(vs=KS + UNITS - 4), "k_scale and v_scale"),
    (dict(vs=KS - UNITS + 4), "k_scale and v_scale"),
    (dict(ks=K), "units overlap a cache"),
    (dict(ks=V + POOL[2] - 4), "units overlap a cache"),
    (dict(vs=K - UNITS + 4), "units overlap a cache"),
    (dict(vs=V + 64), "units overlap a cache"),
])
def test_the_units_must_lie_apart(at, what):
    status, why = _write(2, **at)
    assert status == INVALID and what in why


def test_nothing_is_refused_without_tokens():
    for dtype in (0, 1, 2):
        assert _write(dtype, v=K, vs=KS, n=0)[0] == OK
