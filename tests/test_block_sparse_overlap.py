"""pa_rope_and_cache refuses a q_out that lies over what the call still reads,
before any device work."""
import ctypes

import pytest

from paged_kv_cache_108_gb300 import _lib
from tests.test_block_sparse_refusals import INVALID, _desc, _rope, _rope_call


def _at(address):
    return ctypes.c_void_p(address)


@pytest.mark.parametrize("n", [2 ** 30, 2 ** 31 - 1])
def test_an_overlap_is_found_whatever_the_number_of_tokens(n):
    # the output's bytes pass 32 bits; it begins a row into the queries
    assert _rope_call(n=n, q=_at(0x100000), q_out=_at(0x100000 + 512)) == INVALID
    assert "overlaps query" in _lib.lib().pa_last_error().decode()
    # and ends in them
    assert _rope_call(n=n, q=_at(0x10000000000), q_out=_at(0x10000000000 - 512)) == INVALID
    assert "overlaps query" in _lib.lib().pa_last_error().decode()


K, V, KC, VC, Q = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000


def _call(q_out, n=5, heads=4, q_stride=256, k_stride=256, kv=(K, V, KC, VC), dtype=0):
    # 4 query and 2 KV heads of 64 channels: rows of 512 and 256 bytes
    scale = _at(0x100000) if dtype else None
    return _lib.lib().pa_rope_and_cache(
        _at(q_out), _at(Q), q_stride, heads, _at(kv[0]), k_stride, _at(kv[1]), 128, _at(kv[2]),
        _at(kv[3]), _desc(dtype=dtype), _at(0x100000), _at(0x100000), _at(0x100000), _rope(), n,
        scale, scale, None)


POOL = 32 * 16 * 128 * 2  # bytes of a bf16 cache


@pytest.mark.parametrize("q_out,kw,match", [
    (K, {}, "key or value"),
    (K + 4 * 512 + 240, {}, "key or value"),             # the last key row's last 16 bytes
    (K - 5 * 512 + 16, {}, "key or value"),              # q_out ends in the first
    (K + 256, dict(k_stride=4096, n=30), "key or value"),  # runs from between two rows into the next
    (V, {}, "key or value"),
    (V + 5 * 256 - 16, {}, "key or value"),
    (KC, {}, "a cache"),
    (KC + POOL - 16, {}, "a cache"),
    (VC - 5 * 512 + 16, {}, "a cache"),
    (VC + POOL // 2 - 16, dict(dtype=1), "a cache"),
    (Q + 512, dict(q_stride=512, n=2), "query"),         # between the rows, and into the second
])
def test_an_output_over_what_the_call_reads_is_refused(q_out, kw, match):
    assert _call(q_out, **kw) == INVALID
    assert match in _lib.lib().pa_last_error().decode()


def test_strides_beyond_any_address_are_refused():
    for kw in (dict(q_stride=2 ** 40 + 8), dict(k_stride=2 ** 62), dict(q_stride=2 ** 62, n=2 ** 31 - 1)):
        assert _call(0x9000000, **kw) == INVALID
        assert "strides" in _lib.lib().pa_last_error().decode()


def test_rows_of_one_buffer_do_not_meet_themselves():
    # the arithmetic of the check, restated row by row
    def meet(base, stride, row, n, o0, o1):
        t = 0 if o0 < base + row else (o0 - base - row) // stride + 1
        return t < n and base + t * stride < o1

    for stride in (16, 24, 48):
        for n in (1, 2, 5):
            for o0 in range(60, 400):
                for size in (8, 16, 100):
                    want = any(100 + t * stride < o0 + size and o0 < 100 + t * stride + 16 for t in range(n))
                    assert meet(100, stride, 16, n, o0, o0 + size) == want
