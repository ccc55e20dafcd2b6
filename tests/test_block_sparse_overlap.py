"""pa_rope_and_cache refuses a q_out that lies over what the call still reads,
before any device work."""
import ctypes

import pytest

from paged_kv_cache_108_gb300 import _lib
from tests.test_block_sparse_refusals import INVALID, _rope_call


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
