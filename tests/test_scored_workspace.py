"""Sizes of the scored step's workspaces: one for the largest batch serves
every smaller one."""
import pytest

from paged_kv_cache_108_gb300 import _lib, ops

ROWS = [0, 1, 2, 8, 9, 100, 227, 228, 300, 2000, 20_000, 10 ** 5, 10 ** 6]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 2), (32, 8), (32, 32), (64, 8), (320, 320), (400, 400)])
def test_sizes_do_not_fall_as_rows_grow(H, Hkv, d):
    sizes = [ops.scored_workspace_size(n, H, Hkv, d) for n in ROWS]
    assert sizes == sorted(sizes) and sizes[1] > 256
    # what the library asks for at any number of rows is within
    asked = [_lib.lib().pa_scored_workspace_size(n, H, Hkv, d) for n in ROWS]
    assert all(max(asked[:i + 1]) <= s for i, s in enumerate(sizes))


def test_bad_sizes_stay_zero():
    assert ops.scored_workspace_size(-1, 4, 2, 64) == ops.scored_workspace_size(3, 5, 2, 64) == 0
