"""The scored step's prompt tiles: steps of more than 65535 new tokens."""
import numpy as np
import pytest
import torch

from tests.test_gpu_scored import _attn_case, _check_rows, _dev
from tests.test_gpu_scored_edges import _rows, _step, _varlen

pytestmark = pytest.mark.gpu


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
