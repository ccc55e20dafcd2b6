"""Workspaces of the scored step that are allocated once: for the largest
batch, and for errors to be read from.  Tolerances as in the parity tests."""
import numpy as np
import pytest
import torch

from paged_kv_cache_108_gb300 import ops
from tests.test_gpu_scored import DEV, _attn_case, _bf16, _check_rows, _dev, _mod

pytestmark = pytest.mark.gpu


def _decode(c, q, ws):
    out = torch.full_like(q, 7.0)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(c["lens"]), c["scale"],
                      workspace=ws, **_mod(c, 30.0, 0, False))
    _check_rows(c, out, q, [(i, i, n - 1) for i, n in enumerate(c["lens"])], 30.0, 0, False)
    return out


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_workspace_for_the_largest_batch_serves_all(kv, d):
    """Allocated for more rows than are ever split, used by a few long ones."""
    H, Hkv = 8, 4
    lens = [3000, 17, 900]
    c = _attn_case(121, kv, lens, H, Hkv, d, 16)
    q = _bf16(c["rng"], 3, H, d)
    for rows in (3, 300, 100000):
        ws = ops.alloc_scored_workspace(rows, H, Hkv, d)
        want = _decode(c, q, ws)
    # the bytes that many rows take by themselves serve a few too
    n = ops._lib.lib().pa_scored_workspace_size(10 ** 6, H, Hkv, d)
    _decode(c, q, torch.empty(n, dtype=torch.uint8, device=DEV))
    _decode(c, q, torch.empty(256, dtype=torch.uint8, device=DEV))
    assert torch.equal(want, _decode(c, q, None))
    out = torch.full_like(q, 7.0)
    ops.varlen_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), _dev([0, 1, 2, 3]),
                      c["scale"], workspace=torch.empty(256, dtype=torch.uint8, device=DEV),
                      **_mod(c, 30.0, 0, False))
    _check_rows(c, out, q, [(i, i, n - 1) for i, n in enumerate(lens)], 30.0, 0, False)
