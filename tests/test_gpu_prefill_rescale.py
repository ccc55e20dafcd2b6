"""Prefill tiles on peaked logits: rows whose running max grows by more than
the rescale threshold from one 128-key chunk to a later one, alone among the
rows of their warp.  The scale is several times the usual one, so that a
logit's spread is about 8 in log2 units and such rows are common."""
import pytest
import torch

from tests.test_gpu_prefill import _check
from tests.test_gpu_varlen import _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (8, 8), (8, 1)])
def test_tiles_rescale_single_rows(kv, hq, hkv):
    c = _setup([900, 450, 300], [300, 450, 1], hq, hkv, 128, 16, kv, seed=170)
    _check(c, 0.5)
    torch.cuda.synchronize()
