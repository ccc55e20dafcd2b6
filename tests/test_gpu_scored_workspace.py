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


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_a_long_row_among_many(kv):
    """A batch of many short sequences with one of 64 K tokens."""
    lens = [int(x) for x in np.random.default_rng(2).integers(0, 60, 600)]
    lens[217] = 65_536
    c = _attn_case(122, kv, lens, 8, 4, 64, 16)
    q = _bf16(c["rng"], len(lens), 8, 64)
    out = torch.full_like(q, 7.0)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"],
                      **_mod(c, 30.0, 0, False))
    rows = [(i, i, n - 1) for i, n in enumerate(lens)]
    _check_rows(c, out, q, rows[::9] + [rows[217]], 30.0, 0, False)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("H,Hkv,width", [(16, 16, 1104), (32, 16, 1104), (16, 16, 4000)])
def test_batches_of_many_heads_whole_and_split(kv, H, Hkv, width):
    """Both sides of the rule that hands whole rows of many heads to CTAs: the
    table's width bounds the lengths."""
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 40, 300)]
    lens[7], lens[299] = 1090, 700
    c = _attn_case(123, kv, lens, H, Hkv, 64, 16)
    wide = np.full((300, width // 16), -1, np.int64)
    wide[:, :c["tables"].shape[1]] = c["tables"]
    c["tables"] = wide
    q = _bf16(c["rng"], len(lens), H, 64)
    out = torch.full_like(q, 7.0)
    ops.decode_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"],
                      **_mod(c, 0.0, 0, True))
    rows = [(i, i, n - 1) for i, n in enumerate(lens)]
    _check_rows(c, out, q, rows[::11] + [rows[7], rows[299]], 0.0, 0, True)


def test_more_rows_than_threads_of_a_cta():
    """The search for a CTA's rows, each thread over several: lengths of zero and
    rows of no request among them, row by row over 8-bit rows."""
    rng = np.random.default_rng(4)
    new = [int(x) for x in rng.integers(0, 5, 700)]
    lens = [n + int(x) * int(x) for n, x in zip(new, rng.integers(0, 18, 700))]
    lens[13] = max(0, new[13] - 1)  # more new than there are
    c = _attn_case(124, "int8", lens, 2, 1, 64, 16)
    starts = np.cumsum([9] + new)
    q = _bf16(rng, int(starts[-1]) + 50, 2, 64)
    outs = []
    for _ in range(2):
        out = torch.full_like(q, 7.0)
        ops.varlen_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), _dev(starts),
                          c["scale"], **_mod(c, 30.0, 0, False))
        outs.append(out)
    assert torch.equal(*outs)
    assert (outs[0][:9] == 7.0).all() and (outs[0][int(starts[-1]):] == 7.0).all()
    rows = [(int(starts[i]) + j, i, n - t + j) for i, (n, t) in enumerate(zip(lens, new)) if n >= t
            for j in range(t)]
    _check_rows(c, outs[0], q, rows[::13] + rows[-2:], 30.0, 0, False)


def test_the_error_word_of_a_new_workspace_is_zero():
    for rows, d in ((3, 64), (40, 128)):
        n = ops.scored_workspace_size(rows, 8, 2, d)
        torch.cuda.empty_cache()
        junk = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # its memory is handed on
        del junk
        ws = ops.alloc_scored_workspace(rows, 8, 2, d)
        assert int(ws[:4].view(torch.int32).item()) == 0


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_decode_takes_no_room_for_tiles(kv):
    """Without a workspace of its own a call allocates what it splits rows in,
    with the same result."""
    lens = [900 + 7 * i for i in range(40)]
    c = _attn_case(125, kv, lens, 8, 2, 128, 16)
    q = _bf16(c["rng"], len(lens), 8, 128)
    want = _decode(c, q, ops.alloc_scored_workspace(len(lens), 8, 2, 128))
    args = (q, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"])
    mod, out = _mod(c, 30.0, 0, False), torch.empty_like(q)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    ops.decode_scored(out, *args, **mod)
    assert torch.cuda.max_memory_allocated() - before < 8 << 20
    assert torch.equal(out, want)
