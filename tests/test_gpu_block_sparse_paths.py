"""Block-sparse decode step on a GPU: every launch shape that calls of
ordinary sizes run, at 64 and 128 channels, and the step under capture, on
several streams and threads and around a swap.

Tolerances are those derived in test_gpu_block_sparse.py; selections, ranges
and repeated calls are equal.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import block_sparse as bs
from paged_kv_cache_108_gb300 import ops
from tests.test_gpu_block_sparse import (DEV, _bf16, _check_attend, _check_rope, _check_select, _codes_np, _dev,
                                         _junk_cache, _lists, _np, _ranges, _rope_case, _rope_run, _Step)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ rope_and_cache

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("tokens,H,Hkv,d,rot,sections,in_turn,adjacent", [
    (320, 32, 8, 128, 128, None, False, False),        # a token a CTA, several items a thread
    (2501, 20, 2, 128, 128, [16, 24, 24], False, False),  # two tokens a CTA, the last one alone
    (2433, 6, 1, 128, 64, [12, 10, 10], True, True),   # six
    (2500, 40, 4, 64, 64, None, False, True),
    (8001, 1, 1, 64, 32, None, False, False),          # eight
])
def test_rope_long_calls_of_every_kind(tokens, H, Hkv, d, rot, sections, in_turn, adjacent, kv):
    c = _rope_case(tokens, H, Hkv, d, rot, sections, in_turn, adjacent, kv, seed=60)
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    _check_rope(c, _rope_run(c), kc0, vc0)


def test_rope_long_call_in_place_and_skipped_tokens():
    c = _rope_case(2500, 16, 4, 128, 96, None, False, False, "bf16", seed=61)
    c["pos"][0, [0, 1, 777, 2499]] = [-1, 5000, -2 ** 31, 2 ** 31 - 1]
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    want = _rope_run(c)
    _check_rope(c, want, kc0, vc0, skipped=(0, 1, 777, 2499))
    k, v = c["kc"], c["vc"]
    c["kc"], c["vc"] = kc0.clone(), vc0.clone()
    q = c["q"].contiguous()
    before = q.clone()
    _rope_run(c, out=q, q=q)
    gone = torch.tensor([0, 1, 777, 2499], device=DEV)
    want[gone] = before[gone]  # a skipped token's row stays
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(q, want) and same(c["kc"], k) and same(c["vc"], v)


@pytest.mark.parametrize("heads", [4, 32])
def test_rope_of_one_token_in_its_projection(heads):
    # one token's queries are contiguous in the projection's output: in place there
    c = _rope_case(1, heads, 2, 128, 128, None, False, False, "bf16", seed=75)
    want = _rope_run(c)
    k = c["kc"].clone()
    row = torch.cat([c[x].reshape(1, -1) for x in ("q", "k", "v")], 1)
    q, c["k"], c["v"] = (x.view(1, -1, 128) for x in row.split([heads * 128, 256, 256], 1))
    c["kc"].zero_()
    kept = row[:, heads * 128:].clone()
    _rope_run(c, out=q, q=q)
    assert torch.equal(row[:, :heads * 128].view(1, heads, 128), want)
    assert torch.equal(row[:, heads * 128:], kept)
    slot = int(c["slots"][0])
    flat = lambda t: t.view(-1, 2, 128)[slot]  # noqa: E731
    assert torch.equal(flat(c["kc"]), flat(k))


def test_rope_without_query_heads_writes_the_cache():
    c = _rope_case(77, 8, 2, 128, 64, None, False, False, "bf16", seed=62)
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    _rope_run(c)
    k, v = c["kc"], c["vc"]
    c["kc"], c["vc"] = kc0.clone(), vc0.clone()
    none = torch.empty(77, 0, 128, device=DEV, dtype=torch.bfloat16)
    _rope_run(c, out=none, q=none)
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    assert torch.equal(bits(c["kc"]), bits(k)) and torch.equal(bits(c["vc"]), bits(v))
    assert not torch.equal(bits(k), bits(kc0)) and not torch.equal(bits(v), bits(vc0))


# --------------------------------------------------------- summarize_blocks

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,Hkv,d", [(2, 8, 128), (16, 8, 128), (64, 8, 128), (16, 5, 64), (128, 9, 64)])
def test_ranges_of_a_prompt_with_several_columns(B, Hkv, d, kv):
    rng = np.random.default_rng(63)
    tokens = 1500 + B // 2
    NB = -(-tokens // B)
    kc = _bf16(rng, NB, B, Hkv, d) if kv == "bf16" else _junk_cache(rng, kv, NB, B, Hkv, d)
    order = rng.permutation(NB)
    slots = order[np.arange(tokens) // B] * B + np.arange(tokens) % B
    slots[5 * B % tokens] = -1  # not a last slot (B > 1)
    codes, scales = ops.alloc_block_ranges(kc)
    ops.summarize_blocks(kc, _dev(slots), codes, scales)
    values = _np(kc) if kv == "bf16" else _codes_np(kc)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    full = set((slots[slots % B == B - 1] // B).tolist())
    for b in range(NB):
        if b not in full:
            assert (scales[b] == 0).all() and (codes[b] == 0).all()
        elif b % max(1, NB // 12) == 0:
            want, u = bs.block_range(values[b])
            assert np.array_equal(codes[b], want) and np.array_equal(scales[b], u)
        else:
            assert (scales[b] > 0).all()


# ------------------------------------------------------------ select_blocks

# 4, 2 and 1 warps to a row and KV head (by the number of those and the query heads)
UNITS = [(4, 50, 8), (8, 45, 8), (1, 50, 8), (4, 80, 8), (8, 80, 8), (1, 100, 8), (1, 160, 8), (2, 160, 8)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,rows,Hkv", UNITS)
@pytest.mark.parametrize("blocks", [150, 600])  # up to 256 candidates, and more
def test_select_for_many_rows(G, rows, Hkv, blocks, d):
    rng = np.random.default_rng(rows + G + blocks)
    # the oracle's time goes by the long rows
    lens = [(blocks - r % 11) * 16 - r % 16 if r % 16 == 0 else (20 + r % 9) * 16 - r % 16 for r in range(rows)]
    _check_select(rng, lens, G, Hkv, d, 16, 17, NB=211)


@pytest.mark.parametrize("G,rows,Hkv", [(4, 50, 8), (4, 80, 8), (1, 160, 8)])
@pytest.mark.parametrize("top", [3, 40, 580])
def test_select_for_many_rows_with_ties(G, rows, Hkv, top):
    rng = np.random.default_rng(64)
    c = rng.integers(0, 2, (97, Hkv, 2, 128)).astype(np.int8) * (rng.random((97, 1, 1, 1)) < 0.1)
    c[:, :, 1] = 0
    s = np.ones((97, Hkv), np.float32)
    lens = [600 * 16 if r % 25 == 0 else 300 for r in range(rows)]
    got = _check_select(rng, lens, G, Hkv, 128, 16, top, sink=1, recent=2, codes=(c.astype(np.int8), s), NB=97)
    assert (np.diff(got[0]) > 0).all()


def test_select_rows_of_long_contexts():
    # a batch of long contexts, several rows to each sequence
    rng = np.random.default_rng(65)
    tables = rng.integers(0, 300, (8, 2000)).astype(np.int32)
    row_seqs = np.repeat(np.arange(8), 4)
    lens = [32000 - 1000 * s + j if s % 4 == 0 else 400 + j for s in range(8) for j in range(4)]
    _check_select(rng, lens, 4, 8, 128, 16, 64, row_seqs=row_seqs, tables=tables, NB=300)


# ---------------------------------------------------------- decode_selected

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attention_of_a_batch(kv):
    rng = np.random.default_rng(66)
    lens = [600 - 5 * r for r in range(64)]
    out, args = _check_attend(rng, lens, _lists(rng, lens, 8, 16, 24), 4, 8, 128, 16, kv)
    for _ in range(3):  # the same call, the same bits
        again = torch.full_like(out, 5.0)
        ops.decode_selected(again, *args)
        assert torch.equal(again, out)


def test_calls_on_a_stream_given_by_object_and_by_handle():
    rng = np.random.default_rng(67)
    lens = [500, 77]
    out, args = _check_attend(rng, lens, _lists(rng, lens, 2, 16, 12), 4, 2, 64, 16, "bf16")
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        again = torch.full_like(out, 5.0)
        torch.cuda.synchronize()
        ops.decode_selected(again, *args, stream=stream)
        side.synchronize()
        assert torch.equal(again, out)


# ------------------------------------------------------------- the whole step

class _LongRow:
    """One row of a long context: few units, so that the selection runs in
    clusters of 8 CTAs and the attention in clusters of 8 or 12."""

    def __init__(self, kv, top, seed=70):
        rng = np.random.default_rng(seed)
        self.B, self.H, self.Hkv, self.d, self.top, self.kv = 16, 8, 2, 128, top, kv
        self.blocks, NB = 4000, 4001
        self.n = self.blocks * self.B - 3
        self.table = rng.permutation(NB)[None, :self.blocks].astype(np.int32)
        self.kc, self.vc = _bf16(rng, NB, self.B, self.Hkv, self.d), _bf16(rng, NB, self.B, self.Hkv, self.d)
        self.ks = self.vs = None
        if kv == "fp8":
            self.kc, self.vc = ((x.float() * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                                for x in (self.kc, self.vc))
            self.ks = self.vs = _dev([1 / 64], torch.float32)
        self.q = _bf16(rng, 1, self.H, self.d)
        self.codes, self.scales = ops.alloc_block_ranges(self.kc)
        self.slots = _dev(np.arange(NB) * self.B + self.B - 1)
        self.bt, self.cl = _dev(self.table), _dev([0])
        self.sel = torch.full((1, self.Hkv, top), 12345, device=DEV, dtype=torch.int32)
        self.out = torch.full_like(self.q, 9.0)

    def run(self):
        ops.summarize_blocks(self.kc, self.slots, self.codes, self.scales)
        ops.select_blocks(self.sel, self.q, self.codes, self.scales, self.bt, self.cl, self.B)
        ops.decode_selected(self.out, self.q, self.kc, self.vc, self.bt, self.cl, self.sel, self.d ** -0.5,
                            self.ks, self.vs)

    def check(self):
        torch.cuda.synchronize()
        codes, scales = self.codes.cpu().numpy(), self.scales.cpu().numpy().astype(np.float64)
        k, v = ((_np(x) if self.kv == "bf16" else _codes_np(x) / 64) for x in (self.kc, self.vc))
        sel, q = self.sel[0].cpu().numpy(), _np(self.q)[0]
        want = bs.select(q, codes, scales, self.table[0], self.n, self.B, self.top, 1, 1)
        assert np.array_equal(sel, want)
        want, mag = bs.decode_selected(q, k, v, self.table[0], self.n, sel, self.d ** -0.5)
        assert (np.abs(_np(self.out)[0] - want) <= 2 ** -8 * np.abs(want) + 2 ** -11 * mag).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("top", [130, 400])  # attention in clusters of 8, of 12
def test_clusters_captured_on_their_first_use(top, kv):
    # a fresh process whose first call of each kernel is captured
    code = f"""
import torch
from tests.test_gpu_block_sparse_paths import _LongRow
s = _LongRow({kv!r}, {top})
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s.run()
s.cl.fill_(s.n)
for _ in range(2):
    s.sel.fill_(12345)
    s.out.fill_(9.0)
    g.replay()
    s.check()
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert "captured first" in r.stdout, r.stderr[-2000:]


def test_two_host_threads_on_outputs_that_hold_nothing_yet():
    steps = [_Step("bf16", seed=71), _Step("fp8", seed=72)]
    for s in steps:
        s.stage()
        s.run()
    torch.cuda.synchronize()
    names = ("q", "sel", "out", "codes", "scales", "kc", "vc")
    want = [[getattr(s, x).clone() for x in names] for s in steps]
    failed = []

    def work(s, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(100):
                    s.q.fill_(7.0), s.sel.fill_(12345), s.out.fill_(9.0)
                    full = (s.slots % s.B == s.B - 1).nonzero().flatten()
                    s.codes[(s.slots[full] // s.B).long()] = 55
                    flat = s.kc.view(-1, s.Hkv, s.d)
                    flat.index_fill_(0, s.slots.long(), 0)
                    s.run()
                    torch.cuda.current_stream().synchronize()
                    for x, ref in zip(names, w):
                        a, b = getattr(s, x), ref
                        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), x
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(steps, want)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed, failed
    for s in steps:
        s.check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_ranges_of_blocks_that_were_swapped_in(kv):
    # blocks that come back from the host under other numbers get their ranges
    # from their last slots; a forked copy of a full block likewise
    rng = np.random.default_rng(73)
    NB, B, Hkv, d = 24, 16, 2, 64
    make = lambda *s: _bf16(rng, *s) if kv == "bf16" else _dev(rng.integers(0, 120, s), torch.uint8)  # noqa: E731
    kc, vc = make(NB, B, Hkv, d), make(NB, B, Hkv, d)
    codes, scales = ops.alloc_block_ranges(kc)
    ops.summarize_blocks(kc, _dev(np.arange(NB) * B + B - 1), codes, scales)
    pinned = lambda: torch.empty(6, B, Hkv, d, dtype=kc.dtype, pin_memory=True)  # noqa: E731
    ks, vs = pinned(), pinned()
    out = [3, 17, 8, 20]
    ops.swap_blocks(ks, vs, kc, vc, _dev([[b, i] for i, b in enumerate(out)]))
    to = [5, 3, 22, 8]  # other places, some of them just left
    ops.swap_blocks(kc, vc, ks, vs, _dev([[i, b] for i, b in enumerate(to)]))
    was = {b: (codes[a].clone(), scales[a].clone()) for a, b in zip(out, to)}
    ops.copy_blocks(kc, vc, _dev([[1, 11]]))
    was[11] = (codes[1].clone(), scales[1].clone())
    ops.summarize_blocks(kc, _dev([b * B + B - 1 for b in was]), codes, scales)
    torch.cuda.synchronize()
    for b, (c, s) in was.items():
        assert torch.equal(codes[b], c) and torch.equal(scales[b], s)


def test_selection_answers_as_the_whole_context_does():
    # one token answers the query; attention over the selection gives its
    # value, as attention over every block does
    rng = np.random.default_rng(74)
    S, H, Hkv, d, B, nb, top = 2, 4, 1, 64, 16, 120, 8
    tables = rng.permutation(S * nb).reshape(S, nb).astype(np.int32)
    k = rng.standard_normal((S * nb, B, Hkv, d)).astype(np.float32)
    q = _bf16(rng, S, 1, d).expand(S, H, d).contiguous()
    for i, j in enumerate((37, 101)):
        k[tables[i, j], 5, 0] = _np(q)[i, 0] * 4
    kc = torch.from_numpy(k).to(DEV).to(torch.bfloat16)
    vc = _bf16(rng, S * nb, B, Hkv, d)
    codes, scales = ops.alloc_block_ranges(kc)
    ops.summarize_blocks(kc, _dev(np.arange(S * nb) * B + B - 1), codes, scales)
    n = nb * B - 2
    sel, some, every = torch.empty(S, Hkv, top, device=DEV, dtype=torch.int32), torch.empty_like(q), torch.empty_like(q)
    ops.select_blocks(sel, q, codes, scales, _dev(tables), _dev([n] * S), B)
    ops.decode_selected(some, q, kc, vc, _dev(tables), _dev([n] * S), sel, d ** -0.5)
    ops.decode_selected(every, q, kc, vc, _dev(tables), _dev([n] * S),
                        _dev(np.broadcast_to(np.arange(nb), (S, Hkv, nb))), d ** -0.5)
    for i, j in enumerate((37, 101)):
        assert j in sel[i, 0].tolist()
        value = _np(vc)[tables[i, j], 5, 0]
        x = np.einsum("bthd,d->bth", _np(kc)[tables[i]], _np(q)[i, 0])[..., 0].reshape(-1)[:n] * d ** -0.5
        rest = 1 - 1 / np.exp(x - x[j * B + 5]).sum()  # what the other tokens weigh
        assert rest < 1e-4
        # every output is within the others' weight of the token's value
        far = rest * (np.abs(value) + np.abs(_np(vc)).max())
        bound = far + 2 ** -8 * (np.abs(value) + far) + 2 ** -11 * (np.abs(value) + far)
        for out in (some, every):
            assert (np.abs(_np(out)[i] - value) <= bound).all()
