"""The scored step's attention where its work split, its masks and its number
formats are at their edges: tiles whose parts are joined while other items
run, graphs that share a workspace, odd head counts, large blocks, alignment,
caps of any size, scales of any sign.  Tolerances as in the parity tests."""
import numpy as np
import pytest
import torch

from paged_kv_cache_108_gb300 import ops
from tests.test_gpu_scored import DEV, _attn_case, _bf16, _check_rows, _dev, _mod, _np

pytestmark = pytest.mark.gpu


def _step(c, new, seed=5, before=0, **kw):
    """Inputs of a varlen step over a case: `before` rows lie before the first
    request's."""
    starts = np.cumsum([before] + list(new))
    q = _bf16(np.random.default_rng(seed), int(starts[-1]), c["H"], c["d"], scale=c["scale_q"])
    return q, starts


def _varlen(c, q, starts, cap=0.0, window=0, bias=False, prefix=None, out=None, ws="own", **kw):
    out = torch.full_like(q, 7.0) if out is None else out
    if isinstance(ws, str):
        ws = ops.alloc_scored_workspace(q.shape[0], c["H"], c["Hkv"], c["d"]).random_(0, 256)
        ws[:4] = 0
    ops.varlen_scored(out, q, c["kc"], c["vc"], _dev(c["tables"]), _dev(c["lens"]), _dev(starts),
                      c["scale"], prefix_lens=None if prefix is None else _dev(prefix), workspace=ws,
                      **_mod(c, cap, window, bias), **kw)
    if ws is not None:
        assert int(ws[:4].view(torch.int32).item()) == 0
    return out


def _rows(c, starts, every=1):
    rows = []
    for i, n in enumerate(c["lens"]):
        t = int(starts[i + 1] - starts[i])
        mine = [(int(starts[i]) + j, i, n - t + j) for j in range(t)]
        rows += mine[::every] + mine[-1:]
    return rows


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (4, 4), (8, 1)])
def test_parts_are_joined_while_one_tile_still_works(kv, H, Hkv):
    """Items of one tile and of two by turns, all over long contexts, so that a
    CTA joins a split item's parts behind an item of its first tile alone."""
    mq = 128 // (H // Hkv)
    new = [2 * mq, mq // 2, 2 * mq, 3, mq + 1, mq, 2 * mq, 1]
    lens = [n + x for n, x in zip(new, [3000, 2500, 1700, 4100, 900, 3300, 600, 2900])]
    c = _attn_case(71, kv, lens, H, Hkv, 128, 16)
    q, starts = _step(c, new)
    outs = [_varlen(c, q, starts, cap=30.0) for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    _check_rows(c, outs[0], q, _rows(c, starts, 13), 30.0, 0, False, None, True)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv,B", [(3, 3, 16), (10, 5, 256), (8, 1, 1024), (28, 7, 64)])
def test_tiles_over_odd_heads_and_large_blocks(kv, H, Hkv, B):
    new, lens = [70, 1, 129], [1100, 513, 129]
    c = _attn_case(72, kv, lens, H, Hkv, 128, B)
    q, starts = _step(c, new)
    out = _varlen(c, q, starts, cap=20.0, window=600, bias=True)
    _check_rows(c, out, q, _rows(c, starts, 17), 20.0, 600, True, None, True)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_more_heads_than_sms(kv):
    H = Hkv = 320
    new, lens = [19, 3], [90, 40]
    c = _attn_case(73, kv, lens, H, Hkv, 128, 8)
    q, starts = _step(c, new)
    out = _varlen(c, q, starts, cap=30.0)
    _check_rows(c, out, q, _rows(c, starts, 9), 30.0, 0, False, None, kv != "int8")
    q1 = q[:2].contiguous()
    out = torch.empty_like(q1)
    ops.decode_scored(out, q1, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), c["scale"],
                      **_mod(c, 30.0, 0, False))
    _check_rows(c, out, q1, [(0, 0, 89), (1, 1, 39)], 30.0, 0, False)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-30, 3.0])
@pytest.mark.parametrize("cap", [0.0, 1.5, 50.0, 60.0])
def test_scales_and_caps_of_any_size(kv, scale, cap):
    """Logits far above their cap and far below it, of either sign."""
    new, lens = [40, 33], [300, 33]
    c = _attn_case(74, kv, lens, 8, 2, 128, 16)
    c["scale"] = scale
    q, starts = _step(c, new)
    out = _varlen(c, q, starts, cap=cap)
    _check_rows(c, out, q, _rows(c, starts, 8), cap, 0, False, None, kv != "int8")
    last = q[[39, 72]].contiguous()
    out = torch.empty_like(last)
    ops.decode_scored(out, last, c["kc"], c["vc"], _dev(c["tables"]), _dev(lens), scale,
                      **_mod(c, cap, 0, False))
    _check_rows(c, out, last, [(0, 0, 299), (1, 1, 32)], cap, 0, False)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_tiles_rescale_rows_that_grow(kv):
    """Keys whose logits grow towards the first of a context, which the tiles
    visit last: the running max rises in every chunk, in some rows alone."""
    c = _attn_case(75, kv, [1500], 4, 2, 128, 16, scale_q=1.0)
    t = c["tables"][0]
    ramp = _dev(np.linspace(12.0, 0.1, 1500), torch.float32)
    for j in range(1500):
        b, o = int(t[j // 16]), j % 16
        row = c["kc"][b, o]
        if kv == "bf16":
            c["kc"][b, o] = row * ramp[j]
        else:
            x = row.view(torch.float8_e4m3fn).float() * ramp[j] / 12
            c["kc"][b, o] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    if kv == "fp8":
        c["ks"] *= 12
    q, starts = _step(c, [150])
    q[::3] *= 8.0
    out = _varlen(c, q, starts)
    _check_rows(c, out, q, _rows(c, starts, 7), 0.0, 0, False, None, True)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_pointers_aligned_to_16_bytes_only(kv):
    new, lens = [30, 25], [200, 25]
    c = _attn_case(76, kv, lens, 8, 2, 128, 16)
    q0, starts = _step(c, new)
    q = torch.empty(q0.numel() + 8, dtype=q0.dtype, device=DEV)[8:].view(q0.shape)
    q.copy_(q0)
    room = torch.full((q0.numel() + 8,), 7.0, dtype=q0.dtype, device=DEV)
    out = _varlen(c, q, starts, cap=30.0, out=room[8:].view(q0.shape))
    assert out.data_ptr() % 32 == 16
    assert torch.equal(out, _varlen(c, q0, starts, cap=30.0))
    assert (room[:8] == 7.0).all()


def test_many_requests_take_rows_and_a_batch_may_start_late():
    rng = np.random.default_rng(77)
    new = [int(x) for x in rng.integers(0, 9, 300)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 60, 300))]
    c = _attn_case(77, "bf16", lens, 4, 2, 128, 16)
    q, starts = _step(c, new, before=5)
    out = _varlen(c, q, starts, cap=30.0, window=20)
    assert (out[:5] == 7.0).all()
    _check_rows(c, out, q, _rows(c, starts, 4)[::5], 30.0, 20, False)
    # the same in the tiles: few requests
    few = dict(c, tables=c["tables"][:100], lens=lens[:100])
    out = _varlen(few, q[:int(starts[100])].contiguous(), starts[:101], cap=30.0, window=20)
    assert (out[:5] == 7.0).all()
    _check_rows(few, out, q, [r for r in _rows(few, starts, 4)[::3] if new[r[1]]], 30.0, 20, False, None,
                True)


def test_a_window_of_one_and_prefixes_that_cover_all():
    c = _attn_case(78, "bf16", [90, 200], 4, 1, 128, 16)
    q, starts = _step(c, [90, 64])
    out = _varlen(c, q, starts, window=1)
    _check_rows(c, out, q, _rows(c, starts, 5), 0.0, 1, False, None, True)
    out = _varlen(c, q, starts, window=1, prefix=[90, 200])
    _check_rows(c, out, q, _rows(c, starts, 5), 0.0, 1, False, [90, 200], True)


def test_capped_values_of_the_documented_range():
    """A cap without a running max, logits at the cap: values up to 2^30."""
    c = _attn_case(79, "bf16", [400], 4, 2, 128, 16, scale_q=30.0)
    c["vc"].copy_(c["vc"].float() * 2.0 ** _dev(c["rng"].uniform(-40, 27, tuple(c["vc"].shape[:3])),
                                               torch.float32)[..., None])
    q, starts = _step(c, [140])
    for cap in (50.0, 55.0):
        out = _varlen(c, q, starts, cap=cap)
        assert torch.isfinite(out).all()
        _check_rows(c, out, q, _rows(c, starts, 9), cap, 0, False, None, True)


def test_replayed_prompts_share_a_workspace():
    """Two captured steps of tiles and one of rows in one workspace, with eager
    calls of other sizes between their replays."""
    cs = [_attn_case(80, "bf16", [2600, 700], 8, 2, 128, 16),
          _attn_case(81, "fp8", [900, 1800, 60], 8, 2, 128, 16),
          _attn_case(82, "int8", [800, 500], 8, 2, 128, 16)]
    news = [[64, 70], [40, 33, 60], [3, 2]]
    ws = ops.alloc_scored_workspace(134, 8, 2, 128)
    steps = []
    for c, new in zip(cs, news):
        q, starts = _step(c, new)
        steps.append(dict(q=q, out=torch.zeros_like(q), starts=starts, args=(
            c["kc"], c["vc"], _dev(c["tables"]), _dev(c["lens"]), _dev(starts), c["scale"]),
            mod=_mod(c, 30.0, 0, False)))

    def run(s):
        ops.varlen_scored(s["out"], s["q"], *s["args"], workspace=ws, **s["mod"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in steps:
            run(s)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in steps]
    for g, s in zip(graphs, steps):
        with torch.cuda.graph(g):
            run(s)
    for turn in range(3):
        for i, s in enumerate(steps):
            s["q"].copy_(_bf16(cs[i]["rng"], *s["q"].shape, scale=2.0))
            graphs[i].replay()
            run(steps[(i + 1) % 3])
            graphs[i].replay()
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    for c, s in zip(cs, steps):
        _check_rows(c, s["out"], s["q"], _rows(c, s["starts"], 11), 30.0, 0, False, None,
                    c["kv"] != "int8")


def test_prompts_on_another_stream_without_a_workspace():
    c = _attn_case(83, "bf16", [900, 64], 8, 2, 128, 16)
    q, starts = _step(c, [90, 64])
    want = _varlen(c, q, starts, cap=50.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.zeros_like(q) for _ in range(3)]
    torch.cuda.synchronize()
    for out in outs:
        _varlen(c, q, starts, cap=50.0, out=out, ws=None, stream=side)
    side.synchronize()
    for out in outs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_contexts_of_tens_of_thousands(kv):
    """One long context split over every CTA, in prompts and single tokens."""
    n = 40_003
    c = _attn_case(84, kv, [n], 2, 1, 128, 64)
    new = 5 if kv == "int8" else 40
    q, starts = _step(c, [new])
    out = _varlen(c, q, starts, cap=40.0, bias=True)
    _check_rows(c, out, q, [(r, 0, n - new + r) for r in {0, new // 2, new - 1}], 40.0, 0, True, None,
                kv != "int8")
    last = q[-1:].contiguous()
    out = torch.empty_like(last)
    ops.decode_scored(out, last, c["kc"], c["vc"], _dev(c["tables"]), _dev([n]), c["scale"],
                      **_mod(c, 40.0, 0, True))
    _check_rows(c, out, last, [(0, 0, n - 1)], 40.0, 0, True)


def test_infinite_and_nan_queries_stay_in_their_rows():
    for kv in ("bf16", "fp8", "int8"):
        c = _attn_case(85, kv, [200, 77], 8, 2, 128, 16)
        q, starts = _step(c, [40, 30])
        clean = _np(_varlen(c, q, starts, cap=30.0))
        q[3, 2, 5] = float("nan")
        q[50, 7, 1] = float("inf")
        got = _np(_varlen(c, q, starts, cap=30.0))
        assert np.isnan(got[3, 2]).all()
        same = np.ones(got.shape[:2], bool)
        same[3, 2] = same[50, 7] = False
        assert np.isfinite(got[same]).all()
        # (a warp whose rows hold a NaN or an infinity caps by the other formula)
        assert np.abs(got - clean)[same].max() <= 2 ** -6 * np.abs(clean).max()


def test_blocks_of_8_bit_rows_are_copied_as_bytes():
    """A fork's copied blocks: codes and units through copy_blocks."""
    c = _attn_case(86, "int8", [130, 40], 8, 2, 64, 16)
    kc, vc, ks, vs = (torch.cat([t, torch.zeros_like(t)]) for t in (c["kc"], c["vc"], c["ks"], c["vs"]))
    NB = c["kc"].shape[0]
    pairs = _dev(np.stack([np.arange(NB), NB + np.random.default_rng(1).permutation(NB)], 1))
    ops.copy_blocks(kc.view(torch.uint8), vc.view(torch.uint8), pairs)
    units = [t.view(torch.bfloat16).view(2 * NB, 1, -1, 64) for t in (ks, vs)]
    ops.copy_blocks(*units, pairs)
    to = pairs[:, 1].cpu().numpy()
    q = _bf16(c["rng"], 2, 8, 64)
    outs = []
    for tables in (c["tables"], np.where(c["tables"] < 0, -1, to[c["tables"]])):
        out = torch.empty_like(q)
        ops.decode_scored(out, q, kc, vc, _dev(tables), _dev(c["lens"]), c["scale"], cap=30.0,
                          k_scale=ks, v_scale=vs)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    _check_rows(c, outs[0], q, [(0, 0, 129), (1, 1, 39)], 30.0, 0, False)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv,new,n,window,prefix", [
    (2, 2, 256, 1000, 150, 0), (2, 2, 250, 900, 40, 0), (3, 3, 256, 2000, 129, 1700),
    (1, 1, 129, 1500, 300, 0), (4, 4, 200, 1400, 500, 1390), (8, 2, 64, 1300, 20, 0),
])
def test_parts_in_which_a_tile_has_no_keys(kv, H, Hkv, new, n, window, prefix):
    """Few items over windows, each shared by CTAs: some parts hold keys of one
    of the two tiles alone, the joining CTA's own among them."""
    c = _attn_case(87, kv, [n], H, Hkv, 128, 16)
    q, starts = _step(c, [new])
    pre = [prefix] if prefix else None
    outs = [_varlen(c, q, starts, cap=cap, window=window, prefix=pre) for cap in (0.0, 25.0, 25.0)]
    assert torch.equal(outs[1], outs[2])
    _check_rows(c, outs[0], q, _rows(c, starts, 19), 0.0, window, False, pre, True)
    _check_rows(c, outs[1], q, _rows(c, starts, 19), 25.0, window, False, pre, True)


def test_calls_on_two_streams_at_once():
    """Prompts and single tokens on two streams, a workspace each: split work of
    both at the same time."""
    cs = [_attn_case(88, "bf16", [3000, 700], 8, 2, 128, 16),
          _attn_case(89, "fp8", [2500, 1800, 60], 8, 2, 128, 16)]
    jobs = []
    for c, new in zip(cs, ([200, 70], [90, 33, 60])):
        q, starts = _step(c, new)
        last = q[[int(s) - 1 for s in starts[1:]]].contiguous()
        jobs.append(dict(q=q, last=last, starts=_dev(starts), tables=_dev(c["tables"]),
                         lens=_dev(c["lens"]), mod=_mod(c, 30.0, 0, False), side=torch.cuda.Stream(),
                         ws=ops.alloc_scored_workspace(q.shape[0], 8, 2, 128),
                         want=_varlen(c, q, starts, cap=30.0), outs=[], c=c, host=starts))
    torch.cuda.synchronize()
    for _ in range(12):
        for j in jobs:
            with torch.cuda.stream(j["side"]):
                out, one = torch.empty_like(j["q"]), torch.empty_like(j["last"])
            args = (j["c"]["kc"], j["c"]["vc"], j["tables"], j["lens"])
            ops.varlen_scored(out, j["q"], *args, j["starts"], j["c"]["scale"], workspace=j["ws"],
                              stream=j["side"], **j["mod"])
            ops.decode_scored(one, j["last"], *args, j["c"]["scale"], workspace=j["ws"],
                              stream=j["side"], **j["mod"])
            j["outs"].append((out, one))
    torch.cuda.synchronize()
    for j in jobs:
        for out, one in j["outs"]:
            assert torch.equal(out, j["want"]) and torch.equal(one, j["outs"][0][1])
        _check_rows(j["c"], j["outs"][0][1], j["last"],
                    [(i, i, n - 1) for i, n in enumerate(j["c"]["lens"])], 30.0, 0, False)
        _check_rows(j["c"], j["want"], j["q"], _rows(j["c"], j["host"], 23), 30.0, 0, False, None, True)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("cap,bias", [(30.0, False), (60.0, False), (30.0, True)])
def test_unseen_keys_leave_no_trace(kv, cap, bias):
    """Bit for bit: whatever lies behind the contexts and before the windows,
    and whatever ran before (other calls' keys in the SMs' memory)."""
    new, lens = [200, 70], [3003, 717]
    c = _attn_case(90, kv, lens, 8, 2, 128, 16)
    q, starts = _step(c, new)
    loud = _attn_case(91, kv, [900, 900], 8, 2, 128, 16)
    lq, lstarts = _step(loud, [300, 300])
    lq *= 50.0
    outs = []
    for turn in range(6):
        if turn % 2:
            _varlen(loud, lq, lstarts)
        for i, n in enumerate(lens):  # behind the last token
            for cache in (c["kc"], c["vc"]):
                tail = cache[int(c["tables"][i, n // 16]), n % 16:]
                tail.copy_((torch.randn(tail.shape, device=DEV) * 10.0 ** turn).to(tail.dtype)
                           if kv == "bf16" else torch.randint_like(tail, 0, 127))
        outs.append(_varlen(c, q, starts, cap=cap, bias=bias, window=1000))
    for out in outs[1:]:
        assert torch.equal(out, outs[0])
    _check_rows(c, outs[0], q, _rows(c, starts, 17), cap, 1000, bias, None, True)
