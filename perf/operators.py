"""Cases, inputs and plain forms of the block-sparse serving step's operators.

The step: the new tokens' queries and keys are rotated by position and the
keys and values appended to the paged cache (``rope``); blocks that became
full get their keys' range per channel, in 8 bits (``summarize``); each query
chooses the blocks whose range allows the largest logit (``select``) and
attends to those alone (``attend``).

``run`` computes an operator in its plain form (elementary torch operations,
32 bits, one rounding at the end), or, where ``own`` is true, by the
framework's own calls.  ``exact`` gives the result in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
MAX_POSITION = 131072  # rows of the cosine and sine table
ROPE_BASE = 500000.0


def listed():
    """Twelve cases.  The heads are the repository's own: 32 query and 8 KV
    heads of 128 channels (its headline layer), 32 / 32 (its serving mix),
    4 / 2 of 64 channels (its tiny case); 16 tokens a block unless said."""
    return [
        # one user's single new token: latency alone
        rope("rope-step-1", 1, 32, 8, 128, 128, 1, False, False, "bf16", 16),
        # the decode step of a batch of 64, cache in e4m3
        rope("rope-step-64-fp8", 64, 32, 8, 128, 128, 1, False, False, "fp8", 16),
        # a prompt with images: three position axes, sections in a row
        rope("rope-prefill-8192-axes", 8192, 32, 8, 128, 128, 3, False, False, "bf16", 16),
        # a ragged chunk, half the channels rotated in neighbouring pairs,
        # axes taken in turn, large blocks
        rope("rope-chunk-1021-pairs", 1021, 4, 2, 64, 32, 3, True, True, "fp8", 64),
        # the decode step of a batch of 64, cache in e4m3: four blocks became full
        summarize("summarize-step-64-fp8", 64, 1, 8, 128, 16, "fp8"),
        # four long prompts, or a swapped-in batch
        summarize("summarize-prompts-32k", 4, 8190, 8, 128, 16, "bf16"),
        # one user's long context: 8 K blocks to choose from
        select("select-1-128k", 1, 1, 32, 8, 128, 16, 131071, 256),
        # the decode step of a batch of 64
        select("select-64", 64, 1, 32, 8, 128, 16, 2977, 64),
        # MHA, large batch: every head has its own blocks
        select("select-256-mha", 256, 1, 32, 32, 128, 16, 2900, 64),
        # one user's token
        attend("attend-1", 1, 1, 32, 8, 128, 16, 32765, 64, "bf16"),
        # the decode step of a batch of 64, 1024 tokens for each head
        attend("attend-64", 64, 1, 32, 8, 128, 16, 2977, 64, "bf16"),
        # long contexts, 8192 tokens for each head, e4m3
        attend("attend-8-long-fp8", 8, 1, 32, 8, 128, 16, 65531, 512, "fp8"),
    ]


def rope(name, tokens, heads, kv_heads, dim, rot, axes, pairs, turn, kv, block):
    return dict(name=name, op="rope", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                rot=rot, axes=axes, pairs=pairs, turn=turn, kv=kv, block=block)


def summarize(name, seqs, new, kv_heads, dim, block, kv):
    return dict(name=name, op="summarize", seqs=seqs, new=new, kv_heads=kv_heads, dim=dim,
                block=block, kv=kv)


def select(name, seqs, per_seq, heads, kv_heads, dim, block, context, top):
    return dict(name=name, op="select", seqs=seqs, per_seq=per_seq, heads=heads,
                kv_heads=kv_heads, dim=dim, block=block, context=context, top=top)


def attend(name, seqs, per_seq, heads, kv_heads, dim, block, context, top, kv):
    return dict(name=name, op="attend", seqs=seqs, per_seq=per_seq, heads=heads,
                kv_heads=kv_heads, dim=dim, block=block, context=context, top=top, kv=kv)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "summarize", "select", "attend"])
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (32, 32, 128), (4, 2, 64), (8, 1, 128),
                                       (16, 2, 64), (8, 4, 128)])
    block = rng.choice([8, 16, 16, 32, 64, 128])
    kv = rng.choice(["bf16", "fp8"])
    if op == "rope":
        tokens = _log(rng, 1, 8192 if kv_heads < 32 else 4096)
        return {k: v for k, v in rope("", tokens, heads, kv_heads, dim, rng.choice([dim, dim // 2]),
                                      rng.choice([1, 1, 3]), rng.random() < 0.4,
                                      rng.random() < 0.5, kv, block).items() if k != "name"}
    if op == "summarize":
        new = rng.choice([1, _log(rng, 2, 8000)])
        seqs = _log(rng, 1, 256) if new == 1 else rng.randint(1, 4)
        if kv_heads == 32:
            new = min(new, 2000)
        return {k: v for k, v in summarize("", seqs, new, kv_heads, dim, block, kv).items()
                if k != "name"}
    per_seq = rng.choice([1, 1, 1, 4])
    seqs = _log(rng, 1, 64 if per_seq == 1 else 16)
    context = _log(rng, 1, 131072 // max(seqs, 2))
    if kv_heads == 32:
        context = max(1, context // 4)
    top = _log(rng, 4, 256)
    if op == "select":
        return {k: v for k, v in select("", seqs, per_seq, heads, kv_heads, dim, block, context,
                                        top).items() if k != "name"}
    top = max(4, min(top, 8192 // block))
    while seqs * per_seq * kv_heads * min(context, top * block) > 64 * 8 * 1024:
        if top >= 8:
            top //= 2
        else:
            context = max(1, context // 2)
    return {k: v for k, v in attend("", seqs, per_seq, heads, kv_heads, dim, block, context, top,
                                    kv).items() if k != "name"}


# ------------------------------------------------------------------- sizes

def _lens(case):
    """Context length of each query row: rows of one sequence end one token
    after another; the sequences' lengths fall from `context` to half of it."""
    n, t = case["seqs"], case["per_seq"]
    last = [max(1, case["context"] - (case["context"] // 2) * i // n) for i in range(n)]
    return [max(1, m - (t - 1) + j) for m in last for j in range(t)]


def _blocks(case):
    return -(-case["context"] // case["block"])


def _completed(case):
    """Blocks that the step's tokens fill: a chunk starts with a block; of
    single tokens one in `block`, and at least one, is its block's last."""
    if case["new"] == 1:
        return max(1, case["seqs"] // case["block"])
    return case["seqs"] * (case["new"] // case["block"])


def work(case):
    op, d, hk = case["op"], case["dim"], case["kv_heads"]
    b = 1 if case.get("kv") == "fp8" else 2
    if op == "rope":
        n, h = case["tokens"], case["heads"]
        read = n * ((h + 2 * hk) * d * 2 + case["rot"] * 4 + case["axes"] * 4 + 4)
        return {"bytes": read + n * (h * d * 2 + 2 * hk * d * b),
                "flops": n * (h + hk) * case["rot"] * 3}
    if op == "summarize":
        f = _completed(case)
        return {"bytes": f * hk * (case["block"] * d * b + 2 * d + 4) + case["seqs"] * case["new"] * 4,
                "flops": f * hk * case["block"] * d * 2}
    rows, h, top, bs = len(_lens(case)), case["heads"], case["top"], case["block"]
    nb = [-(-n // bs) for n in _lens(case)]
    if op == "select":
        # a sequence's ranges are read once, whatever the number of its queries
        t = case["per_seq"]
        scored = [max(nb[i:i + t]) if max(nb[i:i + t]) > top else 0 for i in range(0, rows, t)]
        return {"bytes": sum(scored) * (hk * (2 * d + 4) + 4) + rows * (h * d * 2 + hk * top * 4 + 4),
                "flops": sum(x if x > top else 0 for x in nb) * h * d * 4}
    tokens = [min(n, min(top, m) * bs) for n, m in zip(_lens(case), nb)]
    return {"bytes": sum(tokens) * hk * d * 2 * b + rows * (2 * h * d * 2 + hk * top * 4 + 4)
            + sum(min(top, m) for m in nb) * 4,
            "flops": sum(tokens) * h * d * 4}


# ------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _cache(g, kv, *shape):
    """Keys or values that a serving loop has cached: N(0, 1) in bf16, or the
    e4m3 codes of such under a scale that puts amax near the type's largest."""
    x = _normal(g, *shape)
    if kv == "bf16":
        return x, None
    s = torch.full((1,), 5.0 / 448.0, device=DEV, dtype=torch.float32)
    return (x.float() / s).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _axis_of_pair(case):
    """Which position axis turns pair i, and the sections' sizes."""
    p, a = case["rot"] // 2, case["axes"]
    if a == 1:
        return [0] * p, [p]
    other = 3 * p // 8 if not case["turn"] else p // 3
    sections = [p - 2 * other, other, other]
    if not case["turn"]:
        return [x for x, n in enumerate(sections) for _ in range(n)], sections
    return [i % 3 if i % 3 and i < 3 * sections[i % 3] else 0 for i in range(p)], sections


_tables = {}


def _table(rot):
    """Cosines, then sines, of every position's angles: a model's constant,
    computed in 64 bits and kept for the process's life."""
    if rot not in _tables:
        inv = ROPE_BASE ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(MAX_POSITION, device=DEV, dtype=torch.float64)[:, None] * inv
        _tables[rot] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    return _tables[rot]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    d, hk, bs = case["dim"], case["kv_heads"], case["block"]
    s = {"case": case}

    def dev(x, dtype=torch.int32):
        return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).to(DEV)

    if case["op"] == "rope":
        n, h, p = case["tokens"], case["heads"], case["rot"] // 2
        # one projection's result; queries, keys and values are views of it
        qkv = _normal(g, n, (h + 2 * hk) * d)
        s["q"] = qkv[:, :h * d].view(n, h, d)
        s["k"] = qkv[:, h * d:(h + hk) * d].view(n, hk, d)
        s["v"] = qkv[:, (h + hk) * d:].view(n, hk, d)
        step = n <= 256  # a decode step (each token in a block of its own), else a prompt
        nb = n + 2 if step else -(-n // bs) + 2
        blocks = rng.permutation(nb)[:nb - 2]
        slots = blocks * bs + rng.integers(0, bs, n) if step else blocks[np.arange(n) // bs] * bs + np.arange(n) % bs
        if n >= 32:
            slots[-3:] = -1  # the batch's padding
        s["slots"] = dev(slots)
        first = rng.integers(0, MAX_POSITION - n)
        pos = rng.integers(0, MAX_POSITION, n) if step else first + np.arange(n)
        if case["axes"] == 1:
            s["pos"] = dev(pos)
        else:  # time, height, width of a patch
            s["pos"] = dev(np.stack([pos, pos - rng.integers(0, 64, n), pos - rng.integers(0, 64, n)]).clip(0))
        s["table"] = _table(case["rot"])
        axis, s["sections"] = _axis_of_pair(case)
        s["axis"] = dev(axis, torch.long)
        s["kc"], s["ks"] = _cache(g, case["kv"], nb, bs, hk, d)
        s["vc"], s["vs"] = _cache(g, case["kv"], nb, bs, hk, d)
        s["out"] = torch.empty(n, h, d, device=DEV, dtype=torch.bfloat16)
        return s
    if case["op"] == "summarize":
        n, new = case["seqs"], case["new"]
        if new == 1:
            nb = n + 2
            off = rng.integers(0, max(1, bs - 1), n)
            off[rng.permutation(n)[:_completed(case)]] = bs - 1
            slots = rng.permutation(nb)[:n] * bs + off
        else:
            per = -(-new // bs)
            nb = n * per + 2
            blocks = rng.permutation(nb)[:n * per].reshape(n, per)
            slots = (blocks[:, np.arange(new) // bs] * bs + np.arange(new) % bs).reshape(-1)
        s["slots"] = dev(slots)
        # keys of a layer: channels differ in mean and width
        width = 0.25 + torch.rand(hk, d, generator=g, device=DEV) * 2
        mean = torch.randn(hk, d, generator=g, device=DEV)
        k = torch.randn(nb, bs, hk, d, generator=g, device=DEV) * width + mean
        s["kc"] = k.to(torch.bfloat16) if case["kv"] == "bf16" else (k * 20).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["codes"] = torch.zeros(nb, hk, 2, d, device=DEV, dtype=torch.int8)
        s["scales"] = torch.zeros(nb, hk, device=DEV, dtype=torch.float32)
        return s
    seqs, per = case["seqs"], case["per_seq"]
    lens = _lens(case)
    rows, width = len(lens), _blocks(case)
    need = [-(-max(lens[i * per:(i + 1) * per]) // bs) for i in range(seqs)]
    nb = sum(need) + 2
    order, tables, at = rng.permutation(nb), np.zeros((seqs, width), np.int32), 0
    for i, m in enumerate(need):
        tables[i, :m] = order[at:at + m]
        at += m
    s["tables"], s["lens"] = dev(tables), dev(lens)
    s["row_seqs"] = None if per == 1 else dev(np.repeat(np.arange(seqs), per))
    s["q"] = _normal(g, rows, case["heads"], d)
    top = case["top"]
    if case["op"] == "select":
        # ranges as a layer's keys give them: a middle and a half-width per
        # block and channel, rounded outward to multiples of a power of two
        mid = torch.randn(nb, hk, d, generator=g, device=DEV) * 0.5 + torch.randn(hk, d, generator=g, device=DEV)
        half = 1.2 + torch.rand(nb, hk, d, generator=g, device=DEV)
        hi, lo = mid + half, mid - half
        amax = torch.maximum(hi.abs(), lo.abs()).amax(-1)
        s["scales"] = torch.exp2(torch.ceil(torch.log2(amax / 126.0)))
        s["codes"] = torch.stack([torch.ceil(hi / s["scales"][..., None]), torch.floor(lo / s["scales"][..., None])], 2).to(torch.int8)
        s["selected"] = torch.empty(rows, hk, top, device=DEV, dtype=torch.int32)
        return s
    # what a selection hands over: the first and the last block and, in
    # rising order, others between them; -1 behind the last entry
    u = torch.rand(rows, hk, width, generator=g, device=DEV)
    j = torch.arange(width, device=DEV)
    have = ((s["lens"] + bs - 1) // bs).long()
    u = torch.where((j == 0) | (j == (have - 1)[:, None, None]), 2.0, u)
    u = torch.where(j < have[:, None, None], u, -1.0)
    k = min(top, width)
    val, idx = torch.topk(u, k, dim=-1)
    idx = torch.where(val < 0, width, idx).sort(-1).values
    sel = torch.full((rows, hk, top), -1, device=DEV, dtype=torch.int32)
    sel[..., :k] = torch.where(idx == width, -1, idx).int()
    s["selected"] = sel
    s["kc"], s["ks"] = _cache(g, case["kv"], nb, bs, hk, d)
    s["vc"], s["vs"] = _cache(g, case["kv"], nb, bs, hk, d)
    s["scale"] = d ** -0.5
    s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        from paged_kv_cache_108_gb300 import ops
        if op == "rope":
            ops.rope_and_cache(s["out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"],
                               s["pos"], s["table"], s["ks"], s["vs"], sections=s["sections"],
                               sections_in_turn=s["case"]["turn"], adjacent_pairs=s["case"]["pairs"])
            return s["out"], s["kc"], s["vc"]
        if op == "summarize":
            ops.summarize_blocks(s["kc"], s["slots"], s["codes"], s["scales"])
            return s["codes"], s["scales"]
        if op == "select":
            ops.select_blocks(s["selected"], s["q"], s["codes"], s["scales"], s["tables"],
                              s["lens"], s["case"]["block"], row_seqs=s["row_seqs"])
            return s["selected"]
        ops.decode_selected(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"],
                            s["selected"], s["scale"], s["ks"], s["vs"], row_seqs=s["row_seqs"])
        return s["out"]
    return {"rope": _rope, "summarize": _summarize, "select": _select, "attend": _attend}[op](s)


def _rotated(x, cos, sin, pairs):
    p = cos.shape[-1]
    x = x.float()
    a, b = (x[..., 0:2 * p:2], x[..., 1:2 * p:2]) if pairs else (x[..., :p], x[..., p:2 * p])
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if pairs else -2).flatten(-2)
    return torch.cat([y, x[..., 2 * p:]], -1)


def _rope(s):
    pos, table, p = s["pos"].long(), s["table"], s["case"]["rot"] // 2
    at = pos[s["axis"]].T if pos.dim() == 2 else pos[:, None]  # [tokens, pairs or 1]
    pair = torch.arange(p, device=DEV)
    cos, sin = table[at, pair][:, None], table[at, pair + p][:, None]
    q = _rotated(s["q"], cos, sin, s["case"]["pairs"]).to(torch.bfloat16)
    k, v = _rotated(s["k"], cos, sin, s["case"]["pairs"]), s["v"].float()
    there = s["slots"] >= 0
    to = s["slots"][there].long()
    for cache, x, scale in ((s["kc"], k, s["ks"]), (s["vc"], v, s["vs"])):
        flat = cache.view(-1, *cache.shape[2:])
        if scale is None:
            flat[to] = x[there].to(torch.bfloat16)
        else:
            codes = (x[there] / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            flat.view(torch.uint8)[to] = codes.view(torch.uint8)
    return q, s["kc"], s["vc"]


def _power_above(amax):
    """The smallest power of two u >= 2^-50 with amax / u <= 127."""
    m, e = torch.frexp(amax / 127.0)
    e = torch.where(m == 0.5, e - 1, e)  # amax / 127 is a power of two itself
    e = torch.where(amax > 127.0 * torch.exp2((e).float()), e + 1, e)
    return torch.exp2(torch.where(amax > 0, e, -50).clamp(min=-50).float())


def _summarize(s):
    bs = s["case"]["block"]
    blocks = s["slots"][s["slots"] % bs == bs - 1].long() // bs
    k = s["kc"][blocks] if s["kc"].dtype == torch.bfloat16 else s["kc"].view(torch.uint8)[blocks].view(torch.float8_e4m3fn)
    k = k.float().clamp(-2.0 ** 50, 2.0 ** 50)
    hi, lo = k.amax(1), k.amin(1)
    u = _power_above(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    s["codes"][blocks] = torch.stack([torch.ceil(hi / u[..., None]), torch.floor(lo / u[..., None])], 2).to(torch.int8)
    s["scales"][blocks] = u
    return s["codes"], s["scales"]


def _select(s):
    case, top = s["case"], s["case"]["top"]
    bs, hk, d = case["block"], case["kv_heads"], case["dim"]
    q = s["q"].float()
    rows = q.shape[0]
    u = _power_above(q.abs().amax(-1, keepdim=True))
    c = torch.round(q / u).view(rows, hk, -1, d)
    tables = s["tables"].long() if s["row_seqs"] is None else s["tables"][s["row_seqs"].long()].long()
    f, us = s["codes"][tables].float(), s["scales"][tables]  # [rows, blocks, hk, 2, d]
    # whole numbers below 2^24 times powers of two: 32 bits hold them exactly
    dot = (torch.einsum("rhgd,rbhd->rhgb", c.clamp(min=0), f[..., 0, :])
           + torch.einsum("rhgd,rbhd->rhgb", c.clamp(max=0), f[..., 1, :]))
    score = (dot * u.view(rows, hk, -1, 1)).amax(2) * us.transpose(1, 2)
    j = torch.arange(tables.shape[1], device=DEV)
    have = ((s["lens"] + bs - 1) // bs)[:, None, None]
    score = torch.where((j < 1) | (j >= have - 1), math.inf, score)
    score = torch.where(j < have, score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    order = torch.where(order < have, order, tables.shape[1]).sort(-1).values
    out = torch.full((rows, hk, top), -1, device=DEV, dtype=torch.int32)
    out[..., :order.shape[-1]] = torch.where(order < have, order, -1).int()
    return out


def _attend(s):
    case, sel = s["case"], s["selected"].long()
    bs, hk, d = case["block"], case["kv_heads"], case["dim"]
    rows = sel.shape[0]
    tables = s["tables"].long() if s["row_seqs"] is None else s["tables"][s["row_seqs"].long()].long()
    block = tables[torch.arange(rows, device=DEV)[:, None, None], sel.clamp(min=0)][..., None]
    off, head = torch.arange(bs, device=DEV), torch.arange(hk, device=DEV)[:, None, None]
    there = ((sel >= 0)[..., None] & (sel[..., None] * bs + off < s["lens"][:, None, None, None])).flatten(2)

    def rows_of(cache, scale):
        if scale is None:
            return cache[block, off, head].float().flatten(2, 3)
        return cache.view(torch.uint8)[block, off, head].view(torch.float8_e4m3fn).float().flatten(2, 3) * scale

    q = s["q"].float().view(rows, hk, -1, d)
    logit = torch.matmul(q, rows_of(s["kc"], s["ks"]).transpose(2, 3)) * s["scale"]
    logit = torch.where(there[:, :, None], logit, -math.inf)
    p = torch.exp(logit - logit.amax(-1, keepdim=True))
    out = torch.matmul(p, rows_of(s["vc"], s["vs"])) / p.sum(-1, keepdim=True)
    return out.view(rows, -1, d).to(torch.bfloat16)


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope64, "summarize": _summarize64, "select": _select64,
            "attend": _attend64}[case["op"]](s, case)


def _f64(x):
    return x.to(torch.float32).double().cpu().numpy()


def _rope64(s, case):
    n, p = case["tokens"], case["rot"] // 2
    pos = s["pos"].cpu().numpy().reshape(-1, n)
    table = s["table"][torch.as_tensor(pos.reshape(-1), device=DEV).long()].double().cpu().numpy().reshape(-1, n, 2 * p)
    axis = s["axis"].cpu().numpy()
    # each pair as a complex number, turned by e^(i angle)
    turn = np.stack([table[axis[i] if len(pos) > 1 else 0, :, i] + 1j * table[axis[i] if len(pos) > 1 else 0, :, p + i] for i in range(p)], -1)
    first = np.arange(p) * 2 if case["pairs"] else np.arange(p)
    second = first + 1 if case["pairs"] else first + p

    def turned(x):
        z = (x[..., first] + 1j * x[..., second]) * turn[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k, v = turned(_f64(s["q"])), turned(_f64(s["k"])), _f64(s["v"])
    kc, vc, slots = _f64(s["kc"]), _f64(s["vc"]), s["slots"].cpu().numpy()
    for cache, x, scale in ((kc, k, s["ks"]), (vc, v, s["vs"])):
        x = x if scale is None else np.clip(x / float(scale.item()), -448.0, 448.0)
        cache.reshape(-1, *cache.shape[2:])[slots[slots >= 0]] = x[slots >= 0]
    return q, kc, vc


def _summarize64(s, case):
    bs = case["block"]
    codes, scales = s["codes"].cpu().numpy().astype(np.int64), _f64(s["scales"])
    slots = s["slots"].cpu().numpy()
    for b in sorted(set((slots[slots >= 0] // bs)[slots[slots >= 0] % bs == bs - 1].tolist())):
        k = _f64(s["kc"][b:b + 1].view(torch.uint8).view(s["kc"].dtype))[0] if case["kv"] == "fp8" else _f64(s["kc"][b])
        k = np.clip(k, -2.0 ** 50, 2.0 ** 50)
        hi, lo = k.max(0), k.min(0)
        amax = np.maximum(np.abs(hi), np.abs(lo)).max(-1)
        e = np.full(amax.shape, -50)
        while (amax > 127 * np.exp2(e)).any():
            e = e + (amax > 127 * np.exp2(e))
        u = np.exp2(e.astype(np.float64))
        codes[b, :, 0], codes[b, :, 1] = np.ceil(hi / u[:, None]), np.floor(lo / u[:, None])
        scales[b] = u
    return codes, scales


def _select64(s, case):
    bs, hk, top, d = case["block"], case["kv_heads"], case["top"], case["dim"]
    q = _f64(s["q"])
    rows, group = q.shape[0], case["heads"] // hk
    tables, lens = s["tables"].cpu().numpy(), s["lens"].cpu().numpy()
    seq = np.arange(rows) if s["row_seqs"] is None else s["row_seqs"].cpu().numpy()
    out = np.full((rows, hk, top), -1, np.int64)
    for r in range(rows):
        nb = -(-int(lens[r]) // bs)
        if nb <= top:
            out[r, :, :nb] = np.arange(nb)
            continue
        ids = torch.as_tensor(tables[seq[r], 1:nb - 1].astype(np.int64), device=DEV)
        f, us = s["codes"][ids].double(), s["scales"][ids].double()
        for h in range(hk):
            score = np.full(nb - 2, -np.inf)
            for i in range(group):
                x = q[r, h * group + i]
                e = -50
                while np.abs(x).max() > 127 * 2.0 ** e:
                    e += 1
                c = torch.as_tensor(np.rint(x * 2.0 ** -e), device=DEV)
                most = torch.maximum(f[:, h, 0] * c, f[:, h, 1] * c).sum(-1) * us[:, h] * 2.0 ** e
                score = np.maximum(score, most.cpu().numpy())
            best = 1 + np.argsort(-score, kind="stable")[:top - 2]
            out[r, h] = np.sort(np.concatenate([[0, nb - 1], best]))
    return out


def _attend64(s, case):
    bs, hk, d = case["block"], case["kv_heads"], case["dim"]
    group = case["heads"] // hk
    lens, sel = s["lens"].cpu().numpy(), s["selected"].cpu().numpy()
    seq = np.arange(len(lens)) if s["row_seqs"] is None else s["row_seqs"].cpu().numpy()
    kk, vv = (c.view(-1, hk, d) for c in (s["kc"].view(torch.uint8), s["vc"].view(torch.uint8))) if case["kv"] == "fp8" \
        else (c.view(-1, hk, d) for c in (s["kc"], s["vc"]))
    tables = s["tables"].cpu().numpy()
    out = torch.zeros(len(lens), case["heads"], d, dtype=torch.float64, device=DEV)
    a = 1.0 if s["ks"] is None else float(s["ks"].item())
    b = 1.0 if s["vs"] is None else float(s["vs"].item())
    for r in range(len(lens)):
        for h in range(hk):
            pos = (sel[r, h][sel[r, h] >= 0][:, None] * bs + np.arange(bs)).reshape(-1)
            pos = pos[pos < lens[r]]
            slot = torch.as_tensor(tables[seq[r]][pos // bs].astype(np.int64) * bs + pos % bs, device=DEV)
            k, v = kk[slot, h], vv[slot, h]
            if case["kv"] == "fp8":
                k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            k, v = k.float().double() * a, v.float().double() * b
            x = s["q"][r, h * group:(h + 1) * group].double()
            out[r, h * group:(h + 1) * group] = torch.softmax(x @ k.T * s["scale"], -1) @ v
    return out
