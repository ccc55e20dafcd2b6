"""Cases, inputs and plain forms of the scored serving step's operators.

The step of a layer that normalises its queries and keys and changes its
scores: each head's queries and keys are normalised, rotated by position and
the keys and values appended to the paged cache, which may hold them in 8
bits under a scale for each token and head (``store``); a cache is read back
as contiguous bf16 rows (``read``); a new token of every sequence attends to
the cache with its scores capped by a tanh, biased by distance or kept to a
window (``decode``); so do the tokens of prompts and chunks, whose first
tokens may also see a whole prefix (``prompt``).

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
EPS = 1e-6


def listed():
    """Twelve cases.  The heads are the repository's own: 32 query and 8 KV
    heads of 128 channels (its headline layer), 32 / 32 (its serving mix),
    4 / 2 of 64 channels (its tiny case); 16 tokens a block unless said."""
    return [
        # one user's single new token: latency alone
        store("store-step-1", 1, 32, 8, 128, 128, True, False, "bf16", 16),
        # the decode step of a batch of 64 into 8 bits, and the tokens as
        # later steps will see them
        store("store-step-64-int8", 64, 32, 8, 128, 128, True, False, "int8", 16),
        # a long prompt
        store("store-prompt-8192", 8192, 32, 8, 128, 128, True, False, "bf16", 16),
        # a ragged chunk into 8 bits, read back for its attention; half the
        # channels rotated in neighbouring pairs, large blocks
        store("store-chunk-1021-int8", 1021, 4, 2, 64, 32, True, True, "int8", 64),
        # the context of one user's next chunk
        read("read-chunk-fp8", 1, 32, 8, 128, 16, 8187, 0, "fp8"),
        # a batch's contexts, for prompts' attention or for another pool
        read("read-64-int8", 64, 32, 8, 128, 16, 2977, 0, "int8"),
        # one user's long context in 8 bits, scores capped
        decode("decode-1-128k-int8", 1, 32, 8, 128, 16, 131071, "int8", 30.0, 0, False),
        # the decode step of a batch of 64, scores capped
        decode("decode-64-cap", 64, 32, 8, 128, 16, 2977, "bf16", 50.0, 0, False),
        # the same batch in a layer with a window
        decode("decode-64-window-int8", 64, 32, 8, 128, 16, 2977, "int8", 50.0, 1000, False),
        # MHA, large batch, biased by distance, e4m3
        decode("decode-256-mha-bias-fp8", 256, 32, 32, 128, 16, 2900, "fp8", 0.0, 0, True),
        # four prompts, scores capped
        prompt("prompt-4x2048-cap", 4, 2048, 2048, 32, 8, 128, 16, "bf16", 50.0, 0, False, 0),
        # ragged chunks behind longer contexts: capped, biased by distance, a
        # window, and a prefix whose tokens all see each other
        prompt("prompt-chunks-prefix-fp8", 3, 509, 4093, 32, 8, 128, 16, "fp8", 30.0, 1500, True,
               3900),
    ]


def store(name, tokens, heads, kv_heads, dim, rot, norm, pairs, kv, block):
    return dict(name=name, op="store", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                rot=rot, norm=norm, pairs=pairs, kv=kv, block=block)


def read(name, seqs, heads, kv_heads, dim, block, context, first, kv):
    return dict(name=name, op="read", seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim,
                block=block, context=context, first=first, kv=kv)


def decode(name, seqs, heads, kv_heads, dim, block, context, kv, cap, window, bias):
    return dict(name=name, op="decode", seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim,
                block=block, context=context, kv=kv, cap=cap, window=window, bias=bias)


def prompt(name, seqs, new, context, heads, kv_heads, dim, block, kv, cap, window, bias, prefix):
    return dict(name=name, op="prompt", seqs=seqs, new=new, context=context, heads=heads,
                kv_heads=kv_heads, dim=dim, block=block, kv=kv, cap=cap, window=window, bias=bias,
                prefix=prefix)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "decode", "decode", "prompt", "prompt"])
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (32, 32, 128), (4, 2, 64), (8, 1, 128),
                                       (16, 2, 64), (8, 4, 128)])
    block = rng.choice([8, 16, 16, 32, 64, 128])
    kv = rng.choice(["bf16", "fp8", "int8"])
    if op == "store":
        tokens = _log(rng, 1, 8192 if kv_heads < 32 else 2048)
        case = store("", tokens, heads, kv_heads, dim, rng.choice([dim, dim, dim // 2, 0]),
                     rng.random() < 0.8, rng.random() < 0.4, kv, block)
    elif op == "read":
        seqs = _log(rng, 1, 64)
        context = _log(rng, 1, 131072 // max(seqs, 2) * 8 // max(8, kv_heads))
        case = read("", seqs, heads, kv_heads, dim, block, context,
                    rng.choice([0, rng.randint(0, context - 1)]), kv)
    else:
        cap = rng.choice([0.0, 30.0, 50.0])
        bias = rng.random() < 0.3
        if op == "decode":
            seqs = _log(rng, 1, 256)
            context = _log(rng, 1, 131072 // max(seqs, 2) * 8 // max(8, kv_heads))
            window = rng.choice([0, 0, _log(rng, 1, 4096)])
            case = decode("", seqs, heads, kv_heads, dim, block, context, kv, cap, window, bias)
        else:
            if dim != 128 or kv == "int8":  # 64 channels and 8-bit rows: a few tokens each
                seqs, new = _log(rng, 1, 16), rng.randint(1, 8)
                context = new + _log(rng, 1, 2000)
            else:
                seqs = rng.randint(1, 4)
                new = _log(rng, 1, 2048 // seqs)
                context = new + rng.choice([0, _log(rng, 1, 4096)])
            window = rng.choice([0, 0, _log(rng, 1, 4096)])
            prefix = rng.choice([0, 0, rng.randint(1, context)])
            case = prompt("", seqs, new, context, heads, kv_heads, dim, block, kv, cap, window,
                          bias, prefix)
    del case["name"]
    return case


# ------------------------------------------------------------------- sizes

def _lens(case):
    """The sequences' lengths fall from `context` to half of it."""
    n = case["seqs"]
    return [max(1, case["context"] - (case["context"] // 2) * i // n) for i in range(n)]


def _news(case):
    """New tokens of each request of a prompt call: from `new` down to half."""
    n = case["seqs"]
    return [max(1, min(m, case["new"] - (case["new"] // 2) * i // n))
            for i, m in enumerate(_lens(case))]


def _element(case):
    return 2 if case["kv"] == "bf16" else 1


def _row_bytes(case):
    """A token's keys (or values) of all heads in the cache, scales included."""
    return case["kv_heads"] * (case["dim"] * _element(case) + (4 if case["kv"] == "int8" else 0))


def work(case):
    op, d, hk, h = case["op"], case["dim"], case["kv_heads"], case["heads"]
    row = _row_bytes(case)
    if op == "store":
        n = case["tokens"]
        moved = n * ((h + 2 * hk) * d * 2 + case["rot"] * 4 + (4 if case["rot"] else 0) + 4
                     + h * d * 2 + 2 * row)
        if case["kv"] == "int8":  # and read back
            moved += n * (2 * row + 2 * hk * d * 2 + 4)
        return {"bytes": moved, "flops": n * (h + hk) * (3 * case["rot"] + 4 * d * case["norm"])}
    if op == "read":
        n = sum(max(0, m - case["first"]) for m in _lens(case))
        return {"bytes": n * (2 * row + 2 * hk * d * 2) + -(-n // case["block"]) * 4,
                "flops": n * 2 * hk * d}
    w = case["window"] or 1 << 40
    if op == "decode":
        seen = [min(m, w) for m in _lens(case)]
        return {"bytes": sum(seen) * 2 * row + sum(-(-m // case["block"]) for m in seen) * 4
                + case["seqs"] * (2 * h * d * 2 + 4), "flops": sum(seen) * h * d * 4}
    pairs = keys = 0
    for m, t in zip(_lens(case), _news(case)):
        pre = min(case["prefix"], m)
        pos = np.arange(m - t, m)
        end = np.maximum(pos + 1, np.where(pos < pre, pre, 0))
        start = np.maximum(0, pos + 1 - w)
        pairs += int((end - start).sum())
        keys += int(end.max() - start.min())
    return {"bytes": keys * 2 * row + sum(_news(case)) * 2 * h * d * 2, "flops": pairs * h * d * 4}


# ------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _cache(g, kv, *shape):
    """(cache, scale) of keys or values that a serving loop has cached: N(0, 1)
    in bf16; the e4m3 codes of such under a scale that puts amax near the
    type's largest; or codes in 8 bits under each token's and head's own
    scale, rows differing in size."""
    x = _normal(g, *shape)
    if kv == "bf16":
        return x, None
    if kv == "fp8":
        s = torch.full((1,), 5.0 / 448.0, device=DEV, dtype=torch.float32)
        return (x.float() / s).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), s
    x = x.float()
    s = x.abs().amax(-1) / 127.0
    codes = torch.round(x / s[..., None]).to(torch.int8)
    return codes, s * torch.exp2(torch.randn(s.shape, generator=g, device=DEV) * 0.3)


_tables = {}


def _table(rot):
    """Cosines, then sines, of every position's angles: a model's constant,
    computed in 64 bits and kept for the process's life."""
    if rot not in _tables:
        inv = ROPE_BASE ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(MAX_POSITION, device=DEV, dtype=torch.float64)[:, None] * inv
        _tables[rot] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    return _tables[rot]


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    h, d, hk, bs = case["heads"], case["dim"], case["kv_heads"], case["block"]
    s = {"case": case}
    if case["op"] == "store":
        n = case["tokens"]
        # one projection's result; queries, keys and values are views of it
        qkv = _normal(g, n, (h + 2 * hk) * d)
        s["q"] = qkv[:, :h * d].view(n, h, d)
        s["k"] = qkv[:, h * d:(h + hk) * d].view(n, hk, d)
        s["v"] = qkv[:, (h + hk) * d:].view(n, hk, d)
        if n <= 256:  # a decode step: each token the last of a sequence of its own
            lens = rng.integers(1, 4097, n)
            width, nb = -(-int(lens.max()) // bs), n + 2
            tables = rng.integers(0, nb, (n, width))
            tables[np.arange(n), (lens - 1) // bs] = rng.permutation(nb)[:n]
            first, starts, pos = lens - 1, np.arange(n + 1), lens - 1
            slots = tables[np.arange(n), pos // bs] * bs + pos % bs
            if n >= 32:
                slots[-3:] = -1  # the batch's padding
        else:  # a prompt, or a chunk in the midst of one
            at = int(rng.integers(0, 4096))
            width, nb = -(-(at + n) // bs), n // bs + 4
            tables = rng.integers(0, nb, (1, width))
            tables[0, at // bs:] = rng.permutation(nb)[:width - at // bs]
            first, lens, starts, pos = np.array([at]), np.array([at + n]), np.array([0, n]), at + np.arange(n)
            slots = tables[0, pos // bs] * bs + pos % bs
        s["slots"], s["tables"], s["lens"] = _dev(slots), _dev(tables), _dev(lens)
        s["first"], s["starts"] = _dev(first), _dev(starts)
        s["pos"] = _dev(pos) if case["rot"] else None
        s["table"] = _table(case["rot"]) if case["rot"] else None
        s["qw"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
        s["kw"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
        s["kc"], s["ks"] = _cache(g, case["kv"], nb, bs, hk, d)
        s["vc"], s["vs"] = _cache(g, case["kv"], nb, bs, hk, d)
        s["out"] = torch.empty(n, h, d, device=DEV, dtype=torch.bfloat16)
        s["k_rows"] = torch.empty(n, hk, d, device=DEV, dtype=torch.bfloat16)
        s["v_rows"] = torch.empty_like(s["k_rows"])
        return s
    lens = _lens(case)
    width = -(-case["context"] // bs)
    need = [-(-m // bs) for m in lens]
    nb = sum(need) + 2
    order, tables, at = rng.permutation(nb), np.zeros((len(lens), width), np.int32), 0
    for i, m in enumerate(need):
        tables[i, :m] = order[at:at + m]
        at += m
    s["tables"], s["lens"] = _dev(tables), _dev(lens)
    s["kc"], s["ks"] = _cache(g, case["kv"], nb, bs, hk, d)
    s["vc"], s["vs"] = _cache(g, case["kv"], nb, bs, hk, d)
    if case["op"] == "read":
        n = [max(0, m - case["first"]) for m in lens]
        s["starts"] = _dev(np.cumsum([0] + n))
        s["first"] = _dev([case["first"]] * len(lens))
        s["k_rows"] = torch.zeros(sum(n), hk, d, device=DEV, dtype=torch.bfloat16)
        s["v_rows"] = torch.zeros_like(s["k_rows"])
        return s
    rows = len(lens) if case["op"] == "decode" else sum(_news(case))
    # queries of some size, so that the largest scores come near the cap
    s["q"] = (_normal(g, rows, h, d) * 3).to(torch.bfloat16)
    s["scale"] = d ** -0.5
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, h + 1, device=DEV) / h) if case["bias"] else None
    s["out"] = torch.empty_like(s["q"])
    if case["op"] == "prompt":
        s["starts"] = _dev(np.cumsum([0] + _news(case)))
        s["prefix"] = _dev([min(case["prefix"], m) for m in lens]) if case["prefix"] else None
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        from paged_kv_cache_108_gb300 import ops
        if op == "store":
            ops.norm_rope_and_cache(s["out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"],
                                    s["pos"], s["table"], s["qw"], s["kw"], EPS, s["ks"], s["vs"],
                                    adjacent_pairs=case["pairs"])
            if case["kv"] != "int8":
                return s["out"], s["kc"], s["vc"]
        if op in ("store", "read"):
            ops.gather_cache(s["k_rows"], s["v_rows"], s["kc"], s["vc"], s["tables"], s["lens"],
                             s["starts"], s["first"], s["ks"], s["vs"])
            rows = s["k_rows"], s["v_rows"]
            return rows if op == "read" else (s["out"], *rows, s["ks"], s["vs"])
        if "ws" not in s:  # kept between calls, as a program keeps it
            s["ws"] = ops.alloc_scored_workspace(s["q"].shape[0], case["heads"], case["kv_heads"],
                                                 case["dim"])
        if op == "decode":
            ops.decode_scored(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"],
                              s["scale"], case["cap"], case["window"], s["slopes"], s["ks"],
                              s["vs"], s["ws"])
        else:
            ops.varlen_scored(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"],
                              s["starts"], s["scale"], case["cap"], case["window"], s["slopes"],
                              s["prefix"], s["ks"], s["vs"], s["ws"])
        return s["out"]
    return {"store": _store, "read": _read, "decode": _decode, "prompt": _prompt}[op](s)


def _values(cache, scale, *at):
    """What the cache holds at an index, in 32 bits."""
    if cache.dtype == torch.float8_e4m3fn:
        return cache.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale
    if cache.dtype == torch.int8:
        return cache[at].float() * scale[at][..., None]
    return cache[at].float()


def _read(s):
    row = torch.arange(s["k_rows"].shape[0], device=DEV)
    seq = torch.searchsorted(s["starts"][1:].contiguous(), row, right=True)
    pos = s["first"][seq] + row - s["starts"][seq]
    bs = s["case"]["block"]
    block = s["tables"][seq, pos // bs].long()
    return (_values(s["kc"], s["ks"], block, pos % bs).to(torch.bfloat16),
            _values(s["vc"], s["vs"], block, pos % bs).to(torch.bfloat16))


def _normalised(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _rotated(x, s):
    p = s["case"]["rot"] // 2
    if not p:
        return x
    row = s["table"][s["pos"].long()]
    cos, sin = row[:, None, :p], row[:, None, p:]
    pairs = s["case"]["pairs"]
    a, b = (x[..., 0:2 * p:2], x[..., 1:2 * p:2]) if pairs else (x[..., :p], x[..., p:2 * p])
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if pairs else -2).flatten(-2)
    return torch.cat([y, x[..., 2 * p:]], -1)


def _write(cache, scale, to, x):
    flat = cache.view(-1, *cache.shape[2:])
    if cache.dtype == torch.bfloat16:
        flat[to] = x.to(torch.bfloat16)
    elif cache.dtype == torch.float8_e4m3fn:
        codes = (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        flat.view(torch.uint8)[to] = codes.view(torch.uint8)
    else:
        unit = x.abs().amax(-1, keepdim=True) / 127.0
        flat[to] = torch.round(x / unit).clamp(-127, 127).to(torch.int8)
        scale.view(-1, scale.shape[2])[to] = unit[..., 0]


def _store(s):
    q = _rotated(_normalised(s["q"], s["qw"]), s).to(torch.bfloat16)
    k = _rotated(_normalised(s["k"], s["kw"]), s)
    there = s["slots"] >= 0
    to = s["slots"][there].long()
    _write(s["kc"], s["ks"], to, k[there])
    _write(s["vc"], s["vs"], to, s["v"].float()[there])
    if s["case"]["kv"] != "int8":
        return q, s["kc"], s["vc"]
    return (q, *_read(s), s["ks"], s["vs"])


def _context(s):
    """Keys and values of every sequence, [sequences, tokens, heads, d]."""
    t = s["tables"].long()
    return _values(s["kc"], s["ks"], t).flatten(1, 2), _values(s["vc"], s["vs"], t).flatten(1, 2)


def _attention(s, q, pos, end):
    """q: [sequences, kv heads, group, rows, d]; pos, end: [sequences, rows]."""
    case = s["case"]
    k, v = _context(s)
    x = torch.matmul(q.flatten(2, 3), k.permute(0, 2, 3, 1)).view(*q.shape[:-1], -1) * s["scale"]
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    at = torch.arange(k.shape[1], device=DEV)
    back = pos[..., None] - at
    if s["slopes"] is not None:
        x = x - s["slopes"].view(q.shape[1], -1, 1, 1) * back[:, None, None].abs().float()
    seen = at < end[..., None]
    if case["window"]:
        seen &= back < case["window"]
    x = torch.where(seen[:, None, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    out = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).view(q.shape)
    return out / p.sum(-1, keepdim=True)


def _decode(s):
    n, hk, d = s["q"].shape[0], s["case"]["kv_heads"], s["case"]["dim"]
    q = s["q"].float().view(n, hk, -1, 1, d)
    lens = s["lens"][:, None]
    return _attention(s, q, lens - 1, lens).view(n, -1, d).to(torch.bfloat16)


def _prompt(s):
    case, hk, d = s["case"], s["case"]["kv_heads"], s["case"]["dim"]
    n, seqs = s["q"].shape[0], case["seqs"]
    row = torch.arange(n, device=DEV)
    seq = torch.searchsorted(s["starts"][1:].contiguous(), row, right=True)
    j = row - s["starts"][seq]
    new = s["starts"][1:] - s["starts"][:-1]
    most = max(_news(case))
    q = torch.zeros(seqs, most, hk, case["heads"] // hk, d, device=DEV)
    q[seq, j] = s["q"].float().view(n, hk, -1, d)
    pos = (s["lens"] - new)[:, None] + torch.arange(most, device=DEV)
    end = pos + 1
    if s["prefix"] is not None:
        end = torch.where(pos < s["prefix"][:, None], s["prefix"][:, None], end)
    out = _attention(s, q.permute(0, 2, 3, 1, 4), pos, torch.minimum(end, s["lens"][:, None]))
    return out.permute(0, 3, 1, 2, 4)[seq, j].reshape(n, -1, d).to(torch.bfloat16)


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return _store64(s, case)
    if case["op"] == "read":
        return _rows64(s, case)
    return _attention64(s, case)


def _f64(x):
    return x.to(torch.float32).double()


def _token64(s, which, slot):
    """Rows [slots, kv heads, d] of one cache ("k" or "v") in 64 bits."""
    cache, scale = s[which + "c"], s[which + "s"]
    flat = cache.view(-1, *cache.shape[2:])
    if cache.dtype == torch.bfloat16:
        return _f64(flat[slot])
    if cache.dtype == torch.int8:
        return flat[slot].double() * scale.reshape(-1, scale.shape[2])[slot].double().unsqueeze(-1)
    return _f64(flat.view(torch.uint8)[slot].view(torch.float8_e4m3fn)) * float(scale.item())


def _slots64(s, case, seq, lo, hi):
    table = s["tables"][seq].cpu().numpy().astype(np.int64)
    t = np.arange(lo, hi)
    return torch.as_tensor(table[t // case["block"]] * case["block"] + t % case["block"], device=DEV)


def _rows64(s, case):
    first, lens = s["first"].cpu().numpy(), s["lens"].cpu().numpy()
    slot = torch.cat([_slots64(s, case, i, int(first[i]), max(int(first[i]), int(lens[i])))
                      for i in range(len(lens))])
    return _token64(s, "k", slot), _token64(s, "v", slot)


def _store64(s, case):
    p = case["rot"] // 2

    def turned(x, weight):
        x = _f64(x)
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
        if not p:
            return x
        # each pair as a complex number, turned by e^(i angle)
        row = s["table"][s["pos"].long()].double()
        turn = torch.complex(row[:, :p], row[:, p:]).unsqueeze(1)
        i = torch.arange(p, device=DEV)
        one, two = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + p)
        z = torch.complex(x[..., one], x[..., two]) * turn
        x = x.clone()
        x[..., one], x[..., two] = z.real, z.imag
        return x

    q, new = turned(s["q"], s["qw"]), {"k": turned(s["k"], s["kw"]), "v": _f64(s["v"])}
    slots = s["slots"].long()
    hit = slots >= 0
    if case["kv"] == "int8":
        # each written row's codes and scale, and what they stand for
        units = {}
        rows = dict(zip("kv", _rows64(s, case)))
        for w in "kv":
            unit = new[w].abs().max(-1).values / 127
            units[w] = s[w + "s"].double()
            units[w].view(-1, case["kv_heads"])[slots[hit]] = unit[hit]
            held = torch.round(new[w] / unit.unsqueeze(-1)) * unit.unsqueeze(-1)
            rows[w][hit] = held[hit]  # row i of the read is token i
        return q, rows["k"], rows["v"], units["k"], units["v"]
    out = [q]
    for w in "kv":
        cache = s[w + "c"]
        all_rows = _f64(cache.view(torch.uint8).view(cache.dtype)).clone()
        x = new[w] if case["kv"] == "bf16" else (new[w] / float(s[w + "s"].item())).clamp(-448, 448)
        all_rows.view(-1, case["kv_heads"], case["dim"])[slots[hit]] = x[hit]
        out.append(all_rows)
    return tuple(out)


def _attention64(s, case):
    hk, d, group = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    lens = _lens(case)
    news = [1] * len(lens) if case["op"] == "decode" else _news(case)
    out = torch.empty(sum(news), case["heads"], d, dtype=torch.float64, device=DEV)
    at = 0
    for i, (m, t) in enumerate(zip(lens, news)):
        pos = torch.arange(m - t, m, device=DEV)
        limit = pos + 1
        if case.get("prefix"):
            pre = min(case["prefix"], m)
            limit = torch.where(pos < pre, torch.full_like(pos, pre).maximum(limit), limit)
        low = max(0, m - t + 1 - case["window"]) if case["window"] else 0
        slot = _slots64(s, case, i, low, m)
        k, v = _token64(s, "k", slot), _token64(s, "v", slot)
        key = torch.arange(low, m, device=DEV)
        gap = pos[:, None] - key[None, :]
        hidden = key[None, :] >= limit[:, None]
        if case["window"]:
            hidden = hidden | (gap >= case["window"])
        for c in range(case["heads"]):
            x = (_f64(s["q"][at:at + t, c]) @ k[:, c // group].T) * s["scale"]
            if case["cap"]:
                x = torch.tanh(x / case["cap"]) * case["cap"]
            if s["slopes"] is not None:
                x = x - float(s["slopes"][c].item()) * gap.abs()
            x = x.masked_fill(hidden, -math.inf)
            out[at:at + t, c] = torch.softmax(x, -1) @ v[:, c // group]
        at += t
    return out
