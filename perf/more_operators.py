"""What stands between the projection's rows and a cache in 4 bits, at the sizes it is used at: norms of
queries and keys with the rotation by position, attention of whole prompts packed behind one another,
keys and values written into pages in 4 bits and read back, and attention of drafted trees over such a
cache. Each in its plain form (elementary torch operations, 32 bits, 64 for the angles of far positions)
and as the framework's calls (`own`)."""

import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GROUP = 32  # elements of a row that share a scale and a minimum


def listed():
    return [
        # One sequence, one token a step: what an interactive user waits for.
        {"name": "rotate one token", "op": "rotate", "b": 1, "n": 1, "hq": 40, "hkv": 8, "d": 128, "rot": 128, "pos": 1021,
         "dt": "bf16", "norm": True, "pairs": False},
        # The rows of long prompts, far positions among them.
        {"name": "rotate prompts", "op": "rotate", "b": 4, "n": 4099, "hq": 32, "hkv": 8, "d": 128, "rot": 64, "pos": 100000,
         "dt": "bf16", "norm": True, "pairs": False},
        # A short question.
        {"name": "prompt, short", "op": "prompt", "b": 1, "len": 77, "hq": 40, "hkv": 8, "d": 128, "pad": 0, "dt": "bf16"},
        # A batch of ragged prompts in a buffer of a fixed size, as a captured graph has them.
        {"name": "prompts, ragged", "op": "prompt", "b": 24, "len": 2050, "hq": 32, "hkv": 8, "d": 128, "pad": 61, "dt": "f16"},
        # One document.
        {"name": "prompt, long", "op": "prompt", "b": 1, "len": 16384, "hq": 32, "hkv": 8, "d": 128, "pad": 0, "dt": "bf16"},
        # The accepted path of every sequence goes into its pages after a step, and is looked at there.
        {"name": "append accepted", "op": "append", "b": 64, "n": 16, "hkv": 8, "d": 128, "len": 4099, "page": 16,
         "dt": "bf16", "path": True, "heads_first": False},
        # A prompt's keys and values go into pages, and come back.
        {"name": "append prompts", "op": "append", "b": 4, "n": 8192, "hkv": 8, "d": 128, "len": 1000, "page": 64,
         "dt": "bf16", "path": False, "heads_first": True},
        # One sequence moves to a cache in 16 bits.
        {"name": "read one sequence", "op": "read", "b": 1, "len": 1021, "hkv": 8, "d": 128, "page": 16, "dt": "f16",
         "heads_first": False},
        # A serving batch moves.
        {"name": "read a batch", "op": "read", "b": 8, "len": 16384, "hkv": 8, "d": 128, "page": 128, "dt": "bf16",
         "heads_first": True},
        # One sequence, one token a step.
        {"name": "attn one token", "op": "attn", "b": 1, "n": 1, "hq": 40, "hkv": 8, "d": 128, "len": 1021,
         "page": 16, "dt": "bf16", "heads_first": False},
        # Chains of 7 drafts and the last token over ragged sequences: a serving batch.
        {"name": "attn chains, ragged", "op": "attn", "b": 24, "n": 8, "hq": 32, "hkv": 8, "d": 128, "len": 4099,
         "page": 64, "dt": "f16", "heads_first": False},
        # A full serving batch over long contexts: what the 4 bits are for.
        {"name": "attn long contexts", "op": "attn", "b": 32, "n": 16, "hq": 32, "hkv": 8, "d": 128, "len": 16384,
         "page": 128, "dt": "bf16", "heads_first": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "prompt", "prompt", "append", "read", "attn", "attn", "attn"])
    hkv, d = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 96, 128, 128, 256])
    group, page, heads_first = rng.choice([1, 2, 4, 5, 6, 8]), rng.choice([1, 16, 24, 32, 64, 100, 256]), rng.random() < 0.5
    half = rng.choice(["bf16", "f16"])
    if op == "rotate":
        c = {"op": op, "b": _log(rng, 1, 32), "n": _log(rng, 1, 4096), "hq": hkv * group, "hkv": hkv, "d": d,
             "rot": rng.choice([d, d, d // 2, d // 4]), "pos": _log(rng, 1, 1 << 20), "dt": rng.choice(["bf16", "f16", "f32"]),
             "norm": rng.random() < 0.8, "pairs": rng.random() < 0.4}
        while c["b"] * c["n"] * (c["hq"] + hkv) * d > 1 << 26:
            c["n"] = max(1, c["n"] // 2)
        return c
    if op == "prompt":
        c = {"op": op, "b": _log(rng, 1, 48), "len": _log(rng, 1, 8192), "hq": hkv * group, "hkv": hkv, "d": d,
             "pad": rng.choice([0, 0, 1, 200]), "dt": half}
        while c["b"] * c["len"] ** 2 * c["hq"] * d > 1 << 38 or c["b"] * c["len"] * c["hq"] * d > 1 << 27:
            c["b"], c["len"] = max(1, c["b"] // 2), max(1, c["len"] * 3 // 4)
        return c
    if op == "append":
        return {"op": op, "b": _log(rng, 1, 64), "n": _log(rng, 1, 512), "hkv": hkv, "d": d, "len": _log(rng, 1, 4096),
                "page": page, "dt": rng.choice(["bf16", "f16", "f32"]), "path": rng.random() < 0.5, "heads_first": heads_first}
    if op == "read":
        c = {"op": op, "b": _log(rng, 1, 32), "len": _log(rng, 1, 16384), "hkv": hkv, "d": d, "page": page,
             "dt": rng.choice(["bf16", "f16", "f32"]), "heads_first": heads_first}
        while c["b"] * c["len"] * hkv * d > 1 << 26:
            c["b"], c["len"] = max(1, c["b"] // 2), max(1, c["len"] * 3 // 4)
        return c
    c = {"op": op, "b": _log(rng, 1, 32), "n": _log(rng, 1, 64), "hq": hkv * group, "hkv": hkv, "d": d,
         "len": _log(rng, 1, 32768), "page": page, "dt": half, "heads_first": heads_first}
    while c["b"] * (c["len"] + c["n"]) * hkv * d > 1 << 28 or c["b"] * c["n"] * c["hq"] * d * c["len"] > 1 << 34:
        c["b"], c["len"] = max(1, c["b"] // 2), max(1, c["len"] * 3 // 4)
    return c


def _lengths(case):
    """Tokens of each sequence: the first has them all, the others from a quarter up (long ones near the full length)."""
    r = random.Random(case["len"] * 64 + case["b"])
    full = case["len"]
    if full >= 8192 and case["op"] != "prompt":
        return [full - r.randrange(1 + full // 64) * (b > 0) for b in range(case["b"])]
    return [full if b == 0 else r.randint((full + 3) // 4, full) for b in range(case["b"])]


def _counts(case):
    """Tokens of each sequence that an append takes."""
    r = random.Random(case["b"] * 1000 + case["n"])
    return [r.randint(1, max(1, min(case["n"], 6))) if case["path"] else case["n"] for _ in range(case["b"])]


def _row_bytes(d):
    return d // 2 + d // GROUP * 4


def work(case):
    e, d = (4 if case["dt"] == "f32" else 2), case["d"]
    if case["op"] == "rotate":
        return {"bytes": 2 * case["b"] * case["n"] * (case["hq"] + case["hkv"]) * d * e, "flops": 0}
    if case["op"] == "prompt":
        rows = sum(_lengths(case))
        seen = sum(n * (n + 1) // 2 for n in _lengths(case))
        return {"bytes": rows * (case["hq"] + case["hkv"]) * 2 * d * e, "flops": 4 * seen * case["hq"] * d}
    if case["op"] == "append":  # rows read, written in 4 bits, read there and given back
        rows = 2 * sum(_counts(case)) * case["hkv"]
        return {"bytes": rows * (2 * d * e + 2 * _row_bytes(d)), "flops": 0}
    if case["op"] == "read":
        rows = 2 * sum(_lengths(case)) * case["hkv"]
        return {"bytes": rows * (d * e + _row_bytes(d)), "flops": 0}
    rows = case["b"] * case["n"] * case["hq"]
    seen = sum(n * case["n"] for n in _lengths(case)) + case["b"] * case["n"] * (case["n"] + 1) // 2
    cache = 2 * (sum(_lengths(case)) * _row_bytes(d) + case["b"] * case["n"] * d * e) * case["hkv"]
    return {"bytes": cache + rows * 2 * d * e, "flops": 4 * seen * case["hq"] * d}


def _cache(case, room, g, filled):
    """Caches in 4 bits with `room` positions a sequence behind its length, pages handed out in random order."""
    per = -(-(max(_lengths(case)) + room) // case["page"])
    pages = case["b"] * per + 3
    order = (pages, case["hkv"], case["page"]) if case["heads_first"] else (pages, case["page"], case["hkv"])
    caches = []
    for _ in range(2):
        c = torch.zeros((*order, _row_bytes(case["d"])), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 27) // (case["page"] * case["hkv"] * case["d"]))
        for p in range(0, pages if filled else 0, step):
            x = torch.randn((*c[p:p + step].shape[:3], case["d"]), generator=g, device=DEV)
            c[p:p + step] = _to_bytes(*_quantise(x.to(DT[case["dt"]])))
        caches.append(c.transpose(1, 2) if case["heads_first"] else c)
    table = torch.randperm(pages, generator=g, device=DEV)[: case["b"] * per].view(case["b"], per).to(torch.int32)
    return *caches, table, torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)


def _tree(b, n, g):
    """Masks of drafted trees: node 0 is the last token, every other node hangs on an earlier one; [b, n] and [b, n, n]."""
    i = torch.arange(n, device=DEV)
    back = (torch.rand((b, n), generator=g, device=DEV) * 6).long() + 1
    parents = torch.where(i > 0, (i - back).clamp(min=0), -1)
    up = (parents[:, :, None] == i).double()
    seen = torch.linalg.matrix_power(up + torch.eye(n, device=DEV, dtype=torch.float64), n) > 0
    return (seen * (torch.ones((), dtype=torch.int64, device=DEV) << i)).sum(-1), seen


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    dt = DT[case["dt"]]
    if case["op"] == "rotate":
        b, n, hq, hkv, d = (case[k] for k in ("b", "n", "hq", "hkv", "d"))
        rows = torch.randn((b, n, hq + 2 * hkv, d), generator=g, device=DEV, dtype=dt)  # the fused projection's rows
        rows *= torch.rand((b, n, 1, 1), generator=g, device=DEV).add_(0.1).to(dt) * 10
        s["q"], s["k"], _ = rows.split([hq, hkv, hkv], dim=2)
        begin = torch.randint(0, case["pos"] + 1, (b, 1), generator=g, device=DEV)
        s["positions"] = (begin + torch.arange(n, device=DEV)).to(torch.int32)
        s["frequencies"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV).double() / case["rot"])).float()
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"], s["kw"] = (torch.randn((d,), generator=g, device=DEV).mul_(0.2).add_(1).to(dt) for _ in range(2))
    elif case["op"] == "prompt":
        tokens = sum(_lengths(case)) + case["pad"]
        heads = [case["hq"], case["hkv"], case["hkv"]]
        qkv = torch.randn((tokens, sum(heads), case["d"]), generator=g, device=DEV, dtype=dt)
        s["q"], s["k"], s["v"] = qkv.split(heads, dim=1)
        s["offsets"] = torch.tensor([0] + _lengths(case), device=DEV).cumsum(0).to(torch.int32)
        if case["pad"]:
            s["out"] = torch.zeros((tokens, case["hq"], case["d"]), dtype=dt, device=DEV)
    elif case["op"] == "append":
        b, n = case["b"], case["n"]
        kv = torch.randn((b, n, 2, case["hkv"], case["d"]), generator=g, device=DEV, dtype=dt)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        s["kc"], s["vc"], s["table"], s["lengths"] = _cache(case, n, g, False)
        s["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=DEV)
        s["after"] = s["lengths"] + s["counts"]
        if case["path"]:
            order = torch.rand((b, n), generator=g, device=DEV)
            order[:, 0] = -1.0
            at = torch.arange(n, device=DEV)
            kept = torch.where(at < s["counts"][:, None], order.argsort(1), n).sort(1).values
            s["nodes"] = torch.where(at < s["counts"][:, None], kept, -1).to(torch.int32)
    elif case["op"] == "read":
        s["kc"], s["vc"], s["table"], s["lengths"] = _cache(case, 0, g, True)
    else:
        b, n = case["b"], case["n"]
        heads = [case["hq"], case["hkv"], case["hkv"]]
        qkv = torch.randn((b, n, sum(heads), case["d"]), generator=g, device=DEV, dtype=dt)
        s["q"], s["k"], s["v"] = qkv.split(heads, dim=2)
        s["kc"], s["vc"], s["table"], s["lengths"] = _cache(case, n, g, True)
        s["mask"], s["seen"] = _tree(b, n, g)
    return s


# ---------------------------------------------------------------- plain forms


def _quantise(x):
    """Codes 0 .. 15, scale and minimum (fp16) of each group of a row."""
    x = torch.nan_to_num(x.float().unflatten(-1, (-1, GROUP)), nan=0.0).clamp(-65504.0, 65504.0)
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale, low = ((high - low) / torch.full_like(low, 15.0)).half(), low.half()
    n = torch.round((x - low.float()) / scale.float()).clamp(0, 15)
    return torch.where(scale > 0, n, 0).to(torch.uint8), scale, low


def _to_bytes(n, scale, low):
    """A row's codes, 8 of them in 4 bytes (the even ones below the odd ones), then its scales and minima."""
    e = n.flatten(-2).unflatten(-1, (-1, 8))
    codes = (e[..., [0, 4, 1, 5]] | (e[..., [2, 6, 3, 7]] << 4)).flatten(-2)
    return torch.cat([codes, torch.cat([scale, low], -1).flatten(-2).contiguous().view(torch.uint8)], -1)


def _values(rows, dt):
    """The values that rows of bytes stand for."""
    d = rows.shape[-1] * 8 // 5
    b = rows[..., : d // 2].unflatten(-1, (-1, 4))
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2)[..., [0, 4, 1, 5, 2, 6, 3, 7]].flatten(-2).unflatten(-1, (-1, GROUP))
    pair = rows[..., d // 2:].contiguous().view(torch.float16).unflatten(-1, (-1, 2)).float()
    return (n.float() * pair[..., :1] + pair[..., 1:]).flatten(-2).to(dt)


def _turned(x, w, angle, s):
    if s["norm"]:
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    a, rest = x.float().split([s["rot"], s["d"] - s["rot"]], -1)
    a = a.unflatten(-1, (-1, 2) if s["pairs"] else (2, -1))
    one, two = a.unbind(-1 if s["pairs"] else -2)
    c, n = angle.cos().float(), angle.sin().float()
    a = torch.stack([one * c - two * n, one * n + two * c], -1 if s["pairs"] else -2).flatten(-2)
    return torch.cat([a, rest], -1).to(DT[s["dt"]])


def _rotate(s):
    angle = (s["positions"].double()[..., None] * s["frequencies"].double())[:, :, None]
    return _turned(s["q"], s["qw"], angle, s), _turned(s["k"], s["kw"], angle, s)


def _prompt(s):
    out = s["out"] if s["pad"] else torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    group, begin = s["hq"] // s["hkv"], 0
    for n in _lengths(s):
        rows = slice(begin, begin + n)
        hidden = torch.ones((n, n), dtype=torch.bool, device=DEV).triu(1)
        for h in range(s["hkv"]):
            heads = slice(h * group, (h + 1) * group)
            q, k, v = s["q"][rows, heads].float(), s["k"][rows, h].float(), s["v"][rows, h].float()
            x = torch.matmul(q.transpose(0, 1).contiguous(), k.t().contiguous()) * s["d"] ** -0.5
            x.masked_fill_(hidden, -math.inf)
            x = x.sub_(x.amax(-1, keepdim=True)).exp_()
            x = x.div_(x.sum(-1, keepdim=True))
            out[rows, heads] = torch.matmul(x, v).transpose(0, 1).to(out.dtype)
        begin += n
    return out


def _places(table, positions, page):
    """Page and slot of positions [b, n] by the table."""
    return table.long().gather(1, positions // page), positions % page


def _append(s):
    b, n = s["k"].shape[:2]
    at = torch.arange(n, device=DEV)
    kept = at < s["counts"][:, None]
    node = s["nodes"].long().clamp(min=0) if s["path"] else at.expand(b, n)
    to = _places(s["table"], s["lengths"].long()[:, None] + at, s["kc"].shape[1])
    here = to[0][kept], to[1][kept]
    seq = torch.arange(b, device=DEV)[:, None].expand(b, n)[kept]
    back = []
    for rows, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
        cache[here] = _to_bytes(*_quantise(rows[seq, node[kept]]))
        back.append(torch.where(kept[:, :, None, None], _values(cache[to], rows.dtype), 0))
    return back


def _gather(cache, table, lengths, dt):
    """[b, positions, hkv, d] values of the cache by position, and which of them are there."""
    rows = _values(cache[table.long()], dt).flatten(1, 2)
    there = torch.arange(rows.shape[1], device=DEV) < lengths[:, None]
    return torch.where(there[:, :, None, None], rows, 0), there


def _read(s):
    return [_gather(c, s["table"], s["lengths"], DT[s["dt"]])[0][:, : s["len"]].contiguous() for c in (s["kc"], s["vc"])]


def _attn(s):
    b, n, hq, d = s["q"].shape
    hkv = s["k"].shape[2]
    kc, there = _gather(s["kc"], s["table"], s["lengths"], s["q"].dtype)
    k = torch.cat([kc, s["k"]], 1).transpose(1, 2).float()
    del kc
    q = s["q"].float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    seen = torch.cat([there[:, None].expand(b, n, -1), s["seen"]], 2)[:, None, :, None]
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * d ** -0.5
    del k
    x = x.view(b, hkv, n, hq // hkv, -1).masked_fill(~seen, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    e = (e / e.sum(-1, keepdim=True)).view(b, hkv, -1, x.shape[-1])
    v = torch.cat([_gather(s["vc"], s["table"], s["lengths"], s["q"].dtype)[0], s["v"]], 1).transpose(1, 2).float()
    o = torch.matmul(e, v.contiguous())
    return o.view(b, hkv, n, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d).to(s["q"].dtype)


def run(s):
    if not own:
        return {"rotate": _rotate, "prompt": _prompt, "append": _append, "read": _read, "attn": _attn}[s["op"]](s)
    import trellis_quantized_linear_tf_amd as tq

    if s["op"] == "rotate":
        return tq.norm_rotate(s["q"], s["k"], s["positions"], s["frequencies"], s["qw"], s["kw"],
                              eps=1e-6 if s["norm"] else None, interleaved=s["pairs"])
    if s["op"] == "prompt":
        return tq.prompt_attention(s["q"], s["k"], s["v"], s["offsets"], out=s.get("out"))
    if s["op"] == "append":
        tq.cache_append_q4(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lengths"], s.get("nodes"), s["counts"])
        return tq.cache_read_q4(s["kc"], s["vc"], s["table"], s["after"], s["n"], first=s["lengths"], dtype=s["k"].dtype)
    if s["op"] == "read":
        return tq.cache_read_q4(s["kc"], s["vc"], s["table"], s["lengths"], s["len"], dtype=DT[s["dt"]])
    return tq.tree_attention_q4(s["q"], s["k"], s["v"], s["mask"], s["kc"], s["vc"], s["table"], s["lengths"])


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "prompt": _exact_prompt, "append": _exact_append, "read": _exact_read,
            "attn": _exact_attn}[case["op"]](s)


def _exact_rotate(s):
    t = s["positions"].double()[:, :, None, None] * s["frequencies"].double()
    turn = torch.polar(torch.ones_like(t), t)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double()
        if s["norm"]:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / s["d"] + 1e-6) * w.double()
        y = y.clone()
        r = s["rot"]
        first, second = (slice(0, r, 2), slice(1, r, 2)) if s["pairs"] else (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_prompt(s):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    ends = s["offsets"].tolist()
    for i, j in zip(ends, ends[1:]):
        for h in range(s["hq"]):
            k, v = (s[c][i:j, h * s["hkv"] // s["hq"]].double() for c in "kv")
            for r in range(i, j, 4096):  # rows r .. t - 1 against all keys up to t - 1
                t = min(r + 4096, j)
                x = torch.mm(s["q"][r:t, h].double(), k[: t - i].t().contiguous()) / math.sqrt(s["d"])
                x[torch.arange(t - i, device=DEV) > torch.arange(r - i, t - i, device=DEV)[:, None]] = -math.inf
                o[r:t, h] = torch.mm(torch.softmax(x, 1), v[: t - i].contiguous())
    return o


def _stands_for(x):
    """What a row of numbers becomes in 4 bits."""
    x = x.double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    scale = ((high - low) / 15).float().half().double()
    low = low.float().half().double()
    steps = ((x - low).float().double() / scale).float().double()  # the definition's two roundings to 32 bits
    n = torch.where(scale > 0, steps.round().clamp(0, 15), 0)
    return (low + scale * n).flatten(-2)


def _exact_append(s):
    outs = []
    for x in (s["k"], s["v"]):
        o = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
        for i, count in enumerate(s["counts"].tolist()):
            rows = x[i, s["nodes"][i, :count].long()] if s["path"] else x[i, :count]
            o[i, :count] = _stands_for(rows)
        outs.append(o)
    return outs


def _decoded(rows):
    """[rows, heads, d] in 64 bits of bytes [rows, heads, 5 d / 8], code by code."""
    d = rows.shape[-1] * 8 // 5
    words = rows[..., : d // 2].contiguous().view(torch.int32).long() & 0xFFFFFFFF
    at = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=DEV)
    codes = (words[..., None] >> at & 15).flatten(-2).double()
    pairs = rows[..., d // 2:].contiguous().view(torch.float16).double().unflatten(-1, (-1, 2)).repeat_interleave(GROUP, -2)
    return codes * pairs[..., 0] + pairs[..., 1]


def _exact_read(s):
    outs = []
    for cache in (s["kc"], s["vc"]):
        o = torch.zeros((s["b"], s["len"], s["hkv"], s["d"]), dtype=torch.float64, device=DEV)
        for i, length in enumerate(s["lengths"].tolist()):
            pos = torch.arange(length, device=DEV)
            o[i, :length] = _decoded(cache[s["table"][i, pos // s["page"]].long(), pos % s["page"]])
        outs.append(o)
    return outs


def _exact_attn(s):
    b, n, hq, d = s["q"].shape
    hkv, page = s["k"].shape[2], s["kc"].shape[1]
    o = torch.zeros((b, n, hq, d), dtype=torch.float64, device=DEV)
    for i, length in enumerate(s["lengths"].tolist()):
        pos = torch.arange(length, device=DEV)
        at = s["table"][i, pos // page].long(), pos % page
        k, v = (torch.cat([_decoded(c[at]).to(x.dtype), x[i]]).double() for c, x in ((s["kc"], s["k"]), (s["vc"], s["v"])))
        hidden = torch.cat([torch.zeros((n, length), dtype=torch.bool, device=DEV), ~s["seen"][i]], 1)
        for j in range(hq):
            h = j * hkv // hq
            x = torch.mm(s["q"][i, :, j].double(), k[:, h].t().contiguous()) / math.sqrt(d)
            x[hidden] = -math.inf
            o[i, :, j] = torch.mm(torch.softmax(x, 1), v[:, h].contiguous())
    return o
