"""The operators around the projection at the sizes they are used at: attention of a tree
of drafted tokens over a paged cache, the cache's append, the verification of the drafts
against the head's logits, and the distillation that trains a drafter on a teacher's top
logits. Each in its plain form (elementary torch operations, 32 bits, 64 where a sampled
token stands next to a border) and as the framework's calls (`own`)."""

import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
VOCAB = 129280  # the LM head's columns


def listed():
    return [
        # One sequence, one token a step: what an interactive user waits for.
        {"name": "attn one token", "op": "attn", "b": 1, "n": 1, "hq": 40, "hkv": 8, "d": 128, "len": 1021,
         "page": 16, "dt": "bf16", "heads_first": False},
        # Chains of 7 drafts and the last token over ragged sequences: a serving batch.
        {"name": "attn chains, ragged", "op": "attn", "b": 24, "n": 8, "hq": 32, "hkv": 8, "d": 128, "len": 4099,
         "page": 64, "dt": "f16", "heads_first": False},
        # Wide trees: so many rows share a key that the matrix cores, not the cache, bound the pass.
        {"name": "attn 64-node trees", "op": "attn", "b": 4, "n": 64, "hq": 48, "hkv": 8, "d": 128, "len": 8191,
         "page": 16, "dt": "bf16", "heads_first": True},
        # A full serving batch over long contexts: the cache's bytes are the pass.
        {"name": "attn long contexts", "op": "attn", "b": 32, "n": 16, "hq": 32, "hkv": 8, "d": 128, "len": 16384,
         "page": 128, "dt": "bf16", "heads_first": False},
        # The accepted path of every sequence goes into its pages after a step.
        {"name": "append accepted", "op": "append", "b": 64, "n": 16, "hkv": 8, "d": 128, "len": 4099, "page": 16,
         "dt": "bf16", "path": True, "heads_first": False},
        # A prompt's keys and values go into pages.
        {"name": "append prompts", "op": "append", "b": 4, "n": 8192, "hkv": 8, "d": 128, "len": 1000, "page": 64,
         "dt": "bf16", "path": False, "heads_first": True},
        # One sequence's tree, fp32 logits as the head gives them.
        {"name": "verify one tree", "op": "tree", "b": 1, "n": 16, "v": VOCAB, "dt": "f32", "hot": False},
        # A serving batch of trees, bf16 logits, a part of the users at temperature 0.
        {"name": "verify trees", "op": "tree", "b": 32, "n": 24, "v": VOCAB, "dt": "bf16", "hot": True},
        # A serving batch of sampled chains with the drafter's probabilities.
        {"name": "verify chains", "op": "chain", "b": 64, "n": 8, "v": VOCAB, "dt": "f32", "hot": True},
        # A few rows: a drafter adapted while it serves.
        {"name": "distill few rows", "op": "distill", "r": 16, "v": VOCAB, "k": 64, "dt": "f32", "dirs": "both", "t": 1.0},
        # Another vocabulary, rows that start at odd addresses; loss, then gradient, as autograd asks for them.
        {"name": "distill odd vocabulary", "op": "distill", "r": 1000, "v": 50257, "k": 20, "dt": "f16", "dirs": "apart",
         "t": 2.0},
        # A training step's tokens: loss and gradient together.
        {"name": "distill a batch", "op": "distill", "r": 4096, "v": VOCAB, "k": 64, "dt": "bf16", "dirs": "both", "t": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "tree", "chain", "distill", "distill"])
    if op == "attn":
        c = {"op": op, "b": _log(rng, 1, 32), "n": _log(rng, 1, 64), "hq": 0, "hkv": rng.choice([1, 2, 4, 8, 16]),
             "d": rng.choice([64, 128, 128, 256]), "len": _log(rng, 1, 32768), "page": rng.choice([1, 16, 24, 32, 64, 100, 256]),
             "dt": rng.choice(["bf16", "f16"]), "heads_first": rng.random() < 0.5}
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 5, 6, 8, 12])
        while c["b"] * (c["len"] + c["n"]) * c["hkv"] * c["d"] > 1 << 28 or c["b"] * c["n"] * c["hq"] * c["d"] * c["len"] > 1 << 34:
            c["b"], c["len"] = max(1, c["b"] // 2), max(1, c["len"] * 3 // 4)
        return c
    if op == "append":
        return {"op": op, "b": _log(rng, 1, 64), "n": _log(rng, 1, 512), "hkv": rng.choice([1, 2, 4, 8, 16]),
                "d": rng.choice([64, 80, 128, 256]), "len": _log(rng, 1, 4096), "page": rng.choice([1, 16, 24, 64, 100, 256]),
                "dt": rng.choice(["bf16", "f16"]), "path": rng.random() < 0.5, "heads_first": rng.random() < 0.5}
    if op in ("tree", "chain"):
        return {"op": op, "b": _log(rng, 1, 24), "n": _log(rng, 2, 24), "v": _log(rng, 1000, 140000),
                "dt": rng.choice(["f32", "bf16", "f16"]), "hot": rng.random() < 0.5}
    v = _log(rng, 1000, 140000)
    return {"op": op, "r": _log(rng, 1, 2048), "v": v, "k": _log(rng, 1, 200), "dt": rng.choice(["f32", "bf16", "f16"]),
            "dirs": rng.choice(["both", "apart", "loss"]), "t": rng.choice([1.0, 0.7, 2.0])}


def _lengths(case):
    """Tokens in the cache per sequence: the first has them all, the others from a quarter up."""
    r = random.Random(case["len"] * 64 + case["b"])
    full = case["len"]
    if full >= 8192:  # long contexts: all near the full length
        return [full - r.randrange(1 + full // 64) * (b > 0) for b in range(case["b"])]
    return [full if b == 0 else r.randint((full + 3) // 4, full) for b in range(case["b"])]


def _esize(case):
    return 4 if case["dt"] == "f32" else 2


def work(case):
    e = _esize(case)
    if case["op"] == "attn":
        tokens = sum(_lengths(case)) + case["b"] * case["n"]
        rows = case["b"] * case["n"] * case["hq"]
        seen = sum(n * case["n"] for n in _lengths(case)) + case["b"] * case["n"] * (case["n"] + 1) // 2
        return {"bytes": (tokens * case["hkv"] * 2 + rows * 2) * case["d"] * e, "flops": 4 * seen * case["hq"] * case["d"]}
    if case["op"] == "append":
        kept = case["b"] * case["n"] if not case["path"] else sum(_counts(case))
        return {"bytes": 4 * kept * case["hkv"] * case["d"] * e, "flops": 0}
    if case["op"] == "tree":
        return {"bytes": case["b"] * case["n"] * case["v"] * e, "flops": 0}
    if case["op"] == "chain":  # every row of logits, and the drafter's row where a draft was refused
        return {"bytes": case["b"] * case["v"] * (case["n"] * e + 4), "flops": 0}
    passes = {"loss": 1, "both": 2, "apart": 3}[case["dirs"]]
    return {"bytes": passes * case["r"] * case["v"] * e + case["r"] * case["k"] * (4 + e), "flops": 0}


def _counts(case):
    r = random.Random(case["b"] * 1000 + case["n"])
    return [r.randint(1, max(1, min(case["n"], 6))) for _ in range(case["b"])]


def _pages(case, room, g):
    """A cache with `room` positions a sequence in pages handed out in random order, and the table of them."""
    per = -(-(max(_lengths(case)) + room) // case["page"])
    pages = case["b"] * per + 3
    shape = (pages, case["hkv"], case["page"], case["d"]) if case["heads_first"] else (pages, case["page"], case["hkv"], case["d"])
    kc, vc = (torch.randn(shape, generator=g, device=DEV, dtype=DT[case["dt"]]) for _ in range(2))
    if case["heads_first"]:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    table = torch.randperm(pages, generator=g, device=DEV)[: case["b"] * per].view(case["b"], per).to(torch.int32)
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    return kc, vc, table, lengths


def _tree(b, n, g):
    """Parents of drafted trees: node 0 is the last token, every other node hangs on an earlier one."""
    i = torch.arange(n, device=DEV)
    back = (torch.rand((b, n), generator=g, device=DEV) * 6).long() + 1
    return torch.where(i > 0, (i - back).clamp(min=0), -1).to(torch.int32)


def _ancestors(parents):
    """[b, n, n] truth values: node j is node i or above it."""
    n = parents.shape[1]
    up = (parents[:, :, None] == torch.arange(n, device=parents.device)).double()
    return torch.linalg.matrix_power(up + torch.eye(n, device=parents.device, dtype=torch.float64), n) > 0


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    dt = DT[case["dt"]]
    if case["op"] == "attn":
        b, n, d = case["b"], case["n"], case["d"]
        heads = case["hq"] + 2 * case["hkv"]
        qkv = torch.randn((b, n, heads, d), generator=g, device=DEV, dtype=dt)  # the fused projection's rows
        s["q"], s["k"], s["v"] = qkv.split([case["hq"], case["hkv"], case["hkv"]], dim=2)
        s["kc"], s["vc"], s["table"], s["lengths"] = _pages(case, n, g)
        s["parents"] = _tree(b, n, g)
        bit = torch.ones((), dtype=torch.int64, device=DEV) << torch.arange(n, device=DEV)
        s["mask"] = (_ancestors(s["parents"]) * bit).sum(-1)
    elif case["op"] == "append":
        b, n = case["b"], case["n"]
        kv = torch.randn((b, n, 2, case["hkv"], case["d"]), generator=g, device=DEV, dtype=dt)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        s["kc"], s["vc"], s["table"], s["lengths"] = _pages(case, n, g)
        if case["path"]:
            s["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=DEV)
            order = torch.rand((b, n), generator=g, device=DEV)
            order[:, 0] = -1.0
            kept = order.argsort(1)
            at = torch.arange(n, device=DEV)
            kept = torch.where(at < s["counts"][:, None], kept, n).sort(1).values
            s["nodes"] = torch.where(at < s["counts"][:, None], kept, -1).to(torch.int32)
    elif case["op"] in ("tree", "chain"):
        b, n, v = case["b"], case["n"], case["v"]
        logits = torch.randn((b, n, v), generator=g, device=DEV) * 2
        tops = torch.randint(0, v, (b, n, 4), generator=g, device=DEV)  # each row's likely tokens
        lift = torch.tensor([15.0, 14.0, 13.0, 12.5], device=DEV) + torch.randn((b, n, 4), generator=g, device=DEV)
        logits.scatter_(2, tops, lift)
        s["u"] = torch.rand((b, n), generator=g, device=DEV)
        s["temperature"] = None
        if case["hot"]:
            s["temperature"] = torch.tensor([[0.7, 1.0, 0.0, 1.3][i % 4] for i in range(b)], device=DEV)
        if case["op"] == "tree":
            s["parents"] = _tree(b, n, g)
            p = s["parents"].long().clamp(min=0)
            i = torch.arange(n, device=DEV)
            older = ((p[:, :, None] == p[:, None, :]) & (i > 0) & (i < i[:, None])).sum(-1)  # siblings before this node
            s["tokens"] = tops.gather(1, p[:, :, None].expand(-1, -1, 4)).gather(2, (older % 4)[:, :, None])[:, :, 0].to(torch.int32)
        else:
            near = logits[:, :-1] + 0.5 * torch.randn((b, n - 1, v), generator=g, device=DEV)
            s["q"] = torch.softmax(near, -1)
            del near
            noise = torch.empty((b, n - 1, v), device=DEV).exponential_(generator=g)
            s["tokens"] = torch.zeros((b, n), dtype=torch.int32, device=DEV)
            s["tokens"][:, 1:] = (s["q"] / noise).argmax(-1)
            del noise
        s["logits"] = logits.to(dt)
    else:
        r, v, k = case["r"], case["v"], case["k"]
        x = torch.randn((r, v), generator=g, device=DEV)
        start = torch.randint(0, v, (r, 1), generator=g, device=DEV)
        step = torch.randint(1, max(2, v // k), (r, 1), generator=g, device=DEV)
        at = (start + step * torch.arange(k, device=DEV)) % v
        top = (torch.randn((r, k), generator=g, device=DEV) * 2 + 10).sort(1, descending=True).values
        x.scatter_(1, at, top + torch.randn((r, k), generator=g, device=DEV))
        few = torch.randint((k + 1) // 2, k + 1, (r, 1), generator=g, device=DEV)  # a teacher that kept fewer
        s["index"] = torch.where(torch.arange(k, device=DEV) < few, at, -1).to(torch.int32)
        s["top"] = top.to(dt)
        s["weight"] = (torch.rand((r,), generator=g, device=DEV) > 0.1) / r  # prompt tokens carry no loss
        if case["dt"] == "f16":
            s["weight"] *= 65536.0  # the loss scale that keeps half-precision gradients out of the subnormals
        s["logits"] = x.to(dt)
    return s


# ---------------------------------------------------------------- plain forms


def _gather(cache, table, lengths):
    """[b, hkv, positions, d] fp32 rows of the cache by position, and which of them are there."""
    page = cache.shape[1]
    rows = cache[table.long().clamp(min=0)].flatten(1, 2)
    there = torch.arange(table.shape[1] * page, device=cache.device) < lengths[:, None]
    return torch.where(there[:, :, None, None], rows, 0).float().transpose(1, 2), there


def _attn(s):
    b, n, hq, d = s["q"].shape
    hkv = s["k"].shape[2]
    kc, there = _gather(s["kc"], s["table"], s["lengths"])
    vc, _ = _gather(s["vc"], s["table"], s["lengths"])
    k = torch.cat([kc, s["k"].float().transpose(1, 2)], 2)
    v = torch.cat([vc, s["v"].float().transpose(1, 2)], 2)
    q = s["q"].float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    seen = ((s["mask"][:, :, None] >> torch.arange(n, device=DEV)) & 1).bool()
    seen = torch.cat([there[:, None].expand(b, n, -1), seen], 2)[:, None, :, None]
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * d ** -0.5
    x = x.view(b, hkv, n, hq // hkv, -1).masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top.isinf(), 0, top))
    z = e.sum(-1, keepdim=True)
    o = torch.matmul((e / torch.where(z == 0, 1, z)).view(b, hkv, -1, k.shape[2]), v.contiguous())
    return o.view(b, hkv, n, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d).to(s["q"].dtype)


def _append(s):
    b, n = s["k"].shape[:2]
    page = s["kc"].shape[1]
    node = s["nodes"].long() if s["path"] else torch.arange(n, device=DEV).expand(b, n)
    count = s["counts"] if s["path"] else torch.full((b,), n, device=DEV)
    at = torch.arange(n, device=DEV)
    kept = at < count[:, None]
    pos = (s["lengths"][:, None].long() + at)[kept]
    seq = torch.arange(b, device=DEV)[:, None].expand(b, n)[kept]
    to = s["table"].long()[seq, pos // page], pos % page
    s["kc"][to] = s["k"][seq, node[kept]]
    s["vc"][to] = s["v"][seq, node[kept]]
    return s["kc"], s["vc"]


def _weights(logits, temperature):
    """Softmax weights in 64 bits, not yet divided by their sum; at temperature 0 the largest logit's first place."""
    x = logits.double()
    top = x.amax(-1, keepdim=True)
    if temperature is None:
        return torch.exp(x - top)
    t = temperature.double()[:, None, None]
    return torch.where(t > 0, torch.exp((x - top) / torch.where(t > 0, t, 1)), ((x == top).cumsum(-1) == 1) & (x == top))


def _sample(w, u):
    """The first place whose running sum of weights is over u times their sum."""
    c = w.cumsum(-1)
    return (c <= u.double()[..., None] * c[..., -1:]).sum(-1).clamp(max=w.shape[-1] - 1)


def _verify_tree(s):
    b, n, v = s["logits"].shape
    i = torch.arange(n, device=DEV)
    t = _sample(_weights(s["logits"], s["temperature"]), s["u"])
    p = s["parents"].long()
    hit = s["tokens"] == t.gather(1, p.clamp(min=0))
    twin = (p[:, :, None] == p[:, None, :]) & (s["tokens"][:, :, None] == s["tokens"][:, None, :]) & (i < i[:, None])
    hit = (hit & ~twin.any(-1)) | (i == 0)
    kept = ~(_ancestors(s["parents"]) & ~hit[:, None, :]).any(-1)
    count = kept.sum(-1)
    nodes = torch.where(kept, i, n).sort(1).values
    last = nodes.gather(1, count[:, None] - 1)
    nodes = torch.where(i < count[:, None], nodes, -1)
    return nodes.to(torch.int32), count.to(torch.int32), t.gather(1, last)[:, 0].to(torch.int32)


def _verify_chain(s):
    b, n, v = s["logits"].shape
    w = _weights(s["logits"], s["temperature"])
    p = w / w.sum(-1, keepdim=True)
    del w
    x = s["tokens"][:, 1:, None].long()
    ok = s["u"][:, :-1].double() * s["q"].gather(2, x)[..., 0].double() < p[:, :-1].gather(2, x)[..., 0]
    count = 1 + ok.long().cumprod(1).sum(1)
    seq = torch.arange(b, device=DEV)
    q = s["q"][seq, (count - 1).clamp(max=n - 2)].double() * (count < n)[:, None]
    p = p[seq, count - 1]
    rest = (p - q).clamp(min=0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p)
    return count.to(torch.int32), _sample(rest, s["u"][:, -1]).to(torch.int32)


def _distill(s):
    x = s["logits"].float() / s["t"]
    top = x.amax(-1, keepdim=True)
    x = x - top
    lse = torch.exp(x).sum(-1, keepdim=True).log()
    there = s["index"] >= 0
    at = s["index"].long().clamp(min=0)
    y = (s["top"].float() / s["t"]).masked_fill(~there, -math.inf)
    y = y - y.amax(-1, keepdim=True)
    y = y - torch.exp(y).sum(-1, keepdim=True).log()
    t = torch.exp(y)
    loss = torch.where(t > 0, t * (y - (x.gather(1, at) - lse)), 0).sum(-1)
    if s["dirs"] == "loss":
        return loss
    grad = torch.exp(x - lse).scatter_add_(1, at, -t)
    return loss, (grad * (s["weight"] / s["t"])[:, None]).to(s["logits"].dtype)


def run(s):
    if not own:
        return {"attn": _attn, "append": _append, "tree": _verify_tree, "chain": _verify_chain, "distill": _distill}[s["op"]](s)
    import trellis_quantized_linear_tf_amd as tq

    if s["op"] == "attn":
        return tq.tree_attention(s["q"], s["k"], s["v"], s["mask"], s["kc"], s["vc"], s["table"], s["lengths"])
    if s["op"] == "append":
        tq.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lengths"], s.get("nodes"), s.get("counts"))
        return s["kc"], s["vc"]
    if s["op"] == "tree":
        return tq.verify_tree(s["logits"], s["tokens"], s["parents"], s["u"], s["temperature"])
    if s["op"] == "chain":
        return tq.verify_chain(s["logits"], s["tokens"], s["q"], s["u"], s["temperature"])
    if s["dirs"] == "loss":
        return tq.distill_loss(s["logits"], s["index"], s["top"], temperature=s["t"])
    if s["dirs"] == "both":
        return tq.distill(s["logits"], s["index"], s["top"], s["weight"], temperature=s["t"])
    loss = tq.distill_loss(s["logits"], s["index"], s["top"], temperature=s["t"])
    return loss, tq.distill_grad(s["logits"], s["index"], s["top"], s["weight"], temperature=s["t"])


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "distill":
        return _exact_distill(s)
    return None  # the verifications answer whole numbers


def _exact_attn(s):
    b, n, hq, d = s["q"].shape
    hkv, page = s["k"].shape[2], s["kc"].shape[1]
    o = torch.zeros((b, n, hq, d), dtype=torch.float64, device=DEV)
    for i, length in enumerate(s["lengths"].tolist()):
        pos = torch.arange(length, device=DEV)
        at = s["table"][i, pos // page].long(), pos % page
        k = torch.cat([s["kc"][at], s["k"][i]]).double()
        v = torch.cat([s["vc"][at], s["v"][i]]).double()
        seen = torch.ones((n, length + n), dtype=torch.bool, device=DEV)
        parents = s["parents"][i].tolist()
        for node in range(n):
            seen[node, length:] = False
            up = node
            while up >= 0:
                seen[node, length + up] = True
                up = parents[up]
        for h in range(hkv):
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                x = torch.mm(s["q"][i, :, j].double(), k[:, h].t().contiguous()) / math.sqrt(d)
                x[~seen] = -math.inf
                o[i, :, j] = torch.mm(torch.softmax(x, 1), v[:, h].contiguous())
    return o


def _exact_append(s):
    b, n = s["k"].shape[:2]
    page = s["kc"].shape[1]
    kc, vc = s["kc"].double(), s["vc"].double()
    for i in range(b):
        count = int(s["counts"][i]) if s["path"] else n
        node = s["nodes"][i, :count].long() if s["path"] else torch.arange(n, device=DEV)
        pos = int(s["lengths"][i]) + torch.arange(count, device=DEV)
        to = s["table"][i, pos // page].long(), pos % page
        kc[to] = s["k"][i, node].double()
        vc[to] = s["v"][i, node].double()
    return kc, vc


def _exact_distill(s):
    losses, grads = [], []
    for r0 in range(0, s["r"], 256):
        rows = slice(r0, r0 + 256)
        x = s["logits"][rows].double() / s["t"]
        lp = torch.log_softmax(x, 1)
        there = s["index"][rows] >= 0
        at = s["index"][rows].long().clamp(min=0)
        t = torch.softmax((s["top"][rows].double() / s["t"]).masked_fill(~there, -math.inf), 1)
        losses.append((torch.special.xlogy(t, t) - t * lp.gather(1, at)).sum(1))
        if s["dirs"] != "loss":
            g = (lp.exp() - torch.zeros_like(lp).scatter_add(1, at, t)) * (s["weight"][rows].double() / s["t"])[:, None]
            grads.append(g.to(torch.float32) if s["r"] * s["v"] > 1 << 28 else g)
    return torch.cat(losses) if s["dirs"] == "loss" else (torch.cat(losses), torch.cat(grads))
