"""Sampled serving over a KV cache, case by case: inputs, one pass of each operator, and what a pass cannot do without.

Where ``own`` is false a pass runs in elementary torch operations (fp32, fp64 for angles and where a token is decided); where
it is true it makes the calls of decode_megakernel_03_gb300.mk that a serving program makes.

  share   attention for a batch whose groups share a long prefix (samples of one prompt), single tokens or drafted trees
  verify  drafted nodes verified against the target's probabilities from given random numbers
  norm    queries and keys normalised for each head, rotated and appended to the cache in the same pass
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def _shape(name):
    """(query heads, kv heads, head dim, vocabulary) of the shapes that this repository runs."""
    return {"tiny": (4, 2, 64, 4096), "1b": (32, 8, 64, 128256), "8b": (32, 8, 128, 128256)}[name]


def listed():
    return [
        # four answers of a short prompt, a few tokens in: latency
        {"name": "share-1b-4", "op": "share", "shape": "1b", "groups": 1, "samples": 4, "nodes": 1, "prefix": 512, "low": 8,
         "high": 64, "block": 16, "type": "bf16", "ragged": False},
        # 32 answers of one prompt, one token each
        {"name": "share-8b-32", "op": "share", "shape": "8b", "groups": 1, "samples": 32, "nodes": 1, "prefix": 8192, "low": 16,
         "high": 512, "block": 16, "type": "bf16", "ragged": False},
        # three prompts of unlike lengths, up to eight answers each, odd drafted trees of unlike sizes
        {"name": "share-1b-drafts", "op": "share", "shape": "1b", "groups": 3, "samples": 8, "nodes": 9, "prefix": 2000,
         "low": 1, "high": 900, "block": 64, "type": "bf16", "ragged": True},
        # fp32 activations, as the decode step keeps them, short drafts on a contiguous cache
        {"name": "share-8b-fp32", "op": "share", "shape": "8b", "groups": 2, "samples": 12, "nodes": 4, "prefix": 4096,
         "low": 100, "high": 1000, "block": 0, "type": "fp32", "ragged": False},
        # the largest: two long documents, 32 answers each, short drafts
        {"name": "share-8b-long", "op": "share", "shape": "8b", "groups": 2, "samples": 32, "nodes": 4, "prefix": 32768,
         "low": 256, "high": 2048, "block": 64, "type": "bf16", "ragged": False},
        # one chain of four drafted tokens: latency
        {"name": "verify-1", "op": "verify", "shape": "1b", "batch": 1, "nodes": 5, "type": "fp32", "draft": "fp32",
         "tree": False, "accepted": 3, "temperature": False},
        # full trees of a drafter that proposes without probabilities
        {"name": "verify-8-trees", "op": "verify", "shape": "1b", "batch": 8, "nodes": 64, "type": "fp32", "draft": "none",
         "tree": True, "accepted": 6, "temperature": True},
        # odd trees sampled from a drafter's distributions, a rejected sibling before most accepted nodes
        {"name": "verify-8-sampled", "op": "verify", "shape": "1b", "batch": 8, "nodes": 25, "type": "bf16", "draft": "bf16",
         "tree": True, "accepted": 5, "temperature": True},
        # many sequences with short chains
        {"name": "verify-64", "op": "verify", "shape": "1b", "batch": 64, "nodes": 8, "type": "bf16", "draft": "fp32",
         "tree": False, "accepted": 7, "temperature": True},
        # new tokens of eight sequences in a decode step
        {"name": "norm-1b-step", "op": "norm", "shape": "1b", "batch": 8, "nodes": 1, "low": 128, "high": 4096, "block": 16,
         "type": "fp32", "tree": False, "interleaved": False, "part": 64, "scaling": "bands"},
        # the drafted trees' rows before their attention
        {"name": "norm-8b-trees", "op": "norm", "shape": "8b", "batch": 24, "nodes": 25, "low": 128, "high": 4096, "block": 64,
         "type": "bf16", "tree": True, "interleaved": False, "part": 128, "scaling": "none"},
        # prompts written into the cache, far positions
        {"name": "norm-8b-prompt", "op": "norm", "shape": "8b", "batch": 4, "nodes": 8192, "low": 1000, "high": 90000,
         "block": 64, "type": "bf16", "tree": False, "interleaved": False, "part": 128, "scaling": "yarn"},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _draw(rng):
    op = rng.choice(["share", "share", "share", "verify", "verify", "norm"])
    shape = rng.choice(["tiny", "1b", "8b"])
    block = rng.choice([0, 16, 64, 5, 48])
    kind = rng.choice(["bf16", "fp32"])
    if op == "share":
        high = _log(rng, 1, 2048)
        return {"op": op, "shape": shape, "groups": rng.randint(1, 4), "samples": _log(rng, 1, 48), "nodes": _log(rng, 1, 24),
                "prefix": _log(rng, 1, 32768 if block else 4096), "low": _log(rng, 1, high), "high": high, "block": block,
                "type": kind, "ragged": rng.random() < 0.5}
    if op == "verify":
        nodes, tree = _log(rng, 1, 64), rng.random() < 0.6
        return {"op": op, "shape": shape, "batch": _log(rng, 1, 64), "nodes": nodes, "type": kind,
                "draft": rng.choice(["none", "fp32", "bf16"]), "tree": tree, "accepted": _log(rng, 1, min(nodes, 9)),
                "temperature": rng.random() < 0.7}
    tree = rng.random() < 0.5
    d = _shape(shape)[2]
    return {"op": op, "shape": shape, "batch": _log(rng, 1, 24 if tree else 4), "nodes": _log(rng, 1, 64 if tree else 8192),
            "low": 0, "high": _log(rng, 1, 90000), "block": block, "type": kind if tree else "bf16", "tree": tree,
            "interleaved": rng.random() < 0.5, "part": rng.choice([d, d // 2, d - 4]),
            "scaling": rng.choice(["none", "linear", "bands", "yarn"])}


def draw(rng):
    """A case that costs no more than the largest listed one of its operator."""
    while True:
        case = _draw(rng)
        most = [work(c) for c in listed() if c["op"] == case["op"]]
        mine = work(case)
        rows = case["batch"] * case["nodes"] if case["op"] == "verify" else 0  # what making the inputs costs
        if mine["bytes"] <= max(m["bytes"] for m in most) and mine["flops"] <= max(m["flops"] for m in most) and rows <= 512:
            return case


# ---- inputs -----------------------------------------------------------------------------------------------------------------


def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _type(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _spread(n, low, high):
    """n lengths between low and high, the last one high, the same for every seed (they decide the work)."""
    return [high if i == n - 1 else low + (high - low) * ((i * 5 + 2) % n) // n for i in range(n)]


def _groups(case):
    """Sequences of each group, and the prefix of each."""
    n, s, p = case["groups"], case["samples"], case["prefix"]
    return [max(1, s - 3 * i % max(1, s // 2)) for i in range(n)], [max(1, p - i * p // 5) for i in range(n)]


def _share_lengths(case):
    """Prefix, tail and node count of each sequence."""
    sizes, prefixes = _groups(case)
    b, t = sum(sizes), case["nodes"]
    shared = [p for n, p in zip(sizes, prefixes) for _ in range(n)]
    counts = [t - (i * 7) % max(1, t // 2) for i in range(b)] if case["ragged"] else [t] * b
    return shared, _spread(b, case["low"], case["high"]), counts


def _parents(batch, nodes, seed):
    """Drafted trees: node 0 is the last token itself, every other node hangs off one of the eight before it."""
    r = np.random.default_rng(seed)
    p = np.full((batch, nodes), -1, dtype=np.int32)
    for t in range(1, nodes):
        p[:, t] = r.integers(max(0, t - 8), t, batch)
    return p


def _rope_of(case, d):
    return {"theta": 500000.0, "rotary_dim": case["part"], "interleaved": case["interleaved"], "scaling": case["scaling"],
            "factor": 1.0 if case["scaling"] == "none" else 8.0, "low": 1.0, "high": 4.0 if case["scaling"] == "bands" else 32.0,
            "original_length": 8192}


def _accepted(case):
    """Nodes that each sequence's verification goes through, node 0 among them (by the way the inputs are made)."""
    a = case["accepted"]
    return [1 + (i * 5 + a - 1) % a for i in range(case["batch"])]


EPS = 1e-6


def _prepare_share(case, seed, gen):
    nh, nkv, d, _ = _shape(case["shape"])
    sizes, prefixes = _groups(case)
    shared, tails, counts = _share_lengths(case)
    b, t, bs = len(tails), case["nodes"], case["block"]
    starts = [p + n for p, n in zip(shared, tails)]
    room = max(starts) + t
    first = [sum(sizes[:i]) for i in range(len(sizes))]
    if bs:
        # the full pages of a prefix are held by the whole group, its partly filled last page was copied for each
        entries = -(-room // bs)
        table, n = np.full((b, entries), -1, np.int64), 0
        for f, s, p in zip(first, sizes, prefixes):
            full = p // bs
            table[f:f + s, :full] = np.arange(n, n + full)
            n += full
            for i in range(f, f + s):
                more = -(-(starts[i] + t) // bs) - full
                table[i, full:full + more] = np.arange(n, n + more)
                n += more
        order = np.random.default_rng(seed + 1).permutation(n + 3)
        table = torch.from_numpy(np.where(table >= 0, order[table.clip(0)], -1).astype(np.int32)).to(DEV)
        blocks = n + 3
    else:
        blocks, bs, table = b, room, None
    k, v = (_normal((1, blocks, nkv, bs, d), torch.bfloat16, gen) for _ in range(2))
    if table is not None:
        for f, s, p in zip(first, sizes, prefixes):
            if p % bs:
                page = table[f:f + s, p // bs].long()
                for pool in (k, v):
                    pool[0, page[1:], :, :p % bs] = pool[0, page[:1], :, :p % bs]
    s = {"k": k, "v": v, "table": table, "starts": _ints(starts), "first": _ints(first), "prefix": _ints(prefixes),
         "q": _normal((b, t, nh, d), _type(case["type"]), gen), "parents": torch.from_numpy(_parents(b, t, seed)).to(DEV),
         "counts": _ints(counts), "out": torch.zeros((b, t, nh, d), dtype=_type(case["type"]), device=DEV)}
    if own:
        from decode_megakernel_03_gb300 import mk
        s["cache"] = mk.Cache(list(k), list(v), table)
    return s


def _prepare_verify(case, seed, gen):
    """The target's logits are the drafter's with some noise; a designed path of nodes is to the target's liking, the other
    nodes are not, so that what is accepted does not depend on the seed."""
    vocab, b, t = _shape(case["shape"])[3], case["batch"], case["nodes"]
    r = np.random.default_rng(seed)
    parents = _parents(b, t, seed) if case["tree"] else np.broadcast_to(np.arange(-1, t - 1, dtype=np.int32), (b, t)).copy()
    on_path = np.zeros((b, t), bool)
    for i, a in enumerate(_accepted(case)):
        path = [0] + sorted(1 + r.choice(t - 1, a - 1, replace=False)) if case["tree"] and t > 1 else list(range(a))
        on_path[i, path] = True
        for j in range(1, a):
            parents[i, path[j]] = path[j - 1]
    par, good = torch.from_numpy(parents).to(DEV), torch.from_numpy(on_path).to(DEV)
    logits = torch.randn((b, t, vocab), generator=gen, device=DEV) * 3.0
    draft = torch.exp(logits - logits.amax(-1, keepdim=True))
    draft /= draft.sum(-1, keepdim=True)
    tokens = torch.randint(0, vocab, (b, t), generator=gen, device=DEV)
    for node in range(1, t):
        p = draft[torch.arange(b, device=DEV), par[:, node].long()]
        tokens[:, node] = (p / torch.empty_like(p).exponential_(generator=gen)).argmax(-1)
    if t > 1:
        # no other node has the token of its sibling on the path
        same = (par[:, :, None] == par[:, None, :]) & (tokens[:, :, None] == tokens[:, None, :]) & good[:, None, :]
        tokens = torch.where(same.any(-1) & ~good, (tokens + 1) % vocab, tokens)
        logits += 0.5 * torch.randn((b, t, vocab), generator=gen, device=DEV)
        at = (par[:, 1:].long() * vocab + tokens[:, 1:])
        flat, kept = logits.view(b, t * vocab), good[:, 1:]
        plain = flat.gather(1, at)
        # (several nodes may name the same place: lowered first, then the path's lifted)
        flat.scatter_(1, at, plain - 20.0)
        rows = torch.arange(b, device=DEV)[:, None].expand_as(at)
        flat[rows[kept], at[kept]] = plain[kept] + (25.0 if case["draft"] == "none" else 6.0)
    return {"logits": logits.to(_type(case["type"])), "tokens": tokens.to(torch.int32), "parents": par if case["tree"] else None,
            "draft": None if case["draft"] == "none" else draft.to(_type(case["draft"])),
            "temperature": torch.tensor([0.7 + 0.1 * (i % 6) for i in range(b)], device=DEV) if case["temperature"] else None,
            "uniform": torch.rand((b, t), generator=gen, device=DEV),
            "noise": torch.empty((b, vocab), device=DEV).exponential_(generator=gen)}


def _prepare_norm(case, seed, gen):
    nh, nkv, d, _ = _shape(case["shape"])
    b, t, bs = case["batch"], case["nodes"], case["block"]
    starts = _spread(b, case["low"], case["high"])
    room = max(starts) + t
    if bs:
        # pages for the rows that are written; what lies before them is not looked at
        entries = -(-room // bs)
        pages = [range(n // bs, -(-(n + t) // bs)) for n in starts]
        order = np.random.default_rng(seed + 1).permutation(sum(map(len, pages)) + 3).tolist()
        table = np.full((b, entries), -1, np.int32)
        blocks = len(order)
        for i, own_pages in enumerate(pages):
            table[i, list(own_pages)] = [order.pop() for _ in own_pages]
        table = torch.from_numpy(table).to(DEV)
    else:
        blocks, bs, table = b, room, None
    k, v = (_normal((1, blocks, nkv, bs, d), torch.bfloat16, gen) for _ in range(2))
    s = {"k": k, "v": v, "table": table, "starts": _ints(starts),
         # as a fused projection leaves them: q, k and v side by side in a token's row, heads of unlike sizes
         "qkv": (_normal((b, t, nh + 2 * nkv, d), torch.float32, gen)
                 * torch.exp(_normal((1, 1, nh + 2 * nkv, 1), torch.float32, gen))).to(_type(case["type"])),
         "q_norm": (1 + 0.3 * _normal((d,), torch.float32, gen)).to(torch.bfloat16),
         "k_norm": (1 + 0.3 * _normal((d,), torch.float32, gen)).to(torch.bfloat16),
         "parents": torch.from_numpy(_parents(b, t, seed)).to(DEV) if case["tree"] else None}
    if own:
        from decode_megakernel_03_gb300 import mk
        s["cache"] = mk.Cache(list(k), list(v), table)
        s["rope"] = mk.Rope(d, **_rope_of(case, d))
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    make = {"share": _prepare_share, "verify": _prepare_verify, "norm": _prepare_norm}[case["op"]]
    return {"case": case} | make(case, seed, gen)


# ---- one pass ---------------------------------------------------------------------------------------------------------------


def _family(parents):
    """[b][t][a]: whether node a is node t or one of its ancestors."""
    t = parents.shape[1]
    i = torch.arange(t, device=parents.device)
    p = parents.long()
    m = (((p[:, :, None] == i) & (i < i[:, None])) | (i == i[:, None])).float()
    for _ in range(6):  # paths of up to 64 edges
        m = ((m @ m) > 0).float()
    return m > 0


def _where(s, seqs, slots):
    """Block and row of the slots [b][n] of the sequences [b]."""
    bs = s["k"].shape[3]
    if s["table"] is None:
        return seqs[:, None].expand_as(slots), slots
    return s["table"].long()[seqs].gather(1, (slots // bs).clamp_max(s["table"].shape[1] - 1)), slots % bs


def _softmax_parts(q, k, v, seen, scale):
    """(sum of weights x v, sum of weights, maximum) of q [..][rows][d] over k, v [..][n][d]; seen: [..][rows][n] or None."""
    sc = (q @ k.transpose(-1, -2)) * scale
    if seen is not None:
        sc = torch.where(seen, sc, -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-3e38)
    w = torch.exp(sc - m)
    return w @ v, w.sum(-1, keepdim=True), m


def _share(s):
    q, starts, parents, counts = s["q"], s["starts"].long(), s["parents"], s["counts"]
    b, t, nh, d = q.shape
    nkv = s["k"].shape[2]
    g, scale = nh // nkv, 1.0 / math.sqrt(d)
    sizes, prefixes = _groups(s["case"])
    # each group's prefix, for the rows of all its sequences at once
    o1, l1, m1 = [], [], []
    f = 0
    for size, p in zip(sizes, prefixes):
        blk, row = _where(s, torch.tensor([f], device=DEV), torch.arange(p, device=DEV)[None])
        kk, vv = (s[x][0][blk[0], :, row[0]].float().transpose(0, 1) for x in "kv")  # [nkv][p][d]
        qq = q[f:f + size].float().view(size, t, nkv, g, d).permute(2, 0, 1, 3, 4).reshape(nkv, -1, d)
        for out, x in zip((o1, l1, m1), _softmax_parts(qq, kk, vv, None, scale)):
            out.append(x.view(nkv, size, t, g, -1).permute(1, 0, 2, 3, 4))
        f += size
    o1, l1, m1 = (torch.cat(x).reshape(b, nkv, t * g, -1) for x in (o1, l1, m1))
    # each sequence's own rows behind it
    shared, tails, _ = _share_lengths(s["case"])
    n = max(tails) + t
    slots = torch.tensor(shared, device=DEV)[:, None] + torch.arange(n, device=DEV)
    blk, row = _where(s, torch.arange(b, device=DEV), slots.clamp_max(max(a + c for a, c in zip(shared, tails)) + t - 1))
    kk, vv = (s[x][0][blk, :, row].float().transpose(1, 2) for x in "kv")  # [b][nkv][n][d]
    node = slots - starts[:, None]
    fam = _family(parents).gather(2, node.clamp(0, t - 1)[:, None, :].expand(b, t, n))
    seen = (node < 0)[:, None, :] | ((node < counts[:, None])[:, None, :] & fam)
    qq = q.float().view(b, t, nkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, nkv, t * g, d)
    o2, l2, m2 = _softmax_parts(qq, kk, vv, seen[:, None, :, None].expand(b, nkv, t, g, n).reshape(b, nkv, t * g, n), scale)
    m = torch.maximum(m1, m2)
    e1, e2 = torch.exp(m1 - m), torch.exp(m2 - m)
    o = (o1 * e1 + o2 * e2) / (l1 * e1 + l2 * e2)
    o = o.view(b, nkv, t, g, d).permute(0, 2, 1, 3, 4).reshape(b, t, nh, d).to(q.dtype)
    live = torch.arange(t, device=DEV) < counts[:, None]
    return torch.where(live[:, :, None, None], o, s["out"])


def _verify(s):
    """One look at the nodes in order is the whole walk: a node's children come after it, siblings in ascending order."""
    logits, tokens, draft = s["logits"], s["tokens"].long(), s["draft"]
    b, t, vocab = logits.shape
    every = torch.arange(b, device=DEV)
    parents = s["parents"].long() if s["parents"] is not None else torch.arange(-1, t - 1, device=DEV).expand(b, t)
    heat = s["temperature"].double() if s["temperature"] is not None else torch.ones(b, dtype=torch.float64, device=DEV)

    def target(cur):
        z = logits[every, cur].double() / heat[:, None]
        z = torch.exp(z - z.amax(-1, keepdim=True))
        return z / z.sum(-1, keepdim=True)

    cur = torch.zeros(b, dtype=torch.long, device=DEV)
    p = target(cur)
    rest = p                                      # what is left of the target's probabilities, and how much that is
    mass = torch.ones(b, dtype=torch.float64, device=DEV)
    taken = torch.zeros(b, dtype=torch.float64, device=DEV)
    path = [every * 0]
    for node in range(1, t):
        x = tokens[:, node]
        mine = parents[:, node] == cur
        q = draft[every, cur].double() if draft is not None else None
        chance = q[every, x] if draft is not None else 1.0
        yes = mine & (s["uniform"][:, node].double() * chance * mass < rest[every, x])
        no = mine & ~yes
        if draft is not None:
            more = torch.where(no, taken + mass, taken)
            left = (p - more[:, None] * q).clamp_min(0.0)
        else:
            more = taken
            left = torch.where(torch.arange(vocab, device=DEV) == x[:, None], 0.0, rest)
        rest = torch.where(no[:, None], left, rest)
        mass = torch.where(no, left.sum(-1), mass)
        taken = torch.where(yes, 0.0, more)
        cur = torch.where(yes, node, cur)
        p = torch.where(yes[:, None], target(cur), p)
        rest = torch.where(yes[:, None], p, rest)
        mass = torch.where(yes, 1.0, mass)
        path.append(torch.where(yes, node, t))
    path = torch.stack(path, 1)
    accepted = (path < t).sum(-1)
    path = path.sort(-1).values
    rest = torch.where((rest > 0).any(-1, keepdim=True), rest, p)
    score = rest / s["noise"].double()
    at = torch.arange(vocab, device=DEV)
    last = torch.where(score == score.amax(-1, keepdim=True), at, vocab).amin(-1)
    return {"path": torch.where(path < t, path, -1).to(torch.int32), "accepted": accepted.to(torch.int32),
            "next": last.to(torch.int32)}


def _frequencies(r):
    n, f = r["rotary_dim"], r["theta"] ** (-np.arange(0, r["rotary_dim"], 2) / r["rotary_dim"])
    if r["scaling"] == "linear":
        return f / r["factor"], 1.0
    if r["scaling"] == "bands":
        wave = 2 * np.pi / f
        mix = np.clip((r["original_length"] / wave - r["low"]) / (r["high"] - r["low"]), 0, 1)
        return (1 - mix) * f / r["factor"] + mix * f, 1.0
    if r["scaling"] == "yarn":
        dim = [n * math.log(r["original_length"] / (x * 2 * math.pi)) / (2 * math.log(r["theta"])) for x in (r["high"], r["low"])]
        lo, hi = max(0, math.floor(dim[0])), min(n - 1, math.ceil(dim[1]))
        ramp = np.clip((np.arange(n // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return f / r["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(r["factor"]) + 1.0
    return f, 1.0


def _turn(x, cos, sin, interleaved):
    """x [b][t][h][d] with the pairs of its first dims turned; cos, sin [b][t][1][pairs]."""
    n = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _split(s):
    nh, nkv, _, _ = _shape(s["case"]["shape"])
    return s["qkv"].split([nh, nkv, nkv], 2)


def _norm(s):
    case = s["case"]
    q, k, v = _split(s)
    b, t, nh, d = q.shape
    depth = torch.arange(t, device=DEV).expand(b, t) if s["parents"] is None else _family(s["parents"]).sum(-1) - 1
    f, magnitude = _frequencies(_rope_of(case, d))
    angle = (s["starts"][:, None] + depth).double()[:, :, None, None] * torch.from_numpy(f).to(DEV)
    cos, sin = (torch.cos(angle) * magnitude).float(), (torch.sin(angle) * magnitude).float()

    def normed(x, w):
        x = x.float()
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()

    blk, row = _where(s, torch.arange(b, device=DEV), s["starts"].long()[:, None] + torch.arange(t, device=DEV))
    s["k"][0][blk, :, row] = _turn(normed(k, s["k_norm"]), cos, sin, case["interleaved"]).to(torch.bfloat16)
    s["v"][0][blk, :, row] = v.to(torch.bfloat16)
    return {"q": _turn(normed(q, s["q_norm"]), cos, sin, case["interleaved"]).to(q.dtype), "k": s["k"], "v": s["v"]}


def _run_own(s):
    from decode_megakernel_03_gb300 import mk
    op = s["case"]["op"]
    if op == "share":
        return mk.prefix_attention(s["cache"], 0, s["q"], s["first"], s["prefix"], s["starts"], s["parents"], s["counts"],
                                   out=s["out"])
    if op == "verify":
        path, accepted, last = mk.tree_verify(s["logits"], s["tokens"], s["uniform"], s["noise"], s["parents"],
                                              draft=s["draft"], temperature=s["temperature"])
        return {"path": path, "accepted": accepted, "next": last}
    q, k, v = _split(s)
    q = mk.norm_rope_append(s["rope"], s["cache"], 0, q, k, v, s["q_norm"], s["k_norm"], s["starts"], s["parents"], eps=EPS)
    return {"q": q, "k": s["k"], "v": s["v"]}


def run(state):
    if own:
        return _run_own(state)
    return {"share": _share, "verify": _verify, "norm": _norm}[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------------------------------------------


def work(case):
    nh, nkv, d, vocab = _shape(case["shape"])
    op, size = case["op"], 4 if case["type"] == "fp32" else 2
    if op == "share":
        prefixes = _groups(case)[1]
        shared, tails, counts = _share_lengths(case)
        keys = sum(prefixes) + sum(n + c for n, c in zip(tails, counts))
        rows = sum(counts)
        bs = case["block"]
        table = 4 * sum(-(-(p + n + c) // bs) for p, n, c in zip(shared, tails, counts)) if bs else 0
        return {"bytes": keys * nkv * d * 4 + 2 * rows * nh * d * size + table,
                "flops": 4 * d * nh * sum(c * (p + n + c) for p, n, c in zip(shared, tails, counts))}
    if op == "verify":
        # the logits of the accepted nodes and the random numbers of the last draw; of the drafter's rows that of a chain's
        # last accepted node, whose child was rejected
        a = _accepted(case)
        rows = sum(a)
        drafts = sum(n < case["nodes"] for n in a) if case["draft"] != "none" and not case["tree"] else 0
        draft_size = 4 if case["draft"] == "fp32" else 2
        return {"bytes": vocab * (rows * size + 4 * case["batch"] + drafts * draft_size), "flops": 4 * vocab * rows}
    rows = case["batch"] * case["nodes"]
    return {"bytes": rows * d * (2 * nh * size + 2 * nkv * size + 2 * nkv * 2), "flops": rows * (nh + nkv) * (3 * case["part"] + 4 * d)}


# ---- the definition, in 64 bits -----------------------------------------------------------------------------------------------


def exact(case, seed):
    """Written apart from the plain form: by sequence and head, the masks by walking the parents, the rotation by complex
    numbers. The verification's outputs are whole numbers and have no such value."""
    if case["op"] == "verify":
        return None
    s = prepare(case, seed)
    nh, nkv, d, _ = _shape(case["shape"])
    parents = s["parents"].cpu().numpy() if s.get("parents") is not None else None

    def walk(b, t):
        seen = []
        while t >= 0:
            seen.append(t)
            t = int(parents[b][t])
        return seen

    if case["op"] == "share":
        def rows_of(pool, b, lo, hi):  # cached rows lo to hi of sequence b: [nkv][n][d]
            if s["table"] is None:
                return pool[b][:, lo:hi]
            bs = pool.shape[2]
            pages = s["table"][b].tolist()[lo // bs:-(-hi // bs)]
            return torch.cat([pool[i] for i in pages], 1)[:, lo % bs:lo % bs + hi - lo]

        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        shared, tails, counts = _share_lengths(case)
        leader, common = 0, None
        for b, (p, n, c) in enumerate(zip(shared, tails, counts)):
            if b in s["first"].tolist():
                leader = b
                common = [rows_of(s[x][0], leader, 0, p).double() for x in "kv"]
            kk, vv = (torch.cat([a, rows_of(s[x][0], b, p, p + n + c).double()], 1) for a, x in zip(common, "kv"))
            hidden = torch.ones((c, c), dtype=torch.bool)
            for t in range(c):
                hidden[t, walk(b, t)] = False
            hidden = hidden.to(DEV).repeat_interleave(nh // nkv, 0)
            q = s["q"][b, :c].double().view(c, nkv, nh // nkv, d).transpose(0, 1).reshape(nkv, -1, d)
            sc = torch.einsum("grd,gnd->grn", q, kk) / math.sqrt(d)
            sc[:, :, p + n:].masked_fill_(hidden, -math.inf)
            o = torch.einsum("grn,gnd->grd", torch.softmax(sc, -1), vv)
            out[b, :c] = o.view(nkv, c, nh // nkv, d).transpose(0, 1).reshape(c, nh, d)
        return out

    r = _rope_of(case, d)
    half = r["rotary_dim"] // 2
    wide = np.longdouble
    two_pi = 2 * wide("3.14159265358979323846264338327950288")
    f, magnitude = [], 1.0 + 0.1 * math.log(r["factor"]) if r["scaling"] == "yarn" else 1.0
    for i in range(half):
        base = np.exp(-np.log(wide(r["theta"])) * i / half)
        far = base / wide(r["factor"])
        turns = wide(r["original_length"]) * base / two_pi  # over the original length
        if r["scaling"] == "bands":
            base = far if turns < r["low"] else base if turns > r["high"] else (
                far + (base - far) * (turns - wide(r["low"])) / (wide(r["high"]) - wide(r["low"])))
        elif r["scaling"] == "yarn":
            edge = [half * np.log(wide(r["original_length"]) / (two_pi * x)) / np.log(wide(r["theta"])) for x in (r["high"], r["low"])]
            first, last = max(0, int(np.floor(edge[0]))), min(2 * half - 1, int(np.ceil(edge[1])))
            base = base if i <= first else far if i >= last else base + (far - base) * (i - first) / wide(last - first)
        elif r["scaling"] == "linear":
            base = far
        f.append(base)
    b, t = case["batch"], case["nodes"]
    starts = s["starts"].tolist()
    pos = np.array([[n + (i if parents is None else len(walk(j, i)) - 1) for i in range(t)] for j, n in enumerate(starts)], dtype=wide)
    z = torch.from_numpy(np.mod(pos[:, :, None] * np.array(f, wide), two_pi).astype(np.float64)).to(DEV)
    z = torch.polar(torch.full_like(z, magnitude), z)[:, :, None]
    y = s["qkv"].double()
    for lo, hi, w in ((0, nh, s["q_norm"]), (nh, nh + nkv, s["k_norm"])):
        part = y[:, :, lo:hi]
        y[:, :, lo:hi] = part * w.double() * torch.rsqrt(part.square().sum(-1, keepdim=True) / d + EPS)
    left = torch.tensor(range(0, 2 * half, 2) if r["interleaved"] else range(half), device=DEV)
    right = left + 1 if r["interleaved"] else left + half
    turned = torch.complex(y[:, :, :nh + nkv, left], y[:, :, :nh + nkv, right]) * z
    y[:, :, :nh + nkv, left], y[:, :, :nh + nkv, right] = turned.real, turned.imag
    k, v = s["k"].double(), s["v"].double()
    for j, n in enumerate(starts):
        slots = torch.arange(n, n + t, device=DEV)
        bs = k.shape[3]
        blk, row = (torch.full_like(slots, j), slots) if s["table"] is None else (s["table"][j].long()[slots // bs], slots % bs)
        k[0][blk, :, row], v[0][blk, :, row] = y[j, :, nh:nh + nkv], y[j, :, nh + nkv:]
    return {"q": y[:, :, :nh], "k": k, "v": v}
