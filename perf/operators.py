"""The operators over a KV cache, case by case: their inputs, one pass of each, and what a pass cannot do without.

Where ``own`` is false a pass runs in elementary torch operations (fp32, fp64 for angles); where it is true it makes the
calls of decode_megakernel_03_gb300.mk that a serving program makes.

  attend   attention of a tree of drafted tokens over the cached keys (single tokens are a tree of one)
  rope     rotary positions of new queries and keys, the new k/v rows appended to the cache
  accept   greedy acceptance of a drafted tree from the logits of its nodes
  keep     the accepted nodes' k/v rows moved behind the context, in every layer
  fork     sequences forked from others in a paged cache: page tables, and the partly filled pages copied before a write
  copy     pages of every layer copied to other pages
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def _shape(name):
    """(layers, query heads, kv heads, head dim, vocabulary) of the shapes that this repository runs."""
    return {"tiny": (2, 4, 2, 64, 4096), "1b": (16, 32, 8, 64, 128256), "8b": (32, 32, 8, 128, 128256)}[name]


def listed():
    return [
        # one new token of one sequence behind a short context: latency
        {"name": "attend-1b-token", "op": "attend", "shape": "1b", "batch": 1, "nodes": 1, "low": 512, "high": 512,
         "block": 0, "type": "bf16", "ragged": False},
        # a drafted tree of one sequence behind a long context, paged in small blocks
        {"name": "attend-1b-tree-8k", "op": "attend", "shape": "1b", "batch": 1, "nodes": 16, "low": 8192, "high": 8192,
         "block": 16, "type": "bf16", "ragged": False},
        # eight sequences of unlike lengths, odd trees, some smaller than the batch's largest
        {"name": "attend-1b-batch8", "op": "attend", "shape": "1b", "batch": 8, "nodes": 25, "low": 128, "high": 4096,
         "block": 16, "type": "bf16", "ragged": True},
        # fp32 activations, as the decode step keeps them, short drafts on a contiguous cache
        {"name": "attend-8b-fp32", "op": "attend", "shape": "8b", "batch": 4, "nodes": 6, "low": 2048, "high": 16384,
         "block": 0, "type": "fp32", "ragged": False},
        # the largest: eight long sequences, full trees
        {"name": "attend-8b-long", "op": "attend", "shape": "8b", "batch": 8, "nodes": 64, "low": 16384, "high": 32768,
         "block": 64, "type": "bf16", "ragged": False},
        # the drafted tree's new rows, before its attention
        {"name": "rope-1b-tree", "op": "rope", "shape": "1b", "batch": 8, "nodes": 25, "low": 128, "high": 4096,
         "block": 16, "type": "fp32", "tree": True, "interleaved": False, "part": 64, "scaling": "bands"},
        # prompts written into the cache, far positions
        {"name": "rope-8b-prompt", "op": "rope", "shape": "8b", "batch": 4, "nodes": 8192, "low": 1000, "high": 90000,
         "block": 64, "type": "bf16", "tree": False, "interleaved": True, "part": 64, "scaling": "yarn"},
        # one small tree's verification, and eight full ones
        {"name": "accept-1", "op": "accept", "shape": "1b", "batch": 1, "nodes": 16, "type": "fp32"},
        {"name": "accept-8", "op": "accept", "shape": "1b", "batch": 8, "nodes": 64, "type": "fp32"},
        # the accepted path's rows moved down, every layer
        {"name": "keep-1b", "op": "keep", "shape": "1b", "batch": 8, "nodes": 25, "low": 128, "high": 4096, "block": 16,
         "accepted": 6},
        # parallel samples of a few prompts: tables forked, last pages copied
        {"name": "fork-1b", "op": "fork", "shape": "1b", "batch": 4, "children": 16, "low": 128, "high": 4096, "block": 64},
        # a pool being tidied: whole pages moved in every layer
        {"name": "copy-8b", "op": "copy", "shape": "8b", "pages": 500, "block": 16},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rope", "rope", "accept", "keep", "fork", "copy"])
    shape = rng.choice(["tiny", "1b", "8b"])
    block = rng.choice([0, 16, 64, 5, 48])
    if op == "attend":
        batch, high = _log(rng, 1, 8), _log(rng, 1, 32768)
        return {"op": op, "shape": shape, "batch": batch, "nodes": _log(rng, 1, 64), "low": _log(rng, 1, high), "high": high,
                "block": block, "type": rng.choice(["bf16", "fp32"]), "ragged": rng.random() < 0.5}
    if op == "rope":
        tree = rng.random() < 0.5
        d = _shape(shape)[3]
        return {"op": op, "shape": shape, "batch": _log(rng, 1, 4 if not tree else 8),
                "nodes": _log(rng, 1, 64) if tree else _log(rng, 1, 8192), "low": 0, "high": _log(rng, 1, 90000),
                "block": block, "type": rng.choice(["bf16", "fp32"] if tree else ["bf16"]), "tree": tree,
                "interleaved": rng.random() < 0.5, "part": rng.choice([d, d // 2, d - 4]),
                "scaling": rng.choice(["none", "linear", "bands", "yarn"])}
    if op == "accept":
        return {"op": op, "shape": shape, "batch": _log(rng, 1, 8), "nodes": _log(rng, 1, 64),
                "type": rng.choice(["bf16", "fp32"])}
    if op == "keep":
        nodes = _log(rng, 2, 64)
        return {"op": op, "shape": shape, "batch": _log(rng, 1, 8), "nodes": nodes, "low": 1, "high": _log(rng, 1, 4096),
                "block": block, "accepted": _log(rng, 1, min(nodes, 12))}
    if op == "fork":
        return {"op": op, "shape": shape, "batch": _log(rng, 1, 4), "children": _log(rng, 1, 24), "low": 1,
                "high": _log(rng, 1, 4096), "block": block or 32}
    return {"op": op, "shape": shape, "pages": _log(rng, 1, 500), "block": rng.choice([16, 5, 8])}


# ---- inputs -----------------------------------------------------------------------------------------------------------------


def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _lengths(case):
    """Context lengths, the same for every seed (they decide the work): between low and high, the last sequence's high."""
    b, low, high = case["batch"], case["low"], case["high"]
    return [high if i == b - 1 else low + (high - low) * ((i * 5 + 2) % b) // b for i in range(b)]


def _counts(case):
    b, t = case["batch"], case["nodes"]
    return [t - (i * 7) % max(1, t // 2) for i in range(b)] if case.get("ragged") else [t] * b


def _type(case):
    return torch.float32 if case["type"] == "fp32" else torch.bfloat16


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _parents(batch, nodes, seed):
    """Drafted trees: node 0 is the last token itself, every other node hangs off one of the eight before it."""
    r = np.random.default_rng(seed)
    p = np.full((batch, nodes), -1, dtype=np.int32)
    for t in range(1, nodes):
        p[:, t] = r.integers(max(0, t - 8), t, batch)
    return torch.from_numpy(p).to(DEV)


def _paged(case, nkv, d, layers, room, gen, seed):
    """K and V [layers][blocks][nkv][block][d], and the device block table, shuffled (None: a contiguous cache)."""
    b, bs = case["batch"], case["block"]
    if bs:
        entries = -(-room // bs)
        n = b * entries + 3
        table = np.random.default_rng(seed + 1).permutation(n)[:b * entries].reshape(b, entries).astype(np.int32)
        table = torch.from_numpy(table).to(DEV)
    else:
        n, bs, table = b, room, None
    k, v = (_normal((layers, n, nkv, bs, d), torch.bfloat16, gen) for _ in range(2))
    return k, v, table


def _rope_of(case, d):
    return {"theta": 500000.0, "rotary_dim": case["part"], "interleaved": case["interleaved"], "scaling": case["scaling"],
            "factor": 1.0 if case["scaling"] == "none" else 8.0, "low": 1.0, "high": 4.0 if case["scaling"] == "bands" else 32.0,
            "original_length": 8192}


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    layers, nh, nkv, d, vocab = _shape(case["shape"])
    op, s = case["op"], {"case": case}
    if op in ("attend", "rope", "keep"):
        b, t = case["batch"], case["nodes"]
        starts = _lengths(case)
        k, v, table = _paged(case, nkv, d, layers if op == "keep" else 1, max(starts) + t, gen, seed)
        s |= {"k": k, "v": v, "table": table, "starts": _ints(starts), "longest": max(starts) + t}
        if own:
            from decode_megakernel_03_gb300 import mk
            s["cache"] = mk.Cache(list(k), list(v), table)
    if op == "attend":
        s |= {"q": _normal((b, t, nh, d), _type(case), gen), "parents": _parents(b, t, seed), "counts": _ints(_counts(case)),
              "out": torch.zeros((b, t, nh, d), dtype=_type(case), device=DEV)}
    elif op == "rope":
        # as a fused projection leaves them: q, k and v side by side in a token's row
        s["qkv"] = _normal((b, t, nh + 2 * nkv, d), _type(case), gen)
        s["parents"] = _parents(b, t, seed) if case["tree"] else None
        if own:
            s["rope"] = mk.Rope(d, **_rope_of(case, d))
    elif op == "accept":
        b, t = case["batch"], case["nodes"]
        s["parents"] = _parents(b, t, seed)
        s["tokens"] = torch.randint(0, vocab, (b, t), generator=gen, device=DEV).to(torch.int32)
        logits = _normal((b, t, vocab), torch.float32, gen)
        if t > 1:  # most nodes agree with one of their children
            at = s["parents"][:, 1:].long() * vocab + s["tokens"][:, 1:].long()
            lift = torch.where(torch.rand(at.shape, generator=gen, device=DEV) < 0.7,
                               20.0 + torch.arange(1, t, device=DEV, dtype=torch.float32), 0.0).expand(b, t - 1)
            logits.view(b, t * vocab).scatter_add_(1, at, lift.contiguous())
        s["logits"] = logits.to(_type(case))
    elif op == "keep":
        r = np.random.default_rng(seed + 2)
        path = np.full((b, t), -1, dtype=np.int32)
        for i, a in enumerate(_accepted(case)):
            path[i, 1:a] = 1 + np.sort(r.choice(t - 1, a - 1, replace=False))
            path[i, 0] = 0
        s |= {"path": torch.from_numpy(path).to(DEV), "accepted": _ints(_accepted(case))}
    elif op == "fork":
        b, c, bs = case["batch"], case["children"], case["block"]
        lens = _lengths(case)
        used = [-(-n // bs) for n in lens]
        entries = max(used) + 1
        n = sum(used) + c + 5
        s["k"], s["v"] = (_normal((layers, n, nkv, bs, d), torch.bfloat16, gen) for _ in range(2))
        s |= {"lengths": np.array(lens, dtype=np.int32), "entries": entries,
              "parent": np.random.default_rng(seed).integers(0, b, c).astype(np.int32),
              "child": np.arange(b, b + c, dtype=np.int32)}
        if own:
            from decode_megakernel_03_gb300 import mk
            s["cache"] = mk.Cache(list(s["k"]), list(s["v"]))
            s["pages"] = mk.Pages(n, bs, b + c, entries * bs)
            s["pages"].resize(list(range(b)), lens)
        else:
            table = np.full((b + c, entries), -1, dtype=np.int32)
            first = np.cumsum([0] + used)
            for i in range(b):
                table[i, :used[i]] = np.arange(first[i], first[i] + used[i])
            s["table"] = table
            s["held"] = np.arange(n) < first[-1]
    elif op == "copy":
        n, bs = case["pages"], case["block"]
        s["k"], s["v"] = (_normal((layers, 2 * n + 7, nkv, bs, d), torch.bfloat16, gen) for _ in range(2))
        order = np.random.default_rng(seed).permutation(2 * n + 7).astype(np.int32)
        s["copies"] = np.stack([order[:n], order[n:2 * n], np.full(n, bs)], 1).astype(np.int32)
        if own:
            from decode_megakernel_03_gb300 import mk
            s["cache"] = mk.Cache(list(s["k"]), list(s["v"]))
    return s


def _accepted(case):
    return [1 + (i * 5 + case["accepted"] - 1) % case["accepted"] for i in range(case["batch"])]


# ---- one pass ---------------------------------------------------------------------------------------------------------------


def _family(parents):
    """[b][t][a]: whether node a is node t or one of its ancestors."""
    t = parents.shape[1]
    i = torch.arange(t, device=parents.device)
    p = parents.long()
    step = (p[:, :, None] == i) & (i < i[:, None])
    m = (step | (i == i[:, None])).float()
    for _ in range(6):  # paths of up to 64 edges
        m = ((m @ m) > 0).float()
    return m > 0


def _where(s, slots):
    """Block and row of the slots [b][n] of each sequence."""
    bs = s["k"].shape[3]
    if s["table"] is None:
        return torch.arange(slots.shape[0], device=DEV)[:, None].expand_as(slots), slots
    return s["table"].long().gather(1, slots // bs), slots % bs


def _attend(s):
    q, starts, parents, counts = s["q"], s["starts"], s["parents"], s["counts"]
    b, t, nh, d = q.shape
    nkv, n = s["k"].shape[2], s["longest"]
    slots = torch.arange(n, device=DEV).expand(b, n)
    blk, row = _where(s, slots)
    kk = s["k"][0][blk, :, row].float().permute(0, 2, 3, 1)  # [b][nkv][d][n]
    vv = s["v"][0][blk, :, row].float().permute(0, 2, 1, 3)
    qq = q.float().view(b, t, nkv, nh // nkv, d).permute(0, 2, 3, 1, 4).reshape(b, nkv, -1, d)
    node = slots - starts[:, None]
    fam = _family(parents).gather(2, node.clamp(0, t - 1)[:, None, :].expand(b, t, n))
    seen = (node < 0)[:, None, :] | ((node < counts[:, None])[:, None, :] & fam)
    sc = (qq @ kk).view(b, nkv, nh // nkv, t, n) * (1.0 / math.sqrt(d))
    sc = torch.where(seen[:, None, None], sc, -math.inf)
    w = torch.exp(sc - sc.amax(-1, keepdim=True).clamp_min(-3e38))
    del sc
    total = w.sum(-1, keepdim=True)
    o = (w.view(b, nkv, -1, n) @ vv).view(b, nkv, nh // nkv, t, d) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, t, nh, d).to(q.dtype)
    live = torch.arange(t, device=DEV) < counts[:, None]
    return torch.where(live[:, :, None, None], o, s["out"])


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
    _, nh, nkv, _, _ = _shape(s["case"]["shape"])
    return s["qkv"].split([nh, nkv, nkv], 2)


def _rope(s):
    case = s["case"]
    q, k, v = _split(s)
    b, t, nh, d = q.shape
    depth = torch.arange(t, device=DEV).expand(b, t) if s["parents"] is None else _family(s["parents"]).sum(-1) - 1
    f, magnitude = _frequencies(_rope_of(case, d))
    angle = (s["starts"][:, None] + depth).double()[:, :, None, None] * torch.from_numpy(f).to(DEV)
    cos, sin = (torch.cos(angle) * magnitude).float(), (torch.sin(angle) * magnitude).float()
    blk, row = _where(s, s["starts"].long()[:, None] + torch.arange(t, device=DEV))
    s["k"][0][blk, :, row] = _turn(k.float(), cos, sin, case["interleaved"]).to(torch.bfloat16)
    s["v"][0][blk, :, row] = v.to(torch.bfloat16)
    return {"q": _turn(q.float(), cos, sin, case["interleaved"]).to(q.dtype), "k": s["k"], "v": s["v"]}


def _accept(s):
    logits, tokens, parents = s["logits"], s["tokens"], s["parents"]
    b, t, vocab = logits.shape
    top = logits.amax(-1, keepdim=True)
    at = torch.arange(vocab, device=DEV, dtype=torch.int32)
    choices = torch.where(logits == top, at, vocab).amin(-1)
    i = torch.arange(t, device=DEV)
    p = parents.long()
    fits = (p >= 0) & (p < i) & (tokens == choices.gather(1, p.clamp_min(0)))
    twin = (p[:, :, None] == p[:, None, :]) & (tokens[:, :, None] == tokens[:, None, :]) & (i < i[:, None])
    fits = (fits & ~twin.any(-1)) | (i == 0)
    kept = (~_family(parents) | fits[:, None, :]).all(-1)
    path = torch.where(kept, i, t).sort(-1).values
    accepted = kept.sum(-1)
    last = choices.gather(1, path.gather(1, accepted[:, None] - 1))[:, 0]
    path = torch.where(path < t, path, -1)
    return {"choices": choices, "path": path.to(torch.int32), "accepted": accepted.to(torch.int32), "next": last}


def _keep(s):
    t = s["path"].shape[1]
    i = torch.arange(t, device=DEV)
    path = torch.where(i < s["accepted"][:, None], s["path"], i)
    to = _where(s, s["starts"].long()[:, None] + i)
    of = _where(s, s["starts"].long()[:, None] + path)
    s["k"][:, to[0], :, to[1]] = s["k"][:, of[0], :, of[1]]
    s["v"][:, to[0], :, to[1]] = s["v"][:, of[0], :, of[1]]
    return {"k": s["k"], "v": s["v"]}


def _fork(s):
    """Each child takes its parent's pages; before it grows by a token a partly filled last page becomes its own copy, a
    full one is followed by a new page. The lowest free pages are taken, in the children's order."""
    bs = s["k"].shape[3]
    table, length = s["table"].copy(), s["lengths"][s["parent"]]
    new = np.flatnonzero(~s["held"])[:len(s["child"])]
    rows, at = length % bs, length // bs
    table[s["child"]] = table[s["parent"]]
    old = np.where(rows > 0, table[s["child"], at], 0)
    table[s["child"], at] = new
    old, new, rows = (torch.from_numpy(x.astype(np.int64)).to(DEV) for x in (old, new, rows))
    mine = (torch.arange(bs, device=DEV) < rows[:, None])[None, :, None, :, None]
    s["k"][:, new] = torch.where(mine, s["k"][:, old], s["k"][:, new])
    s["v"][:, new] = torch.where(mine, s["v"][:, old], s["v"][:, new])
    return {"table": table, "k": s["k"], "v": s["v"]}


def _copy(s):
    at = torch.from_numpy(s["copies"].astype(np.int64)).to(DEV)
    s["k"][:, at[:, 1]] = s["k"][:, at[:, 0]]
    s["v"][:, at[:, 1]] = s["v"][:, at[:, 0]]
    return {"k": s["k"], "v": s["v"]}


def _run_own(s):
    from decode_megakernel_03_gb300 import mk
    op = s["case"]["op"]
    if op == "attend":
        return mk.tree_attention(s["cache"], 0, s["q"], s["starts"], s["parents"], s["counts"], out=s["out"])
    if op == "rope":
        q, k, v = _split(s)
        return {"q": mk.rope_append(s["rope"], s["cache"], 0, q, k, v, s["starts"], s["parents"]), "k": s["k"], "v": s["v"]}
    if op == "accept":
        choices, path, accepted, last = mk.tree_accept(s["logits"], s["tokens"], s["parents"])
        return {"choices": choices, "path": path, "accepted": accepted, "next": last}
    if op == "keep":
        mk.cache_compact(s["cache"], s["starts"], s["path"], s["accepted"])
        return {"k": s["k"], "v": s["v"]}
    if op == "fork":
        pages = s["pages"]
        pages.fork(s["parent"], s["child"])
        copies = pages.resize(s["child"], s["lengths"][s["parent"]] + 1)
        mk.cache_copy_blocks(s["cache"], copies)
        table = pages.table()
        pages.resize(s["child"], np.zeros_like(s["child"]))
        return {"table": table, "k": s["k"], "v": s["v"]}
    mk.cache_copy_blocks(s["cache"], s["copies"])
    return {"k": s["k"], "v": s["v"]}


def run(state):
    if own:
        return _run_own(state)
    return {"attend": _attend, "rope": _rope, "accept": _accept, "keep": _keep, "fork": _fork, "copy": _copy}[
        state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------------------------------------------


def work(case):
    layers, nh, nkv, d, vocab = _shape(case["shape"])
    op, b = case["op"], case.get("batch")
    size = 4 if case.get("type") == "fp32" else 2
    if op == "attend":
        pairs = list(zip(_lengths(case), _counts(case)))
        seen = sum(n + c for n, c in pairs)
        rows = sum(c for _, c in pairs)
        table = 4 * sum(-(-(n + c) // case["block"]) for n, c in pairs) if case["block"] else 0
        return {"bytes": seen * nkv * d * 4 + 2 * rows * nh * d * size + table, "flops": 4 * d * nh * sum(c * (n + c) for n, c in pairs)}
    if op == "rope":
        rows = b * case["nodes"]
        return {"bytes": rows * d * (2 * nh * size + 2 * nkv * size + 2 * nkv * 2), "flops": rows * 3 * case["part"] * (nh + nkv)}
    if op == "accept":
        return {"bytes": b * case["nodes"] * (vocab * size + 16), "flops": b * case["nodes"] * vocab}
    if op == "keep":
        return {"bytes": max(1, sum(_accepted(case)) - b) * layers * nkv * d * 2 * 2 * 2, "flops": 0}
    if op == "fork":
        bs = case["block"]
        r = sum(_lengths(case)[i] % bs for i in range(b)) / b  # rows of a copied page, over the parents
        return {"bytes": max(1.0, r * case["children"]) * layers * nkv * d * 2 * 2 * 2, "flops": 0}
    return {"bytes": case["pages"] * layers * nkv * case["block"] * d * 2 * 2 * 2, "flops": 0}


# ---- the definition, in 64 bits -----------------------------------------------------------------------------------------------


def exact(case, seed):
    """Written apart from the plain form: by sequence and by page, the masks by walking the parents."""
    s = prepare(case, seed)
    layers, nh, nkv, d, vocab = _shape(case["shape"])
    op = case["op"]
    parents = s["parents"].cpu().numpy() if s.get("parents") is not None else None

    def walk(b, t):
        seen = []
        while t >= 0:
            seen.append(t)
            t = int(parents[b][t])
        return seen

    def rows_of(pool, b, n):  # the first n cached rows of sequence b: [nkv][n][d]
        if s["table"] is None:
            return pool[b][:, :n]
        bs = pool.shape[2]
        return torch.cat([pool[i] for i in s["table"][b].tolist()[:-(-n // bs)]], 1)[:, :n]

    if op == "attend":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for b, (n, c) in enumerate(zip(_lengths(case), _counts(case))):
            hidden = torch.ones((c, c), dtype=torch.bool)
            for t in range(c):
                hidden[t, walk(b, t)] = False
            hidden = hidden.to(DEV)
            kk, vv = (rows_of(s[x][0], b, n + c).double() for x in "kv")
            for h in range(nh):
                sc = s["q"][b, :c, h].double() @ kk[h * nkv // nh].T / math.sqrt(d)
                sc[:, n:].masked_fill_(hidden, -math.inf)
                out[b, :c, h] = torch.softmax(sc, -1) @ vv[h * nkv // nh]
        return out
    if op == "rope":
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
        pos = np.array([[n + (i if parents is None else len(walk(j, i)) - 1) for i in range(t)]
                        for j, n in enumerate(_lengths(case))], dtype=wide)
        turns = np.mod(pos[:, :, None] * np.array(f, wide), two_pi)
        z = torch.from_numpy(turns.astype(np.float64)).to(DEV)
        z = torch.polar(torch.full_like(z, magnitude), z)[:, :, None]
        x = s["qkv"].double()
        left = range(0, 2 * half, 2) if r["interleaved"] else range(half)
        right = range(1, 2 * half, 2) if r["interleaved"] else range(half, 2 * half)
        left, right = torch.tensor(left, device=DEV), torch.tensor(right, device=DEV)
        w = torch.complex(x[..., left], x[..., right]) * z
        y = x.clone()
        y[..., left], y[..., right] = w.real, w.imag
        k, v = s["k"].double(), s["v"].double()
        for j, n in enumerate(_lengths(case)):
            slots = torch.arange(n, n + t, device=DEV)
            bs = k.shape[3]
            blk, row = (torch.full_like(slots, j), slots) if s["table"] is None else (s["table"][j].long()[slots // bs], slots % bs)
            k[0][blk, :, row], v[0][blk, :, row] = y[j, :, nh:nh + nkv], x[j, :, nh + nkv:]
        return {"q": y[:, :, :nh], "k": k, "v": v}
    return None
