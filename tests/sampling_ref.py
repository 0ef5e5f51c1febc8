"""Plain 64-bit forms of the operators for sampled serving (numpy), for their tests: attention
of groups that share a prefix, verification by rejection sampling, normed rotary append."""
import numpy as np

from tests import cache_ops_ref as ref


def shared_lengths(B, T, cap, first, prefix, starts, counts):
    """(group's first sequence or -1, shared slots) of each sequence."""
    begins, last = [], 0
    for f in first:
        last = max(last, ref.clamp(f, B))
        begins.append(last)
    count = [T if counts is None else ref.clamp(counts[b], T) for b in range(B)]
    start = [ref.clamp(starts[b], cap) for b in range(B)]
    leader, shared = [-1] * B, [0] * B
    for j, f in enumerate(begins):
        end = begins[j + 1] if j + 1 < len(begins) else B
        live = [start[b] for b in range(f, end) if count[b] > 0]
        n = min([max(0, int(prefix[j]))] + live) if live else 0
        for b in range(f, end):
            leader[b], shared[b] = f, n
    return leader, shared


def prefix_attention(q, kpool, vpool, table, first, prefix, starts, parents, counts, scale):
    """ref.attention over rows put together slot by slot: the group's first sequence's
    below the shared length, the sequence's own behind it."""
    B, T = q.shape[:2]
    nkv, bs, d = kpool.shape[1:]
    cap = bs if table is None else table.shape[1] * bs
    leader, shared = shared_lengths(B, T, cap, first, prefix, starts, counts)
    slots, k, v = np.full((B, cap), -1), [], []
    for b in range(B):
        for s in range(cap):
            owner = leader[b] if s < shared[b] else b
            blk, row = (owner, s) if table is None else (int(table[owner, s // bs]), s % bs)
            if 0 <= blk < len(kpool):
                slots[b, s] = len(k)
                k.append(kpool[blk, :, row])
                v.append(vpool[blk, :, row])
    pools = [np.array(x).reshape(-1, nkv, 1, d) for x in (k, v)]
    return ref.attention(q, *pools, slots, starts, parents, counts, scale)


def probabilities(row, temperature):
    """A row's softmax, or None where no logit is above -inf."""
    row = np.where(np.isnan(row), -np.inf, row)
    top = row.max()
    if top == -np.inf:
        return None
    p = np.zeros(len(row))
    if not temperature > 0:
        p[np.flatnonzero(row == top)[0]] = 1
        return p
    at = row > -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(row[at] == top, 0.0, (row[at] - top) / temperature)
    p[at] = np.exp(z)
    return p / p.sum()


def verify(logits, tokens, uniform, noise, parents, counts, draft, temperature):
    """(path, accepted, next, how close the closest comparison was: the difference over the sum
    of what was subtracted or compared, so that an error of e of each changes nothing below it).
    The residual is formed step by step, as the definition has it."""
    B, T, V = logits.shape
    path, accepted, last, near = np.full((B, T), -1), np.zeros(B, int), np.full(B, -1), np.full(B, np.inf)
    for b in range(B):
        n = T if counts is None else ref.clamp(counts[b], T)
        if n == 0:
            continue
        heat = 1.0 if temperature is None else float(temperature[b])
        cur, path[b, 0], accepted[b] = 0, 0, 1
        while True:
            p = probabilities(logits[b, cur], heat)
            if p is None:
                break
            q = None
            if draft is not None:
                q = np.where(draft[b, cur] > 0, draft[b, cur], 0.0)  # (NaN is not above 0)
            r, unsure, raw = p.copy(), p.copy(), p.copy()  # the residual; what its error is a part of; below 0 uncut
            kids = [t for t in range(cur + 1, n) if ref.parent_of(parents, b, t) == cur
                    and 0 <= tokens[b, t] < V]
            took = None
            for t in kids:
                x, u = tokens[b, t], float(uniform[b, t])
                u = min(u, 1.0) if u > 0 else 0.0
                chance = 1.0 if q is None else q[x]
                gap, size = abs(u * chance - r[x]), u * chance + unsure[x]
                if u * chance > 0 and size > 0:
                    near[b] = min(near[b], gap / size)
                if u * chance < r[x]:
                    took = t
                    break
                if q is None:
                    s, su = raw.copy(), unsure.copy()
                    s[x] = su[x] = 0
                else:
                    s, su = raw - q, unsure + q
                left = np.maximum(s, 0).sum()
                if left <= 0:
                    r = None
                    break
                raw, unsure = s / left, (su + np.abs(s) * su.sum() / left) / left
                r = np.maximum(raw, 0)
            if took is not None:
                cur = took
                path[b, accepted[b]] = cur
                accepted[b] += 1
                continue
            if r is None:
                r = raw = unsure = p
            e = np.clip(np.where(np.isnan(noise[b]), 0, noise[b]), 1e-30, 1e30)
            score, slack = r / e, unsure / e
            last[b] = int(np.flatnonzero(score == score.max())[0])
            i = last[b]
            rivals = (np.arange(V) != i) & (unsure > 0)
            if rivals.any():
                gap = (score[i] - raw / e) / (slack[i] + slack)
                near[b] = min(near[b], gap[rivals].min())
            break
    return path, accepted, last, near


def normed(x, w, eps):
    """x [..., D], each head over its root mean square, times w."""
    with np.errstate(invalid="ignore"):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
