"""Plain 64-bit forms of the operators over a KV cache (numpy), for their tests."""
import math

import numpy as np


def rows_of(pool, table, b, n):
    """[nkv][n][D] of the first n slots of sequence b, and which of them exist.
    pool [n_blocks][nkv][bs][D]; table None: contiguous."""
    n_blocks, nkv, bs, d = pool.shape
    out, there = np.zeros((nkv, n, d)), np.zeros(n, bool)
    for s in range(n):
        if table is None:
            blk, row = (b, s) if s < bs else (-1, 0)
        else:
            blk, row = (int(table[b, s // bs]), s % bs) if s // bs < table.shape[1] else (-1, 0)
        if 0 <= blk < n_blocks:
            out[:, s], there[s] = pool[blk, :, row], True
    return out, there


def parent_of(parents, b, t):
    p = t - 1 if parents is None else int(parents[b, t])
    return p if 0 <= p < t else -1


def family(parents, b, t):
    seen = []
    while t >= 0:
        seen.append(t)
        t = parent_of(parents, b, t)
    return seen


def clamp(v, hi):
    return max(0, min(int(v), hi))


def attention(q, kpool, vpool, table, starts, parents, counts, scale):
    """(out, a, e): the outputs; sum of weight x |v|; a bound of the scores' sum of
    |q| |k| x scale over the row's keys. q [B][T][nh][D]; rows behind counts NaN."""
    B, T, nh, d = q.shape
    nkv, bs = kpool.shape[1], kpool.shape[2]
    cap = bs if table is None else table.shape[1] * bs
    out, a, e = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        c = T if counts is None else clamp(counts[b], T)
        start = clamp(starts[b], cap)
        n = min(start + c, cap)
        k, there = rows_of(kpool, table, b, n)
        v, _ = rows_of(vpool, table, b, n)
        for t in range(c):
            seen = there.copy()
            seen[start:] = False
            for j in family(parents, b, t):
                if start + j < n:
                    seen[start + j] = there[start + j]
            at = np.flatnonzero(seen)
            for h in range(nh):
                g = h // (nh // nkv)
                if not len(at):
                    out[b, t, h] = 0
                    continue
                s = k[g, at] @ q[b, t, h] * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[b, t, h] = w @ v[g, at]
                a[b, t, h] = w @ np.abs(v[g, at])
                e[b, t, h] = (np.abs(k[g, at]) @ np.abs(q[b, t, h])).max() * scale
    return out, a, e


def frequencies(n, theta, scaling="none", factor=1.0, low=1.0, high=4.0, original_length=0):
    f = [theta ** (-2.0 * i / n) for i in range(n // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "bands":
        out = []
        for x in f:
            turns = original_length * x / (2 * math.pi)
            mix = min(1.0, max(0.0, (turns - low) / (high - low)))
            out.append((1 - mix) * x / factor + mix * x)
        return out, 1.0
    if scaling == "yarn":
        def pair(turns):
            return n * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(0, math.floor(pair(high))), min(n - 1, math.ceil(pair(low)))
        out = []
        for i, x in enumerate(f):
            ramp = min(1.0, max(0.0, (i - lo) / (hi - lo))) if hi > lo else float(i > lo)
            out.append(x * (1 - ramp) + x / factor * ramp)
        return out, 0.1 * math.log(factor) + 1
    return f, 1.0


def rotate(x, pos, f, magnitude, interleaved):
    """x [..., D] at one position."""
    y, n = x.copy(), len(f)
    for i, w in enumerate(f):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        c, s = math.cos(pos * w) * magnitude, math.sin(pos * w) * magnitude
        y[..., p], y[..., q] = x[..., p] * c - x[..., q] * s, x[..., p] * s + x[..., q] * c
    return y


def accept(logits, tokens, parents, counts):
    B, T, _ = logits.shape
    choices, path = np.full((B, T), -1), np.full((B, T), -1)
    taken, last = np.zeros(B, int), np.full(B, -1)
    for b in range(B):
        c = T if counts is None else clamp(counts[b], T)
        for t in range(c):
            row = np.where(np.isnan(logits[b, t]), -np.inf, logits[b, t])
            ok = ~np.isnan(logits[b, t])
            best = 0
            if ok.any():
                best = int(np.flatnonzero(ok & (row == row[ok].max()))[0])
            choices[b, t] = best
        if c == 0:
            continue
        cur, taken[b], path[b, 0] = 0, 1, 0
        while True:
            kids = [t for t in range(cur + 1, c) if parent_of(parents, b, t) == cur
                    and tokens[b, t] == choices[b, cur]]
            if not kids:
                break
            cur = kids[0]
            path[b, taken[b]] = cur
            taken[b] += 1
        last[b] = choices[b, cur]
    return choices, path, taken, last
