"""Operators over a KV cache on the GPU against their plain 64-bit forms
(tests/cache_ops_ref.py), at the sizes, masks and layouts where they can go
wrong."""
import itertools
import math

import numpy as np
import pytest
import torch

from decode_megakernel_03_gb300 import mk
from tests import cache_ops_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def dev():
    return torch.device("cuda")


def host(t):
    return t.detach().double().cpu().numpy()


def ints(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device=dev())


def make_parents(rng, B, T, kind="tree"):
    p = np.full((B, T), -1, np.int32)
    for t in range(1, T):
        if kind == "tree":
            p[:, t] = rng.integers(max(0, t - 5), t, B)
        elif kind == "odd":  # values that name no earlier node make roots
            p[:, t] = rng.integers(-3, t + 3, B)
    return p


def make_cache(rng, B, room, nkv, D, bs, layers=1, missing=0):
    """Lists of k and v pools with random contents, the table (numpy, or None)."""
    if bs:
        e = -(-room // bs)
        n = B * e + 2
        table = rng.permutation(n)[:B * e].reshape(B, e).astype(np.int32)
        for _ in range(missing):
            table[rng.integers(B), rng.integers(e)] = rng.choice([-1, n, 2**31 - 1, -2**31])
    else:
        n, bs, table = B, room, None
    g = torch.Generator(device=dev()).manual_seed(int(rng.integers(1 << 30)))
    k, v = ([torch.randn((n, nkv, bs, D), generator=g, device=dev()).to(BF16) for _ in range(layers)]
            for _ in range(2))
    return k, v, table


# ---- tree attention ------------------------------------------------------------------


def attention_bound(want, a, e, n_keys, d, dtype):
    """Error that the roundings allow. Scores: d products and adds in fp32 (2^-23
    each, as the matrix unit may truncate) of at most e in all, the scale and the
    exponential: weights off by twice that. Sums: one add per 16 keys and per
    join. bf16 calls: each weight rounded (2^-8), and the output (2^-8)."""
    f = a * (2 * (d + 8) * 2**-23 * np.maximum(e, 1) + (n_keys / 16 + 64) * 2**-23)
    return f + (2**-8 * (1.001 * a + np.abs(want)) if dtype == BF16 else 2**-24 * np.abs(want)) + 1e-30


def check_attention(rng, B, T, nh, nkv, D, dtype, bs, starts, counts=None, parents="tree", missing=0,
                    scale=None, room=None, strided=False, poison=False, ramp=0.0):
    starts = np.asarray(starts)
    room = room or int(max(starts)) + T
    k, v, table = make_cache(rng, B, room, nkv, D, bs, missing=missing)
    if ramp:  # keys of very unlike sizes: the running maximum moves often and far
        f = 1 + ramp * torch.rand(k[0].shape[:3], device=dev(), generator=torch.Generator(dev()).manual_seed(5))
        k[0] = (k[0].float() * f[..., None] ** 2).to(BF16)
    par = None if parents is None else make_parents(rng, B, T, parents)
    cap = table.shape[1] * bs if bs else room
    kp, vp = host(k[0]), host(v[0])
    if poison:
        # what no row may see is NaN or infinite: slots behind the length of each
        # sequence, and blocks that no table names
        mine = np.zeros(kp.shape[:1] + kp.shape[2:3], bool)
        for b in range(B):
            c = T if counts is None else ref.clamp(counts[b], T)
            for s in range(min(ref.clamp(starts[b], cap) + c, cap)):
                blk, row = (b, s) if table is None else (int(table[b, s // bs]), s % bs)
                if 0 <= blk < len(mine):
                    mine[blk, row] = True
        hide = torch.tensor(~mine, device=dev())[:, None, :, None].expand_as(k[0])
        k[0][hide], v[0][hide] = float("nan"), float("inf")
    g = torch.Generator(device=dev()).manual_seed(7)
    if strided:
        q = torch.randn((B, T, nh + 3, D), generator=g, device=dev()).to(dtype)[:, :, 1:nh + 1]
        out = torch.full((B, T, 2 * nh, D), 77.0, device=dev(), dtype=dtype)[:, :, nh:]
    else:
        q = torch.randn((B, T, nh, D), generator=g, device=dev()).to(dtype)
        out = torch.full((B, T, nh, D), 77.0, device=dev(), dtype=dtype)
    cache = mk.Cache(k, v, ints(table))
    got = mk.tree_attention(cache, 0, q, ints(starts), ints(par), ints(counts), scale=scale, out=out)
    want, a, e = ref.attention(host(q), kp, vp, table, starts, par, counts,
                               D ** -0.5 if scale is None else scale)
    got = host(got)
    live = ~np.isnan(want)
    assert (got[~live] == 77.0).all()
    assert np.isfinite(got).all()
    bound = attention_bound(want, a, e, cap, D, dtype)
    off = np.abs(got - want) / bound
    assert (off[live] <= 1).all(), f"{np.nanmax(off):.3g} of the bound"
    return q, cache, got


SHAPES = [(4, 2, 64), (8, 1, 64), (4, 4, 128), (12, 2, 128)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("nh,nkv,D", SHAPES)
@pytest.mark.parametrize("T", [1, 2, 5, 16, 33, 64])
def test_attention_trees(T, nh, nkv, D, dtype):
    rng = np.random.default_rng(T)
    check_attention(rng, 3, T, nh, nkv, D, dtype, 16, [0, 130, 61])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bs", [0, 1, 5, 48, 64, 256])
def test_attention_layouts(bs, dtype):
    rng = np.random.default_rng(bs)
    check_attention(rng, 4, 9, 4, 2, 64, dtype, bs, [300, 0, 17, 128], poison=True)


@pytest.mark.parametrize("start", [0, 1, 7, 55, 63, 64, 65, 127, 128, 500])
@pytest.mark.parametrize("T", [1, 9])
def test_attention_lengths(start, T):
    rng = np.random.default_rng(start)
    check_attention(rng, 1, T, 4, 1, 128, BF16, 16, [start], poison=True)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_long(D, dtype):
    rng = np.random.default_rng(D)
    check_attention(rng, 2, 3, 4, 2, D, dtype, 32, [20000, 3001], strided=True)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_attention_wide_trees_long(dtype):
    rng = np.random.default_rng(3)
    check_attention(rng, 2, 40, 16, 2, 128, dtype, 64, [2500, 90], counts=[40, 31], strided=True)


@pytest.mark.parametrize("parents", [None, "tree", "odd"])
@pytest.mark.parametrize("nh,nkv,D", [(4, 2, 64), (16, 2, 128)])
def test_attention_counts(parents, nh, nkv, D):
    """Smaller trees than the batch's largest, none at all, counts out of range;
    rows behind them are left as they were."""
    rng = np.random.default_rng(5)
    check_attention(rng, 6, 24, nh, nkv, D, BF16, 16, [40, 100, 9, 70, 64, 0],
                    counts=[24, 0, 1, -4, 99, 23], parents=parents, poison=True, strided=True)


def test_attention_no_sequence_at_all():
    rng = np.random.default_rng(5)
    check_attention(rng, 2, 4, 4, 2, 64, BF16, 16, [40, 100], counts=[0, -1])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [4, 40])
def test_attention_missing_pages(T, dtype):
    """Pages that are not there are not seen; starts behind the capacity and below
    0 are taken at the bound, and a row without any key is 0."""
    rng = np.random.default_rng(T)
    check_attention(rng, 5, T, 8, 2, 64, dtype, 8, [40, 3, 500, -6, 64], missing=12, room=64)
    k, v, _ = make_cache(rng, 1, 64, 2, 64, 8)
    none = torch.full((1, 8), -1, dtype=torch.int32, device=dev())
    q = torch.randn((1, T, 8, 64), device=dev()).to(dtype)
    out = mk.tree_attention(mk.Cache(k, v, none), 0, q, ints([30]))
    assert (out == 0).all()


@pytest.mark.parametrize("scale", [1e-6, 3.0])
def test_attention_scale(scale):
    rng = np.random.default_rng(1)
    check_attention(rng, 2, 6, 4, 2, 64, FP32, 16, [200, 30], scale=scale)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,nh,nkv", [(3, 4, 2), (20, 4, 2), (64, 8, 1)])
def test_attention_scores_of_all_sizes(T, nh, nkv, dtype):
    rng = np.random.default_rng(T)
    check_attention(rng, 2, T, nh, nkv, 64, dtype, 16, [900, 130], ramp=3.0)
    check_attention(rng, 2, T, nh, nkv, 128, dtype, 16, [900, 130], ramp=6.0, scale=0.7)


@pytest.mark.parametrize("T", [2, 30, 64])
def test_attention_in_place(T):
    """The output over the queries: every row of q is read before it is written."""
    rng = np.random.default_rng(T)
    k, v, table = make_cache(rng, 3, 400, 2, 64, 16)
    starts, cache = ints([300, 7, 90]), mk.Cache(k, v, ints(table))
    for dtype in (BF16, FP32):
        q = torch.randn((3, T, 16, 64), device=dev()).to(dtype)
        want = mk.tree_attention(cache, 0, q, starts)
        assert mk.tree_attention(cache, 0, q, starts, out=q) is q
        assert torch.equal(q, want)


def test_pools_of_more_than_2_to_the_31_elements():
    """Blocks whose offsets pass 32 bits: attention, append, rows moved, pages
    copied, against a small pool that holds the same pages."""
    nkv, bs, D, blocks = 8, 64, 128, 36000
    assert blocks * nkv * bs * D > 2**31
    big = [torch.empty((blocks, nkv, bs, D), dtype=BF16, device=dev()) for _ in range(2)]
    rng = np.random.default_rng(0)
    table = np.stack([rng.permutation(np.arange(blocks - 60, blocks))[:10],
                      rng.permutation(np.arange(33000, 33060))[:10]]).astype(np.int32)
    small_table = np.arange(20, dtype=np.int32).reshape(2, 10)
    at = torch.tensor(table.ravel(), device=dev(), dtype=torch.int64)
    small = [torch.randn((21, nkv, bs, D), device=dev()).to(BF16) for _ in range(2)]
    for b, s in zip(big, small):
        b[at] = s[:20]
    cb, cs = mk.Cache([big[0]], [big[1]], ints(table)), mk.Cache([small[0]], [small[1]], ints(small_table))
    starts, par = ints([500, 77]), ints(make_parents(rng, 2, 40))

    def same():
        assert all(torch.equal(b[at], s[:20]) for b, s in zip(big, small))

    for dtype, T in ((BF16, 2), (BF16, 40), (FP32, 2), (FP32, 40)):
        q = torch.randn((2, T, 16, D), device=dev()).to(dtype)
        kn, vn = (torch.randn((2, T, nkv, D), device=dev()).to(dtype) for _ in range(2))
        p = par[:, :T].contiguous()
        outs = [mk.tree_attention(c, 0, mk.rope_append(mk.Rope(D), c, 0, q, kn, vn, starts, p), starts, p)
                for c in (cb, cs)]
        assert torch.equal(*outs)
        same()
    path = ints([[0, 3, 7, 30] + [-1] * 36, [0, 1, 2, 39] + [-1] * 36])
    for c in (cb, cs):
        mk.cache_compact(c, starts, path, ints([4, 4]))
    same()
    mk.cache_copy_blocks(cb, [[int(table[0, 3]), 35999 if 35999 not in table else 32990, bs]])
    dst = 35999 if 35999 not in table else 32990
    assert torch.equal(big[0][dst], small[0][3]) and torch.equal(big[1][dst], small[1][3])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,G", [(6, 2), (50, 4)])
def test_attention_odd_values_stay_with_the_rows_that_see_them(T, G, dtype):
    """NaN and infinities in the k and v rows of a drafted node reach its
    descendants only; in a row's q they reach that row only."""
    rng = np.random.default_rng(2)
    B, nkv, D = 2, 2, 64
    k, v, table = make_cache(rng, B, 128 + T, nkv, D, 16)
    par = make_parents(rng, B, T)
    starts = [100, 61]
    q = torch.randn((B, T, nkv * G, D), device=dev()).to(dtype)
    cache = mk.Cache(k, v, ints(table))
    clean = mk.tree_attention(cache, 0, q, ints(starts), ints(par)).clone()
    spots = {0: [(2, "v", 5, float("inf")), (4, "v", 9, float("nan"))],
             1: [(3, "k", 0, float("nan")), (5, "v", 1, -float("inf"))]}
    hit = torch.zeros((B, T), dtype=torch.bool)
    for b, list_ in spots.items():
        for node, which, d, x in list_:
            s = starts[b] + node
            (k if which == "k" else v)[0][table[b, s // 16], :, s % 16, d] = x
            for t in range(T):
                hit[b, t] |= node in ref.family(par, b, t)
    got = mk.tree_attention(cache, 0, q, ints(starts), ints(par))
    assert torch.equal(got[~hit], clean[~hit])
    for b, list_ in spots.items():
        for node, which, d, x in list_:
            rows = [t for t in range(T) if node in ref.family(par, b, t)]
            assert rows
            r = got[b, rows]
            if which == "k":
                assert r.isnan().all()
            elif x != x:
                assert r[..., d].isnan().all()
            else:
                others = [n for n, w, dd, _ in list_ if (w == "k" or dd == d) and n != node]
                only = [i for i, t in enumerate(rows)
                        if not any(n in ref.family(par, b, t) for n in others)]
                assert (r[only][..., d] == x).all()
    q2 = q.clone()
    q2[0, 1, 0, 3] = float("nan")
    got2 = mk.tree_attention(cache, 0, q2, ints(starts), ints(par))
    assert got2[0, 1, 0].isnan().all()
    got2[0, 1, 0] = got[0, 1, 0]
    assert torch.equal(got2.nan_to_num(3.0), got.nan_to_num(3.0))


def test_attention_nan_keys_everywhere():
    """A row whose only key is NaN is NaN, not empty."""
    rng = np.random.default_rng(2)
    k, v, table = make_cache(rng, 1, 16, 1, 64, 16)
    k[0].fill_(float("nan"))
    for dtype, T in ((BF16, 1), (FP32, 1), (BF16, 64)):
        q = torch.randn((1, T, 4, 64), device=dev()).to(dtype)
        room = make_cache(rng, 1, 80, 1, 64, 16)
        room[0][0].fill_(float("nan"))
        got = mk.tree_attention(mk.Cache(room[0], room[1], ints(room[2])), 0, q, ints([0]))
        assert got.isnan().all()


@pytest.mark.parametrize("T,dtype", [(1, BF16), (7, FP32), (64, BF16)])
def test_attention_streams_graphs_and_repeats(T, dtype):
    """The same bits again: repeated, on another stream, captured and replayed
    (two graphs at once, each with its own workspace), after a longer call."""
    rng = np.random.default_rng(4)
    q, cache, _ = check_attention(rng, 3, T, 8, 2, 128, dtype, 16, [700, 20, 333])
    starts = ints([700, 20, 333])
    first = mk.tree_attention(cache, 0, q, starts)
    for _ in range(20):
        assert torch.equal(mk.tree_attention(cache, 0, q, starts), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = mk.tree_attention(cache, 0, q, starts, stream=side)
    side.synchronize()
    assert torch.equal(a, first)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mk.tree_attention(cache, 0, q, starts))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, first) for o in outs)
    # the lengths are read on the device: a replay follows them
    starts.copy_(torch.tensor([5, 90, 0], dtype=torch.int32))
    graphs[0].replay()
    assert torch.equal(outs[0], mk.tree_attention(cache, 0, q, starts))


def test_attention_many_sequences():
    rng = np.random.default_rng(8)
    B = 70
    starts = rng.integers(0, 60, B)
    check_attention(rng, B, 2, 4, 2, 64, BF16, 8, starts, counts=rng.integers(0, 3, B))


@pytest.mark.parametrize("T,nh,nkv,dtype", [(1, 2, 1, BF16), (9, 2, 1, BF16), (17, 2, 2, FP32)])
def test_attention_as_many_sequences_as_there_may_be(T, nh, nkv, dtype):
    """1024 sequences, of which some have no node, on both kernels."""
    rng = np.random.default_rng(T)
    check_attention(rng, 1024, T, nh, nkv, 64, dtype, 16, rng.integers(0, 40, 1024),
                    counts=rng.integers(0, T + 1, 1024))


# ---- rotary positions and append -------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D,part,interleaved", [(64, 64, False), (64, 32, False), (64, 60, False),
                                                (64, 2, True), (128, 128, False), (128, 96, True),
                                                (128, 124, False), (128, 64, True), (128, 16, False)])
@pytest.mark.parametrize("bs", [0, 5, 16])
def test_rope_append(D, part, interleaved, bs, dtype):
    rng = np.random.default_rng(part + bs)
    B, T, nh, nkv = 3, 11, 6, 3
    starts, counts = [40, 0, 3], [11, 4, 0]
    k, v, table = make_cache(rng, B, 60, nkv, D, bs, layers=2)
    par = make_parents(rng, B, T, "odd")
    qkv = torch.randn((B, T, nh + 2 * nkv, D), device=dev()).to(dtype)
    q, kn, vn = qkv.split([nh, nkv, nkv], 2)
    rope = mk.Rope(D, theta=10000.0, rotary_dim=part, interleaved=interleaved)
    f, m = ref.frequencies(part, 10000.0)
    before = [t.clone() for t in k + v]
    qh, kh, vh = host(q), host(kn), host(vn)
    out = torch.full((B, T, nh, D), 77.0, device=dev(), dtype=dtype)
    mk.rope_append(rope, mk.Cache(k, v, ints(table)), 1, q, kn, vn, ints(starts), ints(par),
                   ints(counts), q_out=out)
    assert torch.equal(k[0], before[0]) and torch.equal(v[0], before[2])  # the other layer
    kw, vw = host(before[1]), host(before[3])
    size = bs or 60
    far = 0.0
    for b in range(B):
        for t in range(T):
            if t >= counts[b]:
                assert (out[b, t] == 77.0).all()
                continue
            pos = starts[b] + len(ref.family(par, b, t)) - 1
            want = ref.rotate(qh[b, t], pos, f, m, interleaved)
            # sin and cos to 2^-22, two products and an add, the output's rounding
            near = np.abs(qh[b, t]).max() * 4 * 2**-22 + (2**-8 if dtype == BF16 else 2**-24) * np.abs(want)
            assert (np.abs(host(out[b, t]) - want) <= near).all()
            s = starts[b] + t
            blk = b if table is None else table[b, s // size]
            kw[blk, :, s % size] = ref.rotate(kh[b, t], pos, f, m, interleaved)
            vw[blk, :, s % size] = vh[b, t]
            far = max(far, np.abs(kh[b, t]).max())
    assert (np.abs(host(k[1]) - kw) <= far * 4 * 2**-22 + 2**-8 * np.abs(kw)).all()
    assert (np.abs(host(v[1]) - vw) <= 2**-8 * np.abs(vw)).all()


@pytest.mark.parametrize("scaling", ["none", "linear", "bands", "yarn"])
def test_rope_far_positions(scaling):
    """Angles of positions near 2^20 turn as in 64 bits."""
    kw = dict(theta=500000.0, scaling=scaling, factor=1.0 if scaling == "none" else 8.0, low=1.0,
              high=4.0, original_length=8192)
    D, bs, start = 64, 64, (1 << 20) + 12345
    pool = torch.zeros((2, 1, bs, D), dtype=BF16, device=dev())
    table = torch.full((1, (start + 64) // bs + 1), -1, dtype=torch.int32, device=dev())
    table[0, start // bs] = 1
    q = torch.randn((1, 2, 2, D), device=dev())
    kn = torch.randn((1, 2, 1, D), device=dev())
    got = host(mk.rope_append(mk.Rope(D, **kw), mk.Cache([pool], [pool.clone()], table), 0, q, kn, kn,
                              ints([start])))
    f, m = ref.frequencies(D, **kw)
    for t in range(2):
        want = ref.rotate(host(q[0, t]), start + t, f, m, False)
        # the reference's own angle is off by 2^-53 x 2^20
        assert np.abs(got[0, t] - want).max() <= host(q).__abs__().max() * 2 * m * 4 * 2**-22
    assert (pool[0] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D,part", [(64, 62), (64, 60), (64, 40), (128, 10), (128, 100), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [70, 1027])
def test_rope_layouts(T, interleaved, D, part, dtype):
    """Halves of every alignment, short and long calls; what lies behind
    rotary_dim comes through bit by bit, infinities and NaN too, and stays out
    of the pairs."""
    nh, nkv, start = 3, 2, 5
    kc = torch.zeros((1, nkv, T + start, D), dtype=BF16, device=dev())
    vc = torch.zeros_like(kc)
    q = torch.randn((1, T, nh, D), device=dev()).to(dtype)
    kn = torch.randn((1, T, nkv, D), device=dev()).to(dtype)
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0], device=dev())
    for x in (q, kn):
        x[:, ::3, :, part:] = odd.repeat(D)[:D - part].to(dtype)
    qh, kh = host(q), host(kn)
    out = mk.rope_append(mk.Rope(D, rotary_dim=part, interleaved=interleaved),
                         mk.Cache([kc], [vc]), 0, q, kn, kn, ints([start]), q_out=q)
    f, m = ref.frequencies(part, 10000.0)
    got, keys = host(out)[0], host(kc)[0]
    rest = dict(equal_nan=True)
    assert np.array_equal(got[..., part:], qh[0, ..., part:], **rest)
    assert np.array_equal(keys[:, start:, part:], host(kn.to(BF16))[0, ..., part:].swapaxes(0, 1), **rest)
    assert np.array_equal(host(vc)[0, :, start:], host(kn.to(BF16))[0].swapaxes(0, 1), **rest)
    for t in {0, 1, 33, T - 3, T - 2, T - 1}:
        for x, y, r in ((qh[0, t], got[t], 2**-8 if dtype == BF16 else 2**-24),
                        (kh[0, t], keys[:, start + t], 2**-8)):
            want = ref.rotate(x[:, :part], start + t, f, m, interleaved)
            near = np.abs(x[:, :part]).max() * 4 * 2**-22 + r * np.abs(want)
            assert (np.abs(y[:, :part] - want) <= near).all()


def test_rope_prompt_in_place_and_bounds():
    """A chain longer than a tree may be, rotated in place, running over the end
    of the cache and over a page that is not there: those rows are dropped."""
    rng = np.random.default_rng(0)
    B, T, nh, nkv, D, bs = 2, 2100, 4, 2, 64, 16
    k, v, table = make_cache(rng, B, 2048, nkv, D, bs)
    table[0, 3] = -1
    qkv = torch.randn((B, T, nh + 2 * nkv, D), device=dev()).to(BF16)
    q, kn, vn = qkv.split([nh, nkv, nkv], 2)
    qh, kh, vh = host(q), host(kn), host(vn)
    untouched = [i for i in range(len(k[0])) if i not in table]
    kb, vb = k[0][untouched].clone(), v[0][untouched].clone()
    starts = [0, 1000]
    out = mk.rope_append(mk.Rope(D), mk.Cache(k, v, ints(table)), 0, q, kn, vn, ints(starts), q_out=q)
    assert out is q
    assert torch.equal(k[0][untouched], kb) and torch.equal(v[0][untouched], vb)
    assert np.array_equal(host(qkv[:, :, nh:]), np.concatenate([kh, vh], 2))
    f, m = ref.frequencies(D, 10000.0)
    kg, vg, qg = host(k[0]), host(v[0]), host(q)
    for b, t in itertools.product(range(B), (0, 1, 47, 48, 63, 64, 1047, 1048, 2047, 2099)):
        s = starts[b] + t
        want = ref.rotate(qh[b, t], s, f, m, False)
        assert (np.abs(qg[b, t] - want) <= 5 * 4 * 2**-22 + 2**-8 * np.abs(want)).all()
        if s < 2048 and table[b, s // bs] >= 0:
            want = ref.rotate(kh[b, t], s, f, m, False)
            assert (np.abs(kg[table[b, s // bs], :, s % bs] - want) <= 5 * 4 * 2**-22 + 2**-8 * np.abs(want)).all()
            assert np.array_equal(vg[table[b, s // bs], :, s % bs], vh[b, t])


def test_rope_single_token_matches_the_decode_step():
    """The k row that mk_decode_step appends at a position is the one that
    rope_append makes of the same projection (layer 0 of the tiny shape)."""
    from decode_megakernel_03_gb300 import synth
    shape, ctx = synth.TINY, 77
    w = synth.make_weights(shape, seed=0, device=dev())
    kc, vc = synth.make_kv(shape, 1, 96, (ctx,), seed=1, device=dev())
    k2, v2 = [t.clone() for t in kc], [t.clone() for t in vc]
    d = mk.Decoder(shape, w, kc, vc, 1)
    logits = torch.empty((1, shape.vocab), device=dev())
    d.step([9], [ctx], logits)
    assert d.status() == mk.MK_OK
    d.close()
    x = w["embed"][9].double()
    n = (x / torch.sqrt((x * x).mean() + shape.rms_eps) * w["attn_norm"][0].double())
    q, k, v = (w[m][0].double() @ n for m in ("wq", "wk", "wv"))
    mk.rope_append(mk.Rope(shape.head_dim, theta=shape.rope_theta), mk.Cache(k2, v2), 0,
                   q.float().view(1, 1, shape.n_heads, -1), k.float().view(1, 1, shape.n_kv_heads, -1),
                   v.float().view(1, 1, shape.n_kv_heads, -1), ints([ctx]))
    for a, b in ((kc, k2), (vc, v2)):
        x, y = host(a[0]), host(b[0])
        assert (np.abs(x - y) <= 1e-3 + 2**-7 * np.abs(y)).all()  # one bf16 step
        assert np.array_equal(x[:, :, :ctx], y[:, :, :ctx])


# ---- greedy acceptance -----------------------------------------------------------------------


def check_accept(logits, tokens, parents, counts):
    got = mk.tree_accept(logits, ints(tokens), ints(parents), ints(counts))
    want = ref.accept(host(logits), tokens, parents, counts)
    for g, w, name in zip(got, want, ("choices", "path", "accepted", "next")):
        assert np.array_equal(g.cpu().numpy(), w), name
    return want


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 3, 7), (3, 64, 1000), (1, 16, 50257), (8, 5, 4096),
                                   (2, 33, 12345)])
def test_accept(B, T, V, dtype):
    rng = np.random.default_rng(V)
    par = make_parents(rng, B, T)
    tokens = rng.integers(0, V, (B, T))
    logits = torch.randn((B, T, V), device=dev()).to(dtype)
    for b, t in itertools.product(range(B), range(1, T)):
        if rng.random() < 0.7:
            logits[b, par[b, t], tokens[b, t]] = 30.0  # ties among the lifted ones
    counts = None if B < 3 else [T] * (B - 2) + [0, max(1, T // 2)]
    want = check_accept(logits, tokens, par, counts)
    assert T < 30 or want[2].max() > 2
    check_accept(logits, tokens, None, counts)
    check_accept(logits, tokens, make_parents(rng, B, T, "odd"), counts)


@pytest.mark.parametrize("B,T,V,taken", [(3, 300, 77, [300, 1, 129]), (1024, 63, 5, None)])
def test_accept_long_chains_and_many_sequences(B, T, V, taken):
    rng = np.random.default_rng(T)
    tokens = rng.integers(0, V, (B, T))
    logits = torch.randn((B, T, V), device=dev())
    taken = rng.integers(1, T + 1, B) if taken is None else taken
    for b, n in enumerate(taken):
        logits[b, torch.arange(n - 1), torch.as_tensor(tokens[b, 1:n])] = 9.0
        if n < T:
            logits[b, n - 1, (tokens[b, n] + 1) % V] = 9.0
    want = check_accept(logits, tokens, None, None)
    assert list(want[2]) == list(taken)
    check_accept(logits, tokens, None, [T // 2] * B)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_accept_ties_signs_and_nan(dtype):
    V = 9001
    logits = torch.full((1, 8, V), -1.0, device=dev()).to(dtype)
    logits[0, 1, [17, 5000, 8999]] = 4.0
    logits[0, 2] = float("nan")
    logits[0, 3] = -float("inf")
    logits[0, 3, :40] = float("nan")
    logits[0, 4, 8000], logits[0, 4, 300] = 0.0, -0.0
    logits[0, 5, 4500] = float("inf")
    logits[0, 5, 4400] = float("nan")
    logits[0, 6] = -float("inf")
    logits[0, 7, 9000] = 1.0
    tokens = np.zeros((1, 8), np.int32)
    want = check_accept(logits, tokens, make_parents(np.random.default_rng(0), 1, 8), None)
    assert want[0][0].tolist() == [0, 17, 0, 40, 300, 4500, 0, 9000]


def test_accept_rows_of_other_strides():
    """Rows of a wider buffer, not on 16-byte boundaries; a long chain."""
    rng = np.random.default_rng(1)
    for dtype, width in ((FP32, 1003), (BF16, 1001), (BF16, 1016)):
        buf = torch.randn((2, 100, width), device=dev()).to(dtype)
        logits = buf[:, :, 1:1000] if width % 8 else buf[:, :, :999]
        tokens = host(logits).argmax(-1)
        chain = np.concatenate([tokens[:, :1], tokens[:, :-1]], 1)  # node t holds the choice of t - 1
        chain[1, 71] += 1
        want = check_accept(logits, chain, None, None)
        assert want[2].tolist() == [100, 71]
    del rng


def test_accept_twins_take_the_lowest():
    logits = torch.zeros((1, 6, 50), device=dev())
    logits[0, :, 7] = 1.0
    par = np.array([[-1, 0, 0, 2, 1, 4]])
    tok = np.array([[3, 7, 7, 7, 7, 9]])
    want = check_accept(logits, tok, par, None)
    assert want[1].tolist() == [[0, 1, 4, -1, -1, -1]] and want[3].tolist() == [7]


def test_accept_in_a_graph():
    rng = np.random.default_rng(1)
    logits = torch.randn((2, 9, 5000), device=dev())
    par, tok = make_parents(rng, 2, 9), rng.integers(0, 5000, (2, 9))
    tp, tt = ints(par), ints(tok)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mk.tree_accept(logits, tt, tp)
    logits[0, 0, tok[0, 1]] = 50.0
    g.replay()
    for a, w in zip(out, ref.accept(host(logits), tok, par, None)):
        assert np.array_equal(a.cpu().numpy(), w)


# ---- rows moved down, pages copied -----------------------------------------------------------------


@pytest.mark.parametrize("nkv,D,bs,layers", [(2, 64, 16, 3), (3, 128, 5, 2), (2, 64, 0, 1), (8, 128, 1, 4)])
def test_compact(nkv, D, bs, layers):
    rng = np.random.default_rng(D + bs)
    B, T = 5, 64
    k, v, table = make_cache(rng, B, 200, nkv, D, bs, layers=layers)
    starts = [100, 0, 33, 190, 60]
    path = np.full((B, T), -1, np.int32)
    sizes = [7, 64, 40, 12, 0]
    for b, n in enumerate(sizes):
        path[b, :n] = np.sort(rng.choice(T, n, replace=False))
    if table is not None:
        table[2, (33 + int(path[2, 20])) // bs] = -1  # a page that is not there
    path[0, 3], path[0, 5] = 99, -7  # out of range: skipped
    want = [host(t) for t in k + v]
    cap = table.shape[1] * bs if bs else 200
    for pool in want:
        for b in range(B):
            last = -1
            for i in range(sizes[b]):
                p = int(path[b, i])
                if not i <= p < T or p <= last:
                    continue
                last = p
                at = []
                for s in (starts[b] + p, starts[b] + i):
                    if s >= cap:
                        at.append(None)
                    elif table is None:
                        at.append((b, s))
                    else:
                        at.append((int(table[b, s // bs]), s % bs) if table[b, s // bs] >= 0 else None)
                if None not in at:
                    pool[at[1][0], :, at[1][1]] = pool[at[0][0], :, at[0][1]]
    mk.cache_compact(mk.Cache(k, v, ints(table)), ints(starts), ints(path), ints(sizes))
    for t, w in zip(k + v, want):
        assert np.array_equal(host(t), w)


def test_compact_paths_that_do_not_ascend():
    rng = np.random.default_rng(0)
    k, v, table = make_cache(rng, 1, 100, 1, 64, 16)
    path = np.array([[0, 5, 5, 4, 9, 3, 10, 10, 70, 12]], np.int32)
    moves = [(5, 1), (9, 4), (10, 6)]  # ascending and at or above their place
    path[0, 8] = -1
    path = np.pad(path, ((0, 0), (0, 6)), constant_values=-1)
    moves.append((12, 9))
    want = [host(k[0]), host(v[0])]
    for pool in want:
        for s, d in moves:
            s, d = s + 20, d + 20
            pool[table[0, d // 16], :, d % 16] = pool[table[0, s // 16], :, s % 16]
    mk.cache_compact(mk.Cache(k, v, ints(table)), ints([20]), ints(path), ints([12]))
    assert np.array_equal(host(k[0]), want[0]) and np.array_equal(host(v[0]), want[1])


@pytest.mark.parametrize("n,bs,nkv,D,layers", [(1, 16, 2, 64, 2), (40, 5, 3, 128, 2), (2500, 1, 1, 64, 2),
                                               (3, 256, 8, 128, 3), (32, 16, 2, 64, 1), (33, 16, 2, 64, 1)])
def test_copy_blocks(n, bs, nkv, D, layers):
    rng = np.random.default_rng(n)
    blocks = 2 * n + 3
    k, v = ([torch.randn((blocks, nkv, bs, D), device=dev()).to(BF16) for _ in range(layers)] for _ in range(2))
    order = rng.permutation(blocks)
    copies = np.stack([rng.choice(order[:n], n), order[n:2 * n], rng.integers(0, bs + 1, n)], 1)
    if n == 32:
        copies[:, 2] = 0
    want = [t.clone() for t in k + v]
    for t in want:
        for s, d, r in copies.tolist():
            t[d, :, :r] = t[s, :, :r]
    mk.cache_copy_blocks(mk.Cache(k, v), copies)
    assert all(torch.equal(a, b) for a, b in zip(k + v, want))


# ---- refusals of the binding ----------------------------------------------------------------------


def test_binding_refusals():
    rng = np.random.default_rng(0)
    k, v, table = make_cache(rng, 2, 64, 2, 64, 16)
    c = mk.Cache(k, v, ints(table))
    q = torch.randn((2, 3, 4, 64), device=dev()).to(BF16)
    kn = torch.randn((2, 3, 2, 64), device=dev()).to(BF16)
    s = ints([5, 6])
    rope = mk.Rope(64)
    bad = [lambda: mk.tree_attention(c, 0, q.double(), s), lambda: mk.tree_attention(c, 0, q.cpu(), s),
           lambda: mk.tree_attention(c, 0, q, s.long()), lambda: mk.tree_attention(c, 0, q, ints([5])),
           lambda: mk.tree_attention(c, 0, q, s.cpu()), lambda: mk.tree_attention(c, 1, q, s),
           lambda: mk.tree_attention(c, 0, q, s, parents=ints(np.zeros((2, 4)))),
           lambda: mk.tree_attention(c, 0, q, s, counts=ints([1, 2, 3])),
           lambda: mk.tree_attention(c, 0, q[:, :, :3], s), lambda: mk.tree_attention(c, 0, q[0], s),
           lambda: mk.tree_attention(c, 0, q.transpose(1, 2), s),
           lambda: mk.tree_attention(c, 0, q.transpose(0, 1), s),
           lambda: mk.tree_attention(c, 0, q[..., :32], s),
           lambda: mk.tree_attention(c, 0, q, s, out=torch.empty_like(q).float()),
           lambda: mk.tree_attention(c, 0, q, s, out=torch.empty_like(kn)),
           lambda: mk.tree_attention(c, 0, q.repeat(2, 1, 1, 1), s.repeat(2)),
           lambda: mk.tree_attention(c, 0, q, s, scale=0.0),
           lambda: mk.rope_append(rope, c, 0, q, kn, kn.float(), s),
           lambda: mk.rope_append(rope, c, 0, q, q, kn, s),
           lambda: mk.rope_append(mk.Rope(128), c, 0, q, kn, kn, s),
           lambda: mk.rope_append(rope, c, 0, q, kn, kn, s, q_out=kn),
           lambda: mk.tree_accept(torch.zeros((2, 3, 9), device=dev(), dtype=torch.float16), s),
           lambda: mk.tree_accept(torch.zeros((2, 3, 9), device=dev()), s),
           lambda: mk.tree_accept(torch.zeros((2, 3, 18), device=dev())[..., ::2], ints(np.zeros((2, 3)))),
           lambda: mk.cache_compact(c, s, ints(np.zeros((1, 3))), s),
           lambda: mk.cache_copy_blocks(c, [[0, 1]]), lambda: mk.cache_copy_blocks(c, [[0, 99, 1]]),
           lambda: mk.Cache(k, v, table), lambda: mk.Cache([k[0].float()], v),
           lambda: mk.Cache(k, [v[0][:, :1]]), lambda: mk.Cache([k[0].transpose(1, 2)], v)]
    before = [t.clone() for t in k + v]
    for i, f in enumerate(bad):
        with pytest.raises(mk.MkError) as e:
            f()
        assert e.value.code == mk.MK_ERR_INVALID, i
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(k + v, before))


# ---- together ----------------------------------------------------------------------------------------


def norm(x, w, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def verify(shape, w, cache, rope, tokens, starts, parents):
    """Logits of every node of the trees: the model in torch, over the cache."""
    B, T = tokens.shape
    x = w["embed"][tokens.long()].float()
    for l in range(shape.n_layers):
        n = norm(x, w["attn_norm"][l], shape.rms_eps)
        q, k, v = ((n @ w[m][l].float().T).view(B, T, -1, shape.head_dim) for m in ("wq", "wk", "wv"))
        q = mk.rope_append(rope, cache, l, q, k, v, starts, parents)
        a = mk.tree_attention(cache, l, q, starts, parents)
        x = x + a.reshape(B, T, -1) @ w["wo"][l].float().T
        n = norm(x, w["mlp_norm"][l], shape.rms_eps)
        x = x + (torch.nn.functional.silu(n @ w["wgate"][l].float().T) * (n @ w["wup"][l].float().T)) @ w["wdown"][l].float().T
    return norm(x, w["final_norm"], shape.rms_eps) @ (w["lm_head"] if w["lm_head"] is not None else w["embed"]).float().T


def test_drafts_verified_over_the_decoders_pages():
    """A prompt, forked in two; each fork's drafted tree verified, its accepted
    rows kept; the decoder's own paged step goes on from there. Every node's
    logits agree with the decoder stepping through the node's path, and the
    last step with the decoder on a cache of its own."""
    from decode_megakernel_03_gb300 import synth
    shape, bs, cap, n_seqs = synth.TINY, 16, 96, 4
    D = shape.head_dim
    w = synth.make_weights(shape, seed=3, device=dev())
    pages = mk.Pages(40, bs, n_seqs, cap)
    k, v = ([torch.zeros((40, shape.n_kv_heads, bs, D), dtype=BF16, device=dev()) for _ in range(shape.n_layers)]
            for _ in range(2))
    dec = mk.Decoder(shape, w, k, v, 2, paged=(bs, 40, cap))
    rope = mk.Rope(D, theta=shape.rope_theta)
    logits = torch.empty((2, shape.vocab), device=dev())

    def solo(tokens):
        """Logits after each token, from the decoder on a contiguous cache."""
        kc, vc = synth.empty_kv(shape, 1, cap, device=dev())
        d = mk.Decoder(shape, w, kc, vc, 1)
        out, l1 = [], torch.empty((1, shape.vocab), device=dev())
        for i, t in enumerate(tokens):
            d.step([int(t)], [i], l1)
            assert d.status() == mk.MK_OK
            out.append(l1[0].clone())
        d.close()
        return out

    def near(a, b):
        a, b = host(a), host(b)
        assert np.linalg.norm(a - b) <= 1e-2 * np.linalg.norm(b) and np.abs(a - b).max() <= 5e-2

    prompt = synth.make_tokens(shape.vocab, 21, seed=5).tolist()
    pages.resize([0], [len(prompt)])
    table = ints(pages.table())
    cache1 = mk.Cache(k, v, table[:1].contiguous())
    first = verify(shape, w, cache1, rope, ints([prompt]), ints([0]), None)  # the prompt is a chain
    near(first[0, -1], solo(prompt)[-1])
    pages.fork([0, 0], [1, 2])
    pages.resize([0], [0])
    said = {1: list(prompt), 2: list(prompt)}
    last = {1: int(first[0, -1].argmax()), 2: int(first[0, -1].argsort()[-2])}
    rng = np.random.default_rng(1)
    for _ in range(3):
        T = 12
        starts = [len(said[s]) for s in (1, 2)]
        mk.cache_copy_blocks(mk.Cache(k, v), pages.resize([1, 2], [n + T for n in starts]))
        table = ints(pages.table()[1:3])
        cache = mk.Cache(k, v, table)
        parents = make_parents(rng, 2, T)
        tokens = rng.integers(0, shape.vocab, (2, T))
        tokens[:, 0] = [last[1], last[2]]
        # the decoder's own next tokens drafted along one path
        for i, s in enumerate((1, 2)):
            path, t = [0], 0
            while len(path) < 4:
                kids = [c for c in range(t + 1, T) if parents[i, c] == t]
                if not kids:
                    break
                nxt = solo(said[s] + [int(tokens[i, p]) for p in path])[-1]
                t = kids[-1]
                tokens[i, t] = int(nxt.argmax())
                path.append(t)
        got = verify(shape, w, cache, rope, ints(tokens), ints(starts), ints(parents))
        for i, s in enumerate((1, 2)):
            for t in (0, 5, T - 1):
                line = ref.family(parents, i, t)[::-1]
                near(got[i, t], solo(said[s] + [int(tokens[i, p]) for p in line])[-1])
        choices, path, accepted, nxt = mk.tree_accept(got, ints(tokens), ints(parents))
        want = ref.accept(host(got), tokens, parents, None)
        for a, b in zip((choices, path, accepted, nxt), want):
            assert np.array_equal(a.cpu().numpy(), b)
        mk.cache_compact(cache, ints(starts), path, accepted)
        acc = accepted.cpu().tolist()
        for i, s in enumerate((1, 2)):
            said[s] += [int(tokens[i, p]) for p in want[1][i, :acc[i]]]
            last[s] = int(nxt[i])
        pages.resize([1, 2], [len(said[1]), len(said[2])])
    assert sum(len(s) for s in said.values()) > 2 * (len(prompt) + 3)  # something was accepted
    # the pages tidied up, then the decoder's own step
    pages.resize([3], [17])
    pages.resize([3], [0])
    mk.cache_copy_blocks(mk.Cache(k, v), pages.compact())
    pos = [len(said[1]), len(said[2])]
    mk.cache_copy_blocks(mk.Cache(k, v), pages.resize([1, 2], [p + 1 for p in pos]))
    dec.step_paged([last[1], last[2]], pos, pages.table()[1:3], logits)
    assert dec.status() == mk.MK_OK, dec.last_error()
    for i, s in enumerate((1, 2)):
        near(logits[i], solo(said[s] + [last[s]])[-1])
    dec.close()
