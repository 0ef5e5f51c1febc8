"""Attention of groups that share a prefix against its plain 64-bit form, at the group
sizes, lengths, masks and layouts where it can go wrong."""
import numpy as np
import pytest
import torch

from decode_megakernel_03_gb300 import mk
from tests import sampling_ref as ref
from tests.test_gpu_cache_ops import BF16, FP32, attention_bound, dev, host, ints, make_cache, make_parents

pytestmark = pytest.mark.gpu


def check(rng, first, prefix, starts, T, nh, nkv, D, dtype, bs, counts=None, parents="tree", missing=0,
          scale=None, room=None, strided=False, poison=False, seed=7):
    """The call against the plain form; what lies behind counts, in the other slots of a group's later
    sequences (below the shared length) and in blocks of no table plays no part."""
    starts = np.asarray(starts)
    B = len(starts)
    room = room or int(max(starts)) + T
    k, v, table = make_cache(rng, B, room, nkv, D, bs, missing=missing)
    par = None if parents is None else make_parents(rng, B, T, parents)
    cap = table.shape[1] * bs if bs else room
    kp, vp = host(k[0]), host(v[0])
    if poison:
        mine = np.zeros(kp.shape[:1] + kp.shape[2:3], bool)
        leader, shared = ref.shared_lengths(B, T, cap, first, prefix, starts, counts)
        for b in range(B):
            c = T if counts is None else ref.ref.clamp(counts[b], T)
            if c == 0:
                continue
            for s in range(min(ref.ref.clamp(starts[b], cap) + c, cap)):
                o = leader[b] if s < shared[b] else b
                blk, row = (o, s) if table is None else (int(table[o, s // bs]), s % bs)
                if 0 <= blk < len(mine):
                    mine[blk, row] = True
        hide = torch.tensor(~mine, device=dev())[:, None, :, None].expand_as(k[0])
        k[0][hide], v[0][hide] = float("nan"), float("inf")
    g = torch.Generator(device=dev()).manual_seed(seed)
    if strided:
        q = torch.randn((B, T, nh + 3, D), generator=g, device=dev()).to(dtype)[:, :, 1:nh + 1]
        out = torch.full((B, T, 2 * nh, D), 77.0, device=dev(), dtype=dtype)[:, :, nh:]
    else:
        q = torch.randn((B, T, nh, D), generator=g, device=dev()).to(dtype)
        out = torch.full((B, T, nh, D), 77.0, device=dev(), dtype=dtype)
    cache = mk.Cache(k, v, ints(table))
    args = (q, ints(first), ints(prefix), ints(starts), ints(par), ints(counts))
    got = host(mk.prefix_attention(cache, 0, *args, scale=scale, out=out))
    want, a, e = ref.prefix_attention(host(q), kp, vp, table, first, prefix, starts, par, counts,
                                      D ** -0.5 if scale is None else scale)
    live = ~np.isnan(want)
    assert (got[~live] == 77.0).all()
    assert np.isfinite(got).all()
    off = np.abs(got - want) / attention_bound(want, a, e, cap, D, dtype)
    assert (off[live] <= 1).all(), f"{np.nanmax(off):.3g} of the bound"
    return cache, args, want


SHAPES = [(4, 2, 64), (8, 1, 64), (4, 4, 128), (12, 2, 128)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("nh,nkv,D", SHAPES)
@pytest.mark.parametrize("T", [1, 3, 16])
def test_two_groups(T, nh, nkv, D, dtype):
    rng = np.random.default_rng(T)
    check(rng, [0, 3], [130, 40], [130, 141, 200, 61, 40], T, nh, nkv, D, dtype, 16, poison=True)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B,T,G", [(1, 1, 1), (9, 1, 4), (40, 1, 4), (70, 1, 8), (20, 7, 4), (33, 5, 8), (3, 64, 8)])
def test_group_sizes(B, T, G, dtype):
    """From one row to several row tiles, full and begun ones."""
    rng = np.random.default_rng(B)
    starts = 150 + rng.integers(0, 90, B)
    check(rng, [0], [150], starts, T, 2 * G, 2, 64, dtype, 16, poison=True)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bs", [0, 1, 5, 48, 64, 256])
def test_layouts(bs, dtype):
    rng = np.random.default_rng(bs)
    check(rng, [0, 2], [100, 129], [100, 300, 129, 257, 140], 6, 4, 2, 64, dtype, bs, poison=True, strided=True)


@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 127, 128, 129, 256, 400])
@pytest.mark.parametrize("tail", [0, 1, 127, 128])
def test_lengths(prefix, tail):
    """Prefixes and tails around a tile's size, none, and longer than a context."""
    rng = np.random.default_rng(prefix)
    check(rng, [0], [prefix], [min(prefix, 256) + tail, 300 + tail], 2, 4, 1, 128, BF16, 16, poison=True)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (FP32, 64), (FP32, 128)])
def test_long(dtype, D):
    rng = np.random.default_rng(D)
    check(rng, [0], [9001], [9001, 9700, 9050], 2, 4, 2, D, dtype, 32, strided=True)
    check(rng, [0, 20], [3000, 777], np.concatenate([3000 + rng.integers(0, 400, 20), 777 + rng.integers(0, 50, 30)]),
          1, 8, 2, D, dtype, 64)


@pytest.mark.parametrize("first,prefix", [([2], [50]), ([6], [50]), ([0, 0, 3], [9, 60, 60]), ([-5, 99, 2], [60, 60, 60]),
                                          ([0, 4, 1], [60, -3, 2**31 - 1]), ([0, 1, 2, 3, 4, 5], [60, 0, 60, 61, 1, 33]),
                                          ([3, 3, 3, 3], [1, 2, 3, 40]), ([0, 2, 4], [-2**31, 64, 10])])
@pytest.mark.parametrize("counts", [None, [5, 0, 1, -4, 99, 3], [0, 0, 5, 5, 0, 0]])
def test_groups_of_all_kinds(first, prefix, counts):
    """Sequences of no group, empty groups, values out of range, sequences without nodes (the first of a group
    among them, whose rows are read all the same)."""
    rng = np.random.default_rng(len(first))
    check(rng, first, prefix, [64, 70, 130, 61, 64, 200], 5, 8, 2, 64, BF16, 16, counts=counts, poison=True, strided=True)


def test_no_sequence_at_all():
    rng = np.random.default_rng(5)
    check(rng, [0], [30], [40, 100], 4, 4, 2, 64, BF16, 16, counts=[0, -1])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [4, 40])
def test_missing_pages(T, dtype):
    """Pages that are not there, starts behind the capacity and below 0."""
    rng = np.random.default_rng(T)
    check(rng, [0, 3], [40, 64], [45, 64, 500, 64, 64], T, 8, 2, 64, dtype, 8, missing=12, room=64)
    check(rng, [0], [40], [40, -6, 50], T, 8, 2, 64, dtype, 8, missing=5, room=64)
    k, v, _ = make_cache(rng, 2, 64, 2, 64, 8)
    none = torch.full((2, 8), -1, dtype=torch.int32, device=dev())
    q = torch.randn((2, T, 8, 64), device=dev()).to(dtype)
    out = mk.prefix_attention(mk.Cache(k, v, none), 0, q, ints([0]), ints([20]), ints([30, 20]))
    assert (out == 0).all()
    # own keys missing, the prefix there, and the other way round
    table = ints(np.arange(16).reshape(2, 8))
    for gone in (slice(0, 3), slice(3, 8)):
        t = table.clone()
        t[:, gone] = -1
        got = mk.prefix_attention(mk.Cache(k, v, t), 0, q, ints([0]), ints([24]), ints([24, 24]), ints(np.full((2, T), -1)))
        want, _, _ = ref.prefix_attention(host(q), host(k[0]), host(v[0]), t.cpu().numpy(), [0], [24], [24, 24],
                                          np.full((2, T), -1), None, 0.125)
        assert np.abs(host(got) - want).max() <= 0.03


def test_a_full_cache():
    """Contexts as long as the cache: the nodes' own rows are not there."""
    rng = np.random.default_rng(3)
    check(rng, [0], [64], [64, 64, 64], 3, 4, 2, 64, BF16, 16, room=64)


@pytest.mark.parametrize("scale", [1e-6, 3.0])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_scale(scale, dtype):
    rng = np.random.default_rng(1)
    check(rng, [0], [150], [200, 170], 6, 4, 2, 64, dtype, 16, scale=scale)


@pytest.mark.parametrize("T,nh,nkv,dtype", [(1, 2, 1, BF16), (9, 2, 1, BF16), (5, 2, 2, FP32)])
def test_as_many_sequences_as_there_may_be(T, nh, nkv, dtype):
    """1024 sequences in as many groups, in a few, in one; some without a node."""
    rng = np.random.default_rng(T)
    starts, counts = rng.integers(8, 40, 1024), rng.integers(0, T + 1, 1024)
    for first in (np.arange(1024), [0, 5, 600], [0]):
        check(rng, first, rng.integers(0, 30, len(first)), starts, T, nh, nkv, 64, dtype, 16, counts=counts)


def test_equals_tree_attention_where_tables_agree():
    """Forked pages: the result is the tree attention's up to the order of its sums, for every group layout."""
    rng = np.random.default_rng(0)
    B, P, bs, nkv, D, T = 12, 333, 16, 2, 128, 3
    pages = mk.Pages(400, bs, B + 1, 1024)
    k, v = ([torch.randn((400, nkv, bs, D), device=dev()).to(BF16)] for _ in range(2))
    pages.resize([B], [P])
    pages.fork([B] * B, range(B))
    starts = P + rng.integers(0, 300, B)
    starts[3] = P  # the shortest: a longer prefix is taken as P, as far as the tables agree
    mk.cache_copy_blocks(mk.Cache(k, v), pages.resize(range(B), starts + T))
    cache = mk.Cache(k, v, ints(pages.table()[:B]))
    par = ints(make_parents(rng, B, T))
    for dtype in (BF16, FP32):
        q = torch.randn((B, T, 8, D), device=dev()).to(dtype)
        want = host(mk.tree_attention(cache, 0, q, ints(starts), par))
        for first, prefix in (([0], [P]), ([0, 5], [P, 100]), ([3], [P]), ([0], [5000])):
            got = host(mk.prefix_attention(cache, 0, q, ints(first), ints(prefix), ints(starts), par))
            # (bf16: a rounding that falls the other way, 2^-8 of the larger; the sums' order 2^-20)
            off = np.abs(got - want) - ((2**-7 if dtype == BF16 else 0) * np.abs(want) + 2**-18)
            assert off.max() <= 0, (dtype, first, prefix)


@pytest.mark.parametrize("T,dtype", [(1, BF16), (30, BF16), (3, FP32)])
def test_in_place(T, dtype):
    rng = np.random.default_rng(T)
    k, v, table = make_cache(rng, 4, 400, 2, 64, 16)
    cache = mk.Cache(k, v, ints(table))
    args = ints([0, 2]), ints([250, 60]), ints([300, 257, 90, 60])
    q = torch.randn((4, T, 16, 64), device=dev()).to(dtype)
    want = mk.prefix_attention(cache, 0, q, *args)
    assert mk.prefix_attention(cache, 0, q, *args, out=q) is q
    assert torch.equal(q, want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,G", [(6, 2), (40, 4)])
def test_odd_values_stay_with_the_rows_that_see_them(T, G, dtype):
    """NaN and infinities in a node's k or v row reach its descendants only; in a row's q that row only; in a prefix
    the whole group, and no other."""
    rng = np.random.default_rng(2)
    B, nkv, D = 4, 2, 64
    k, v, table = make_cache(rng, B, 128 + T, nkv, D, 16)
    par = make_parents(rng, B, T)
    starts = [100, 101, 70, 64]
    q = torch.randn((B, T, nkv * G, D), device=dev()).to(dtype)
    cache = mk.Cache(k, v, ints(table))
    args = ints([0, 2]), ints([90, 64]), ints(starts), ints(par)
    clean = mk.prefix_attention(cache, 0, q, *args).clone()
    hit = torch.zeros((B, T), dtype=torch.bool)
    for b, node, pool, x in ((0, 2, v, float("inf")), (1, 4, v, float("nan")), (2, 3, k, float("nan")), (3, 5, v, -float("inf"))):
        s = starts[b] + node
        pool[0][table[b, s // 16], :, s % 16, 7] = x
        for t in range(T):
            hit[b, t] |= node in ref.ref.family(par, b, t)
    got = mk.prefix_attention(cache, 0, q, *args)
    assert torch.equal(got[~hit], clean[~hit])
    assert (~torch.isfinite(got[hit])).any(-1).all()
    q2 = q.clone()
    q2[0, 1, 0, 3] = float("nan")
    got2 = mk.prefix_attention(cache, 0, q2, *args)
    assert got2[0, 1, 0].isnan().all()
    got2[0, 1, 0] = got[0, 1, 0]
    assert torch.equal(got2.nan_to_num(3.0), got.nan_to_num(3.0))
    v[0][table[2, 1], :, 5, 9] = float("nan")  # slot 21 of the second group's first sequence
    got3 = mk.prefix_attention(cache, 0, q, *args)
    assert got3[2:, ..., 9].isnan().all()
    assert torch.equal(got3[:2].nan_to_num(3.0), got[:2].nan_to_num(3.0))


@pytest.mark.parametrize("T,dtype", [(1, BF16), (7, FP32), (40, BF16)])
def test_streams_graphs_and_repeats(T, dtype):
    """The same bits again: repeated, on another stream, captured and replayed (two graphs at once), and a
    captured call follows lengths and groups that change."""
    rng = np.random.default_rng(4)
    cache, args, _ = check(rng, [0, 3], [700, 20], [700, 800, 933, 20, 333], T, 8, 2, 128, dtype, 16)
    call = lambda **kw: mk.prefix_attention(cache, 0, *args, **kw)
    first = call()
    for _ in range(20):
        assert torch.equal(call(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = call(stream=side)
    side.synchronize()
    assert torch.equal(a, first)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
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
    args[1].copy_(ints([0, 1]))
    args[2].copy_(ints([100, 333]))
    args[3].copy_(ints([100, 340, 933, 900, 333]))
    graphs[0].replay()
    assert torch.equal(outs[0], call())


def test_pool_of_more_than_2_to_the_31_elements():
    nkv, bs, D, blocks = 8, 64, 128, 36000
    big = [torch.empty((blocks, nkv, bs, D), dtype=BF16, device=dev()) for _ in range(2)]
    rng = np.random.default_rng(0)
    table = rng.permutation(np.arange(blocks - 60, blocks))[:30].reshape(3, 10).astype(np.int32)
    small_table = np.arange(30, dtype=np.int32).reshape(3, 10)
    at = torch.tensor(table.ravel(), device=dev(), dtype=torch.int64)
    small = [torch.randn((30, nkv, bs, D), device=dev()).to(BF16) for _ in range(2)]
    for b, s in zip(big, small):
        b[at] = s
    args = ints([0]), ints([400]), ints([500, 400, 600])
    for dtype, T in ((BF16, 2), (BF16, 20), (FP32, 2), (FP32, 10)):
        q = torch.randn((3, T, 16, D), device=dev()).to(dtype)
        a, b = (mk.prefix_attention(mk.Cache([p[0]], [p[1]], ints(t)), 0, q, *args) for p, t in ((big, table), (small, small_table)))
        assert torch.equal(a, b)


# By norm against 64 bits. fp32: 1e-6, as the tree attention's (a row joins one more share here, a
# rounding of 2^-24). bf16: before its rounding the output is off by e, 2^-17 of itself by norm for weights of
# two bf16 parts and 2^-20 for scores. The rounded value is nearest to what was rounded, so it is off by at most
# the rounding of the exact output and 2 e: by norm that rounding's own error r and 2^-15. (Not against the rounded
# output by a fixed bound: of 512 elements one that falls the other way, 2^-7 of it at twice the usual size, is
# 2 x 2^-7 / sqrt(512) = 6.9e-4 of the norm. Weights of one part, 2^-9, give sqrt(r^2 + 2^-18), 4e-4 above r = 1.65e-3.)
@pytest.mark.parametrize("B,T,nh,nkv,D,dtype", [(3, 1, 4, 2, 64, BF16), (40, 1, 8, 2, 128, BF16), (12, 12, 16, 2, 128, BF16),
                                                (70, 1, 8, 2, 64, BF16), (3, 2, 4, 2, 64, FP32), (12, 5, 8, 2, 128, FP32),
                                                (20, 4, 16, 4, 64, FP32), (2, 2, 8, 2, 128, FP32)])
def test_error_by_norm(B, T, nh, nkv, D, dtype):
    rng = np.random.default_rng(T + D)
    starts = 1500 + rng.integers(0, 300, B)
    k, v, table = make_cache(rng, B, 1800 + T, nkv, D, 16)
    par = make_parents(rng, B, T)
    g = torch.Generator(device=dev()).manual_seed(11)
    q = torch.randn((B, T, nh, D), generator=g, device=dev()).to(dtype)
    got = host(mk.prefix_attention(mk.Cache(k, v, ints(table)), 0, q, ints([0]), ints([1500]), ints(starts), ints(par)))
    want = ref.prefix_attention(host(q), host(k[0]), host(v[0]), table, [0], [1500], starts, par, None, D**-0.5)[0]
    r = host(torch.from_numpy(want).to(BF16)) - want if dtype == BF16 else 0 * want
    for b in range(B):
        off, own = (np.linalg.norm(x) / np.linalg.norm(want[b]) for x in (got[b] - want[b], r[b]))
        assert off <= own + (2.0**-15 if dtype == BF16 else 1e-6), f"sequence {b}: {off:.3g}, {own:.3g}"


def test_binding_refusals():
    rng = np.random.default_rng(0)
    k, v, table = make_cache(rng, 2, 64, 2, 64, 16)
    c = mk.Cache(k, v, ints(table))
    q = torch.randn((2, 3, 4, 64), device=dev()).to(BF16)
    f, x, s = ints([0]), ints([4]), ints([5, 6])
    call = mk.prefix_attention
    bad = [lambda: call(c, 0, q.double(), f, x, s), lambda: call(c, 0, q.cpu(), f, x, s),
           lambda: call(c, 0, q, f.long(), x, s), lambda: call(c, 0, q, f, x.cpu(), s), lambda: call(c, 0, q, f, x, ints([5])),
           lambda: call(c, 0, q, ints([0, 1]), x, s), lambda: call(c, 0, q, ints([[0]]), x, s), lambda: call(c, 1, q, f, x, s),
           lambda: call(c, 0, q, ints([0, 1, 2]), ints([0, 1, 2]), s), lambda: call(c, 0, q, ints([]), ints([]), s),
           lambda: call(c, 0, q, f, x, s, parents=ints(np.zeros((2, 4)))), lambda: call(c, 0, q, f, x, s, counts=ints([1, 2, 3])),
           lambda: call(c, 0, q[:, :, :3], f, x, s), lambda: call(c, 0, q.transpose(1, 2), f, x, s),
           lambda: call(c, 0, q, f, x, s, out=torch.empty_like(q).float()), lambda: call(c, 0, q, f, x, s, scale=0.0),
           lambda: call(c, 0, q.repeat(2, 1, 1, 1), f, x, s.repeat(2))]
    before = [t.clone() for t in k + v]
    for i, f_ in enumerate(bad):
        with pytest.raises(mk.MkError) as e:
            f_()
        assert e.value.code == mk.MK_ERR_INVALID, i
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(k + v, before))
