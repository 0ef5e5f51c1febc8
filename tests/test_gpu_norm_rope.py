"""Queries and keys normalised for each head, rotated and appended in one pass, against the
plain 64-bit form."""
import math

import numpy as np
import pytest
import torch

from decode_megakernel_03_gb300 import mk
from tests import cache_ops_ref as ref
from tests import sampling_ref
from tests.test_gpu_cache_ops import BF16, FP32, dev, host, ints, make_cache, make_parents

pytestmark = pytest.mark.gpu

# Of a normed element: the sum of squares (8 products and adds of a lane, 4 of the lanes, eps: 13 of
# 2^-24, half of them in the root), the root, its product with the weight and with x: 10 x 2^-24.
# Rotated: two such elements at most the head's largest each, sine and cosine to 2^-22, two products
# and an add: (10 x 2^-24 + 2^-22 + 3 x 2^-24) x 2 = 8.5 x 2^-22 of the largest.
NEAR = 9 * 2**-22


def weights(rng, D, kind):
    if kind == "none":
        return None, None
    w = [torch.from_numpy((1 + 0.5 * rng.normal(size=D)).astype(np.float32)).to(BF16).to(dev()) for _ in range(2)]
    return (w[0], None) if kind == "q" else (None, w[1]) if kind == "k" else tuple(w)


def expected(x, w, eps, pos, f, m, interleaved):
    y = sampling_ref.normed(x, None if w is None else host(w), eps)
    return ref.rotate(y, pos, f, m, interleaved), np.abs(y).max(-1, keepdims=True) * m


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D,part,interleaved", [(64, 64, False), (64, 32, False), (64, 60, False), (64, 62, False),
                                                (64, 2, True), (128, 128, False), (128, 96, True), (128, 124, False),
                                                (128, 64, True), (128, 16, False), (128, 126, False)])
@pytest.mark.parametrize("bs,kind", [(0, "both"), (5, "q"), (16, "k"), (16, "none")])
def test_norm_rope_append(D, part, interleaved, bs, kind, dtype):
    rng = np.random.default_rng(part + bs)
    B, T, nh, nkv, eps = 3, 11, 6, 3, 1e-5
    starts, counts = [40, 0, 3], [11, 4, 0]
    k, v, table = make_cache(rng, B, 60, nkv, D, bs, layers=2)
    par = make_parents(rng, B, T, "odd")
    size_of = torch.exp(3 * torch.randn((1, 1, nh + 2 * nkv, 1), device=dev()))
    qkv = (torch.randn((B, T, nh + 2 * nkv, D), device=dev()) * size_of).to(dtype)
    qkv[0, 2, 1], qkv[0, 3, nh + 1] = 0.0, 0.0  # heads of zeros stay zeros
    q, kn, vn = qkv.split([nh, nkv, nkv], 2)
    qw, kw_ = weights(rng, D, kind)
    f, m = ref.frequencies(part, 10000.0)
    before = [t.clone() for t in k + v]
    qh, kh, vh = host(q), host(kn), host(vn)
    out = torch.full((B, T, nh, D), 77.0, device=dev(), dtype=dtype)
    mk.norm_rope_append(mk.Rope(D, theta=10000.0, rotary_dim=part, interleaved=interleaved), mk.Cache(k, v, ints(table)),
                        1, q, kn, vn, qw, kw_, ints(starts), ints(par), ints(counts), eps=eps, q_out=out)
    assert torch.equal(k[0], before[0]) and torch.equal(v[0], before[2])  # the other layer
    k_want, v_want, near = host(before[1]), host(before[3]), np.zeros(before[1].shape)
    size = bs or 60
    r = 2**-8 if dtype == BF16 else 2**-24
    for b in range(B):
        for t in range(T):
            if t >= counts[b]:
                assert (out[b, t] == 77.0).all()
                continue
            pos = starts[b] + len(ref.family(par, b, t)) - 1
            want, top = expected(qh[b, t], qw, eps, pos, f, m, interleaved)
            assert (np.abs(host(out[b, t]) - want) <= NEAR * top + r * np.abs(want)).all()
            s = starts[b] + t
            blk = b if table is None else table[b, s // size]
            want, top = expected(kh[b, t], kw_, eps, pos, f, m, interleaved)
            k_want[blk, :, s % size], near[blk, :, s % size] = want, NEAR * top + 2**-8 * np.abs(want)
            v_want[blk, :, s % size] = host(vn[b, t].to(BF16))
    assert (np.abs(host(k[1]) - k_want) <= near).all()
    assert np.array_equal(host(v[1]), v_want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("interleaved,part", [(False, 128), (True, 128), (False, 100)])
def test_prompts_in_place(interleaved, part, dtype):
    """More tokens than a tree has, queries in place, over the end of the cache and a page that is not there."""
    rng = np.random.default_rng(0)
    B, T, nh, nkv, D, bs = 2, 1300, 4, 2, 128, 16
    k, v, table = make_cache(rng, B, 1280, nkv, D, bs)
    table[0, 3] = -1
    qkv = torch.randn((B, T, nh + 2 * nkv, D), device=dev()).to(dtype)
    q, kn, vn = qkv.split([nh, nkv, nkv], 2)
    qh, kh, vh = host(q), host(kn), host(vn.to(BF16))
    untouched = [i for i in range(len(k[0])) if i not in table]
    kb, vb = k[0][untouched].clone(), v[0][untouched].clone()
    rest = host(qkv[:, :, nh:])
    qw, kw_ = weights(rng, D, "both")
    starts, (f, m) = [0, 500], ref.frequencies(part, 10000.0)
    out = mk.norm_rope_append(mk.Rope(D, rotary_dim=part, interleaved=interleaved), mk.Cache(k, v, ints(table)), 0, q, kn, vn,
                              qw, kw_, ints(starts), q_out=q)
    assert out is q
    assert torch.equal(k[0][untouched], kb) and torch.equal(v[0][untouched], vb) and np.array_equal(host(qkv[:, :, nh:]), rest)
    kg, vg, qg = host(k[0]), host(v[0]), host(q)
    for b in range(B):
        for t in (0, 1, 2, 3, 47, 48, 63, 64, 777, 779, 780, 1279, 1280, 1299):
            s = starts[b] + t
            want, top = expected(qh[b, t], qw, 1e-6, s, f, m, interleaved)
            assert (np.abs(qg[b, t] - want) <= NEAR * top + (2**-8 if dtype == BF16 else 2**-24) * np.abs(want)).all()
            if s < 1280 and table[b, s // bs] >= 0:
                want, top = expected(kh[b, t], kw_, 1e-6, s, f, m, interleaved)
                assert (np.abs(kg[table[b, s // bs], :, s % bs] - want) <= NEAR * top + 2**-8 * np.abs(want)).all()
                assert np.array_equal(vg[table[b, s // bs], :, s % bs], vh[b, t])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128])
def test_sizes_of_all_kinds(D, dtype):
    """Heads whose squares leave fp32's range at either end; an infinity or a NaN stays with its head."""
    T, nh, nkv = 8, 8, 1
    q = torch.randn((1, T, nh, D), device=dev())
    for h, s in enumerate((1e38, 3e30, 1e19, 1e-15, 1e-25, 1e-38)):
        q[:, :, h] *= s / q[:, :, h].abs().amax()
    q[0, 3, 6, 5], q[0, 3, 7, 9] = math.inf, math.nan
    q = q.to(dtype)
    kc = torch.zeros((1, nkv, T, D), dtype=BF16, device=dev())
    got = host(mk.norm_rope_append(mk.Rope(D), mk.Cache([kc], [kc.clone()]), 0, q, q[:, :, :1].contiguous(), q[:, :, 6:7].contiguous(),
                                   None, None, ints([0]), eps=1e-12))
    f, m = ref.frequencies(D, 10000.0)
    qh = host(q)
    for t in range(T):
        want, top = expected(qh[0, t], None, 1e-12, t, f, m, False)
        for h in range(nh):
            if not np.isfinite(qh[0, t, h]).all():
                assert np.isnan(got[0, t, h]).any()
            else:  # (the smallest results are denormal numbers in bf16's and fp32's range alike: a step of 2^-133)
                near = NEAR * top[h] + (2**-8 if dtype == BF16 else 2**-24) * np.abs(want[h]) + 2.0**-133
                assert (np.abs(got[0, t, h] - want[h]) <= near).all(), (t, h)
        want, top = expected(qh[0, t, :1], None, 1e-12, t, f, m, False)
        assert (np.abs(host(kc)[0, :, t] - want) <= NEAR * top + 2**-8 * np.abs(want)).all()


def test_far_positions_and_scaling():
    D, bs, start = 128, 64, (1 << 20) + 12345
    for scaling in ("none", "yarn"):
        kw = dict(theta=500000.0, scaling=scaling, factor=1.0 if scaling == "none" else 8.0, low=1.0, high=4.0, original_length=8192)
        pool = torch.zeros((2, 1, bs, D), dtype=BF16, device=dev())
        table = torch.full((1, (start + 64) // bs + 1), -1, dtype=torch.int32, device=dev())
        table[0, start // bs] = 1
        q, kn = torch.randn((1, 2, 2, D), device=dev()), torch.randn((1, 2, 1, D), device=dev())
        got = host(mk.norm_rope_append(mk.Rope(D, **kw), mk.Cache([pool], [pool.clone()], table), 0, q, kn, kn, None, None, ints([start])))
        f, m = ref.frequencies(D, **kw)
        for t in range(2):
            want, top = expected(host(q[0, t]), None, 1e-6, start + t, f, m, False)
            assert (np.abs(got[0, t] - want) <= (NEAR + 2**-32) * top + 2**-24 * np.abs(want)).all()


def test_streams_graphs_and_repeats():
    rng = np.random.default_rng(0)
    B, T, nh, nkv, D = 4, 5, 8, 2, 128
    k, v, table = make_cache(rng, B, 100, nkv, D, 16)
    q, kn, vn = torch.randn((B, T, nh + 2 * nkv, D), device=dev()).to(BF16).split([nh, nkv, nkv], 2)
    qw, kw_ = weights(rng, D, "both")
    args = mk.Rope(D), mk.Cache(k, v, ints(table)), 0, q, kn, vn, qw, kw_, ints([3, 80, 17, 50]), ints(make_parents(rng, B, T))
    first = mk.norm_rope_append(*args)
    kept = [t.clone() for t in k + v]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = mk.norm_rope_append(*args, stream=side)
    side.synchronize()
    assert torch.equal(a, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mk.norm_rope_append(*args)
    for _ in range(3):
        out.zero_(), k[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    mk.norm_rope_append(*args)
    at = torch.tensor(sorted({int(x) for x in table.ravel()}), device=dev())
    written = (k[0][at] != 0).any(-1)
    assert torch.equal(k[0][at][written], kept[0][at][written]) and written.sum() == B * T * nkv


def test_binding_refusals():
    rng = np.random.default_rng(0)
    k, v, table = make_cache(rng, 2, 64, 2, 64, 16)
    c, rope, s = mk.Cache(k, v, ints(table)), mk.Rope(64), ints([5, 6])
    q = torch.randn((2, 3, 4, 64), device=dev()).to(BF16)
    kn = torch.randn((2, 3, 2, 64), device=dev()).to(BF16)
    w = torch.ones(64, device=dev(), dtype=BF16)
    call = mk.norm_rope_append
    bad = [lambda: call(rope, c, 0, q, kn, kn, w.float(), w, s), lambda: call(rope, c, 0, q, kn, kn, w, w[:32], s),
           lambda: call(rope, c, 0, q, kn, kn, w.cpu(), w, s), lambda: call(rope, c, 0, q, kn, kn, w, w[None], s),
           lambda: call(rope, c, 0, q, kn, kn, torch.ones(128, device=dev(), dtype=BF16)[::2], w, s),
           lambda: call(rope, c, 0, q, kn, kn, torch.ones(65, device=dev(), dtype=BF16)[1:], w, s),
           lambda: call(rope, c, 0, q, kn, kn, w, w, s, eps=0.0), lambda: call(rope, c, 0, q, kn, kn, w, w, s, eps=math.nan),
           lambda: call(rope, c, 0, q, kn, kn, w, w, s, eps=2.0), lambda: call(rope, c, 0, q, kn, kn.float(), w, w, s),
           lambda: call(mk.Rope(128), c, 0, q, kn, kn, w, w, s), lambda: call(rope, c, 2, q, kn, kn, w, w, s)]
    before = [t.clone() for t in k + v]
    for i, f in enumerate(bad):
        with pytest.raises(mk.MkError) as e:
            f()
        assert e.value.code == mk.MK_ERR_INVALID, i
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(k + v, before))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("nh,nkv,D", [(32, 8, 128), (7, 1, 64)])
def test_rows_of_a_block(nh, nkv, D, norm, dtype):
    """Blocks take one, two or four rows by the call's size (1023 to 4097 rows, heads above and below 8 KB a row): a
    row's values do not depend on it."""
    B, T = 3, 1366
    starts, counts = [5, 0, 40], [1366, 1001, 3]
    qkv = (torch.randn((B, T, nh + 2 * nkv, D), device=dev(), generator=torch.Generator(dev()).manual_seed(nh))).to(dtype)
    w = [torch.linspace(0.5, 2, D, device=dev()).to(BF16) for _ in range(2)]
    rope = mk.Rope(D, theta=500000.0)

    def run(parts):
        """(queries, k, v) by calls over runs of the sequences' rows"""
        k, v = ([torch.zeros((B, nkv, 1500, D), dtype=BF16, device=dev())] for _ in range(2))
        out = torch.full((B, T, nh, D), 77.0, device=dev(), dtype=dtype)
        cache = mk.Cache(k, v)
        for a, b in zip(parts, parts[1:]):
            x = qkv[:, a:b].contiguous()
            q, kn, vn = x.split([nh, nkv, nkv], 2)
            left = [min(max(c - a, 0), b - a) for c in counts]
            o = torch.full((B, b - a, nh, D), 77.0, device=dev(), dtype=dtype)
            rest = (ints([s + a for s in starts]), None, ints(left))
            if norm:
                mk.norm_rope_append(rope, cache, 0, q, kn, vn, *w, *rest, q_out=o)
            else:
                mk.rope_append(rope, cache, 0, q, kn, vn, *rest, q_out=o)
            out[:, a:b] = o
        return out, k[0], v[0]

    want = run(list(range(0, T, 341)) + [T])  # 1023 rows a call, 6 the last
    for parts in ([0, T], [0, 1365, T], [0, 342, 1024, T], [0, 683, T]):  # 4098 rows, 4095, 1026, 2046, 2049
        assert all(torch.equal(x, y) for x, y in zip(run(parts), want)), parts
