"""Page tables on the host (mk_pages_*): against a plain model that keeps every
sequence's contents, through random growing, shrinking, forking and compacting;
refusals leave everything as it was."""
import ctypes

import numpy as np
import pytest

from decode_megakernel_03_gb300 import build as mkbuild
from decode_megakernel_03_gb300 import mk


@pytest.fixture(scope="module", autouse=True)
def L():
    mkbuild.build()
    return mk.lib()


def state(p):
    return p.table().copy(), p.lengths().copy(), p.n_free()


class Contents:
    """What a cache would hold: pool[block][row], written through the tables."""

    def __init__(self, n_blocks, bs):
        self.pool, self.bs = np.full((n_blocks, bs), -1, np.int64), bs

    def copy(self, copies):
        assert len(set(copies[:, 1])) == len(copies) and not set(copies[:, 1]) & set(copies[:, 0])
        for s, d, r in copies:
            self.pool[d, :r] = self.pool[s, :r]

    def write(self, table, s, at, value):
        self.pool[table[s, at // self.bs], at % self.bs] = value

    def read(self, table, s, n):
        return [self.pool[table[s, i // self.bs], i % self.bs] for i in range(n)]


@pytest.mark.parametrize("bs,cap,n_blocks", [(1, 9, 60), (4, 30, 40), (5, 23, 30), (16, 64, 20)])
def test_random_histories(bs, cap, n_blocks):
    rng = np.random.default_rng(bs)
    n_seqs = 6
    p, c = mk.Pages(n_blocks, bs, n_seqs, cap), Contents(n_blocks, bs)
    want = [[] for _ in range(n_seqs)]
    mark = 0
    for _ in range(400):
        before = state(p)
        kind = rng.integers(5)
        if kind <= 2:
            seqs = rng.permutation(n_seqs)[:rng.integers(1, 4)]
            lens = [int(rng.integers(0, cap + 1)) if kind else min(cap, len(want[s]) + 1) for s in seqs]
            try:
                copies = p.resize(seqs, lens)
            except mk.MkError as e:
                assert e.code == mk.MK_ERR_OOM
                for a, b in zip(before, state(p)):
                    assert np.array_equal(a, b)
                continue
            c.copy(copies)
            t = p.table()
            for s, n in zip(seqs, lens):
                for i in range(len(want[s]), n):
                    mark += 1
                    want[s].append(mark)
                    c.write(t, s, i, mark)
                del want[s][n:]
        elif kind == 3:
            empty = [s for s in range(n_seqs) if not want[s]]
            full = [s for s in range(n_seqs) if want[s]]
            if empty and full:
                kids = empty[:2]
                par = [full[rng.integers(len(full))] for _ in kids]
                p.fork(par, kids)
                for a, k in zip(par, kids):
                    want[k] = list(want[a])
        else:
            c.copy(p.compact())
            used = {x for x in p.table().ravel() if x >= 0}
            assert used == set(range(len(used)))
        t, n, free = state(p)
        assert list(n) == [len(w) for w in want]
        assert free == n_blocks - len({x for x in t.ravel() if x >= 0})
        for s in range(n_seqs):
            k = -(-len(want[s]) // bs)
            assert (t[s, :k] >= 0).all() and (t[s, k:] == -1).all()
            assert c.read(t, s, len(want[s])) == want[s]
    assert mark > 100


def test_lowest_page_first_and_copy_on_write():
    p = mk.Pages(10, 4, 4, 16)
    p.resize([0, 1], [6, 4])
    assert p.table()[0, :2].tolist() == [0, 1] and p.table()[1, 0] == 2
    p.fork([0], [2])
    assert p.n_free() == 7
    assert p.resize([2], [7]).tolist() == [[1, 3, 2]]       # the shared half-full page
    assert p.resize([0], [7]).tolist() == []                # no longer shared
    p.resize([1], [0])
    p.fork([0], [3])
    assert p.resize([3], [8]).tolist() == [[1, 2, 3]]       # page 2 is the lowest free one
    p.fork([2], [1])
    # one call: 2 lets go of page 3 by shrinking, so 1 need not copy it
    assert p.resize([2, 1], [0, 8]).tolist() == []
    assert p.resize([], []).shape == (0, 3)


def test_a_page_that_a_copy_reads_is_not_free_in_the_same_call():
    p = mk.Pages(7, 4, 4, 16)
    p.resize([0, 1], [6, 6])
    p.fork([0, 1], [2, 3])
    # 0 copies page 1, 2 then lets go of it, 1 needs a page for its own copy
    assert p.resize([0, 2, 1], [7, 0, 7]).tolist() == [[1, 4, 2], [3, 5, 2]]
    assert p.n_free() == 2 and p.resize([2], [8]).tolist() == []
    assert p.table()[2, :2].tolist() == [1, 6]  # free again in the next call
    p = mk.Pages(5, 4, 4, 16)  # the same without a page for it
    p.resize([0, 1], [6, 6])
    p.fork([0, 1], [2, 3])
    before = state(p)
    with pytest.raises(mk.MkError) as e:
        p.resize([0, 2, 1], [7, 0, 7])
    assert e.value.code == mk.MK_ERR_OOM
    for a, b in zip(before, state(p)):
        assert np.array_equal(a, b)
    assert p.resize([0, 2], [7, 0]).tolist() == [[1, 4, 2]]
    assert p.resize([1], [7]).tolist() == [[3, 1, 2]]


def test_full_pages_are_shared_without_a_copy():
    p = mk.Pages(8, 4, 3, 16)
    p.resize(0, 8)
    p.fork([0, 0], [1, 2])
    assert p.resize([0, 1, 2], [9, 9, 9]).tolist() == []
    t = p.table()
    assert (t[:, :2] == t[0, :2]).all() and len(set(t[:, 2])) == 3


def test_refusals():
    p = mk.Pages(4, 4, 3, 12)
    p.resize(0, 7)
    before = state(p)
    for call in (lambda: p.resize([3], [1]), lambda: p.resize([-1], [1]),
                 lambda: p.resize([1], [13]), lambda: p.resize([1], [-1]),
                 lambda: p.resize([1, 1], [1, 2]), lambda: p.resize([1, 2], [1]),
                 lambda: p.fork([0], [0]), lambda: p.fork([1], [0]), lambda: p.fork([0, 0], [1, 1]),
                 lambda: p.fork([0, 1], [1, 2]), lambda: p.fork([0], [3])):
        with pytest.raises(mk.MkError) as e:
            call()
        assert e.value.code == mk.MK_ERR_INVALID
    with pytest.raises(mk.MkError) as e:
        p.resize([1, 2], [5, 4])  # three pages of two free ones
    assert e.value.code == mk.MK_ERR_OOM
    for a, b in zip(before, state(p)):
        assert np.array_equal(a, b)
    for args in ((0, 4, 1, 4), (4, 0, 1, 4), (4, 4, 0, 4), (4, 4, 1, 0), (4, 4, 1, 2**31 - 2)):
        with pytest.raises(mk.MkError):
            mk.Pages(*args)


def test_small_copy_lists_are_refused(L):
    p = mk.Pages(8, 4, 3, 8)
    p.resize([0, 1], [8, 6])
    p.fork([1], [2])
    p.resize([0], [0])
    n, one = ctypes.c_int(7), (ctypes.c_int32 * 3)()
    seq, length = (ctypes.c_int32 * 1)(2), (ctypes.c_int32 * 1)(7)
    assert L.mk_pages_resize(p.h, 1, seq, length, None, 0, ctypes.byref(n)) == mk.MK_ERR_INVALID
    assert L.mk_pages_compact(p.h, one, 1, ctypes.byref(n)) == mk.MK_ERR_INVALID and n.value == 2
    assert L.mk_pages_compact(p.h, None, 2, ctypes.byref(n)) == mk.MK_ERR_INVALID
    assert p.table()[2, :2].tolist() == [2, 3] and p.lengths()[2] == 6
    assert p.compact().tolist() == [[2, 0, 4], [3, 1, 4]]
    for f in (L.mk_pages_read, ):
        assert f(None, None, None, None) == mk.MK_ERR_INVALID
    assert L.mk_pages_fork(None, 0, None, None) == mk.MK_ERR_INVALID
    assert L.mk_pages_destroy(None) == mk.MK_OK
