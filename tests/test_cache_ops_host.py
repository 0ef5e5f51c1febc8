"""Operators over a KV cache, what the host decides: rotary plans against the
formulas, and the refusals of every entry point. Nothing is launched: a call
with bad arguments returns before it touches the device, so made-up pointers do."""
import ctypes
import math

import numpy as np
import pytest

from decode_megakernel_03_gb300 import build as mkbuild
from decode_megakernel_03_gb300 import mk
from tests import cache_ops_ref as ref


@pytest.fixture(scope="module", autouse=True)
def L():
    mkbuild.build()
    return mk.lib()


ROPES = [dict(), dict(rotary_dim=32, interleaved=True, theta=500000.0),
         dict(scaling="linear", factor=4.0), dict(rotary_dim=60, scaling="linear", factor=1.5),
         dict(theta=500000.0, scaling="bands", factor=8.0, low=1.0, high=4.0, original_length=8192),
         dict(scaling="yarn", factor=16.0, low=1.0, high=32.0, original_length=4096),
         dict(scaling="yarn", factor=2.0, low=1.0, high=32.0, original_length=7),
         dict(scaling="yarn", factor=2.0, low=1.0, high=32.0, original_length=2048, magnitude=1.0)]


@pytest.mark.parametrize("kw", ROPES)
@pytest.mark.parametrize("d", [64, 128])
def test_rope_plan(d, kw):
    r = mk.Rope(d, **kw).struct
    n = kw.get("rotary_dim", d)
    f, m = ref.frequencies(n, **{"theta": 10000.0, **{k: v for k, v in kw.items()
                                                      if k not in ("rotary_dim", "interleaved", "magnitude")}})
    assert (r.head_dim, r.rotary_dim, r.interleaved) == (d, n, int(kw.get("interleaved", False)))
    assert r.magnitude == np.float32(kw.get("magnitude", m))
    # fp64 on both sides: a few roundings of 2^-53
    for i, x in enumerate(f):
        assert r.turns[i] / 2.0**64 * 2 * math.pi == pytest.approx(x, rel=1e-14)
    assert all(r.turns[i] == 0 for i in range(n // 2, 64))


@pytest.mark.parametrize("d,kw", [(96, {}), (64, dict(rotary_dim=63)), (64, dict(rotary_dim=66)),
                                  (64, dict(rotary_dim=0)), (64, dict(theta=0.5)),
                                  (64, dict(theta=float("nan"))), (64, dict(factor=0.5)),
                                  (64, dict(scaling="bands")), (64, dict(scaling="cubic")),
                                  (64, dict(scaling="bands", original_length=9, low=4.0, high=1.0)),
                                  (64, dict(scaling="yarn", original_length=9, theta=1.0)),
                                  (64, dict(magnitude=float("inf"))), (64, dict(magnitude=0.0))])
def test_rope_refusals(d, kw):
    with pytest.raises(mk.MkError) as e:
        mk.Rope(d, **kw)
    assert e.value.code == mk.MK_ERR_INVALID


PTR = 0x10000  # never followed


def cache(**kw):
    n = kw.pop("layers", 2)
    k = (ctypes.c_void_p * max(n, 1))(*[kw.pop("at", PTR)] * max(n, 1))
    f = dict(n_layers=n, n_kv_heads=2, head_dim=64, n_blocks=9, block_size=16, batch=3,
             table_entries=4, block_table=PTR, k=ctypes.cast(k, mk._vpp), v=ctypes.cast(k, mk._vpp))
    f.update(kw)
    c = mk.MkCache(**f)
    c.keep = k
    return c


BAD_CACHES = [dict(head_dim=96), dict(layers=0), dict(n_layers=65), dict(n_kv_heads=0),
              dict(n_blocks=0), dict(block_size=0), dict(k=None), dict(v=None), dict(at=PTR + 8),
              dict(at=None), dict(n_blocks=2**31 - 1, block_size=2**10)]
BAD_TABLES = [dict(batch=2), dict(table_entries=0), dict(block_table=PTR + 2),
              dict(block_table=None), dict(block_table=None, table_entries=0, n_blocks=2),
              dict(table_entries=2**30)]


def rope_args(c, rope=None, **kw):
    a = dict(rope=rope or mk.Rope(64).struct, c=c, layer=1, batch=3, n=5, nh=4, type=1, q=PTR,
             qs=256, k=PTR, ks=128, v=PTR, vs=128, out=PTR, os=256, starts=PTR, parents=PTR,
             counts=None, stream=None)
    a.update(kw)
    ref_ = [ctypes.byref(a["rope"]) if a["rope"] else None, ctypes.byref(c) if c else None]
    return ref_ + [a[x] for x in list(a)[2:]]


def attention_args(c, **kw):
    a = dict(layer=1, batch=3, n=5, nh=4, type=0, scale=0.1, q=PTR, qs=256, starts=PTR,
             parents=None, counts=None, out=PTR, os=256, ws=PTR, size=1 << 40, stream=None)
    a.update(kw)
    return [ctypes.byref(c) if c else None] + list(a.values())


def accept_args(**kw):
    a = dict(batch=3, n=5, vocab=100, type=1, logits=PTR, stride=100, tokens=PTR, parents=PTR,
             counts=None, choices=PTR, path=PTR, accepted=PTR, next=PTR, ws=PTR, size=1 << 40,
             stream=None)
    a.update(kw)
    return list(a.values())


def compact_args(c, **kw):
    a = dict(batch=3, n=5, starts=PTR, path=PTR, accepted=PTR, stream=None)
    a.update(kw)
    return [ctypes.byref(c) if c else None] + list(a.values())


def refused(L, rc):
    return rc == mk.MK_ERR_INVALID and len(L.mk_last_error(None)) > 5


@pytest.mark.parametrize("kw", BAD_CACHES + BAD_TABLES)
def test_caches_refused(L, kw):
    c = cache(**dict(kw))
    assert refused(L, L.mk_rope_append(*rope_args(c)))
    assert refused(L, L.mk_tree_attention(*attention_args(c)))
    assert refused(L, L.mk_cache_compact(*compact_args(c)))
    if kw in BAD_CACHES:
        one = (ctypes.c_int32 * 3)(0, 1, 4)
        assert refused(L, L.mk_cache_copy_blocks(ctypes.byref(c), one, 1, None))


def test_null_caches_refused(L):
    assert refused(L, L.mk_rope_append(*rope_args(None)))
    assert refused(L, L.mk_tree_attention(*attention_args(None)))
    assert refused(L, L.mk_cache_compact(*compact_args(None)))
    assert refused(L, L.mk_cache_copy_blocks(None, None, 0, None))
    size = ctypes.c_size_t()
    assert refused(L, L.mk_tree_attention_workspace(None, 1, 1, 1, 0, ctypes.byref(size)))
    assert refused(L, L.mk_tree_attention_workspace(ctypes.byref(cache()), 1, 1, 2, 0, None))
    assert refused(L, L.mk_tree_accept_workspace(1, 1, 10, None))


@pytest.mark.parametrize("kw", [dict(layer=2), dict(layer=-1), dict(batch=0), dict(batch=4),
                                dict(n=0), dict(n=65), dict(nh=0), dict(nh=5000), dict(type=2),
                                dict(q=None), dict(k=None), dict(v=None), dict(out=None),
                                dict(starts=None), dict(q=PTR + 4), dict(out=PTR + 8),
                                dict(qs=252), dict(ks=64), dict(vs=130), dict(os=258),
                                dict(parents=None, n=2**29)])
def test_rope_append_refusals(L, kw):
    assert refused(L, L.mk_rope_append(*rope_args(cache(), **kw)))


def test_rope_append_wants_its_plan(L):
    a = rope_args(cache())
    assert refused(L, L.mk_rope_append(None, *a[1:]))
    assert refused(L, L.mk_rope_append(*rope_args(cache(), mk.Rope(128).struct)))
    assert refused(L, L.mk_rope_append(*rope_args(cache(), mk.MkRope())))


@pytest.mark.parametrize("kw", [dict(batch=0), dict(batch=4), dict(n=0), dict(n=65), dict(nh=3),
                                dict(nh=0), dict(nh=18), dict(type=-1), dict(layer=2),
                                dict(layer=-1), dict(q=None), dict(out=None), dict(starts=None),
                                dict(ws=None), dict(ws=PTR + 128), dict(scale=0.0),
                                dict(scale=-1.0), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(q=PTR + 8), dict(out=PTR + 2),
                                dict(qs=255), dict(qs=248), dict(os=100)])
def test_attention_refusals(L, kw):
    assert refused(L, L.mk_tree_attention(*attention_args(cache(), **kw)))


@pytest.mark.parametrize("kw", [dict(type=2), dict(batch=0), dict(batch=1025), dict(n=0),
                                dict(n=65), dict(vocab=0), dict(stride=99), dict(logits=PTR + 2),
                                dict(logits=None), dict(tokens=None), dict(choices=None),
                                dict(path=None), dict(accepted=None), dict(next=None),
                                dict(ws=None), dict(ws=PTR + 16), dict(size=8),
                                dict(parents=None, n=30000)])
def test_accept_refusals(L, kw):
    assert refused(L, L.mk_tree_accept(*accept_args(**kw)))


@pytest.mark.parametrize("kw", [dict(batch=0), dict(batch=4), dict(n=0), dict(n=65),
                                dict(starts=None), dict(path=None), dict(accepted=None)])
def test_compact_refusals(L, kw):
    assert refused(L, L.mk_cache_compact(*compact_args(cache(), **kw)))


@pytest.mark.parametrize("copies", [[(9, 0, 1)], [(0, 9, 1)], [(-1, 0, 1)], [(0, -1, 1)],
                                    [(0, 1, 17)], [(0, 1, -1)], [(0, 1, 4), (2, 1, 4)],
                                    [(0, 1, 4), (1, 2, 4)], [(3, 3, 4)], [(0, 1, 0), (2, 1, 0)]])
def test_copies_refused(L, copies):
    flat = (ctypes.c_int32 * (3 * len(copies)))(*[x for c in copies for x in c])
    assert refused(L, L.mk_cache_copy_blocks(ctypes.byref(cache()), flat, len(copies), None))


def test_copy_list_arguments(L):
    c = cache()
    assert refused(L, L.mk_cache_copy_blocks(ctypes.byref(c), None, 1, None))
    assert refused(L, L.mk_cache_copy_blocks(ctypes.byref(c), None, -1, None))
    assert L.mk_cache_copy_blocks(ctypes.byref(c), None, 0, None) == mk.MK_OK


def test_binding_wants_device_tensors():
    import torch
    t = torch.zeros((2, 2, 4, 64), dtype=torch.bfloat16)
    for args in (([t], [t]), ([], []), ([t], [t, t])):
        with pytest.raises(mk.MkError):
            mk.Cache(*args)
    with pytest.raises(mk.MkError):
        mk.tree_accept(torch.zeros(1, 1, 8), torch.zeros((1, 1), dtype=torch.int32))
