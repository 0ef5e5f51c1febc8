"""Sampled serving, the refusals of every entry point. Nothing is launched: a call with bad
arguments returns before it touches the device, so made-up pointers do."""
import ctypes

import pytest

from decode_megakernel_03_gb300 import build as mkbuild
from decode_megakernel_03_gb300 import mk
from tests.test_cache_ops_host import BAD_CACHES, BAD_TABLES, PTR, cache, refused, rope_args


@pytest.fixture(scope="module", autouse=True)
def L():
    mkbuild.build()
    return mk.lib()


def norm_args(c, rope=None, q_norm=PTR, k_norm=PTR, eps=1e-6, **kw):
    a = rope_args(c, rope, **kw)
    return [a[0], q_norm, k_norm, eps] + a[1:]


def prefix_args(c, **kw):
    a = dict(layer=1, batch=3, n=5, nh=4, type=0, scale=0.1, q=PTR, qs=256, groups=2, first=PTR, prefix=PTR,
             starts=PTR, parents=None, counts=None, out=PTR, os=256, ws=PTR, size=1 << 40, stream=None)
    a.update(kw)
    return [ctypes.byref(c) if c else None] + list(a.values())


def verify_args(**kw):
    a = dict(batch=3, n=5, vocab=100, type=1, logits=PTR, stride=100, draft_type=0, draft=PTR, draft_stride=100,
             temperature=PTR, tokens=PTR, parents=PTR, counts=None, uniform=PTR, noise=PTR, noise_stride=100, path=PTR,
             accepted=PTR, next=PTR, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", BAD_CACHES + BAD_TABLES)
def test_caches_refused(L, kw):
    c = cache(**dict(kw))
    assert refused(L, L.mk_norm_rope_append(*norm_args(c)))
    assert refused(L, L.mk_prefix_attention(*prefix_args(c)))
    size = ctypes.c_size_t()
    assert refused(L, L.mk_prefix_attention_workspace(ctypes.byref(c), 3, 5, 4, 0, 2, ctypes.byref(size)))


def test_null_arguments_refused(L):
    size = ctypes.c_size_t()
    assert refused(L, L.mk_norm_rope_append(*norm_args(None)))
    assert refused(L, L.mk_prefix_attention(*prefix_args(None)))
    assert refused(L, L.mk_prefix_attention_workspace(None, 1, 1, 2, 0, 1, ctypes.byref(size)))
    assert refused(L, L.mk_prefix_attention_workspace(ctypes.byref(cache()), 1, 1, 2, 0, 1, None))


@pytest.mark.parametrize("kw", [dict(q_norm=PTR + 8), dict(k_norm=PTR + 2), dict(eps=0.0), dict(eps=-1e-6), dict(eps=1e-31),
                                dict(eps=2.0), dict(eps=float("nan")), dict(layer=2), dict(layer=-1), dict(batch=0),
                                dict(batch=4), dict(n=0), dict(n=65), dict(nh=0), dict(nh=5000), dict(type=2), dict(q=None),
                                dict(k=None), dict(v=None), dict(out=None), dict(starts=None), dict(q=PTR + 4),
                                dict(out=PTR + 8), dict(qs=252), dict(ks=64), dict(vs=130), dict(os=258),
                                dict(parents=None, n=2**29), dict(rope=mk.MkRope())])
def test_norm_rope_refusals(L, kw):
    assert refused(L, L.mk_norm_rope_append(*norm_args(cache(), **kw)))


@pytest.mark.parametrize("kw", [dict(batch=0), dict(batch=4), dict(n=0), dict(n=65), dict(nh=3), dict(nh=0), dict(nh=18),
                                dict(type=-1), dict(layer=2), dict(layer=-1), dict(groups=0), dict(groups=-1), dict(groups=4),
                                dict(first=None), dict(prefix=None), dict(q=None), dict(out=None), dict(starts=None),
                                dict(ws=None), dict(ws=PTR + 128), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(q=PTR + 8), dict(out=PTR + 2), dict(qs=255), dict(qs=248),
                                dict(os=100)])
def test_prefix_attention_refusals(L, kw):
    assert refused(L, L.mk_prefix_attention(*prefix_args(cache(), **kw)))


def test_prefix_attention_refuses_more_work_than_it_can_count(L):
    # 1024 sequences of 64 nodes in 8 heads each over 2^27 keys: 8 x 1024 x 2^20 tiles
    c = cache(batch=1024, n_kv_heads=1, table_entries=1 << 23)
    assert refused(L, L.mk_prefix_attention(*prefix_args(c, batch=1024, n=64, nh=8, qs=512, os=512)))


@pytest.mark.parametrize("kw", [dict(type=2), dict(type=-1), dict(draft_type=3), dict(batch=0), dict(batch=1025), dict(n=0),
                                dict(n=65), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(stride=99), dict(draft_stride=99),
                                dict(noise_stride=99), dict(logits=PTR + 2), dict(draft=PTR + 1), dict(noise=PTR + 2),
                                dict(uniform=PTR + 2), dict(temperature=PTR + 1), dict(logits=None), dict(tokens=None),
                                dict(uniform=None), dict(noise=None), dict(path=None), dict(accepted=None), dict(next=None),
                                dict(parents=None, n=30000)])
def test_verify_refusals(L, kw):
    assert refused(L, L.mk_tree_verify(*verify_args(**kw)))


def test_binding_wants_device_tensors():
    import torch
    with pytest.raises(mk.MkError):
        mk.tree_verify(torch.zeros(1, 1, 8), torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, 1), torch.ones(1, 8))
