"""What is no tensor, or a tensor of another library, is refused by every operator of the binding with
MkError, argument by argument."""
import types

import numpy as np
import pytest
import torch

from decode_megakernel_03_gb300 import build as mkbuild
from decode_megakernel_03_gb300 import mk

NO_TENSORS = [None, 1.0, [1, 2], np.zeros((2, 3), np.float32), "x"]


def refused(f, args, name, value):
    with pytest.raises(mk.MkError) as e:
        f(**{**args, name: value})
    assert e.value.code == mk.MK_ERR_INVALID


def calls(device, cache, rope):
    """(operator, its arguments, which of them must be there, which may be left out)"""
    new = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device=device)
    i32 = lambda *s: new(*s, d=torch.int32)
    q, k = new(2, 3, 4, 64), new(2, 3, 2, 64)
    rows = dict(starts=i32(2), parents=i32(2, 3), counts=i32(2))
    append = dict(rope=rope, cache=cache, layer=0, q=q, k=k, v=k, **rows)
    return [(mk.rope_append, append, ["q", "k", "v", "starts"], ["parents", "counts", "q_out"]),
            (mk.norm_rope_append, dict(append, q_norm=new(64, d=torch.bfloat16), k_norm=new(64, d=torch.bfloat16)),
             ["q", "k", "v", "starts"], ["parents", "counts", "q_norm", "k_norm", "q_out"]),
            (mk.tree_attention, dict(cache=cache, layer=0, q=q, **rows), ["q", "starts"], ["parents", "counts", "out"]),
            (mk.prefix_attention, dict(cache=cache, layer=0, q=q, first=i32(1), prefix=i32(1), **rows),
             ["q", "first", "prefix", "starts"], ["parents", "counts", "out"]),
            (mk.tree_accept, dict(logits=new(2, 3, 9), tokens=i32(2, 3)), ["logits", "tokens"], ["parents", "counts"]),
            (mk.tree_verify, dict(logits=new(2, 3, 9), tokens=i32(2, 3), uniform=new(2, 3), noise=new(2, 9)),
             ["logits", "tokens", "uniform", "noise"], ["parents", "counts", "draft", "temperature"]),
            (mk.cache_compact, dict(cache=cache, starts=i32(2), path=i32(2, 3), accepted=i32(2)),
             ["starts", "path", "accepted"], [])]


def test_before_the_library(monkeypatch):
    """Without a GPU: what the binding itself says, up to the first call of the library."""
    mkbuild.build()
    mk._use_torch()
    monkeypatch.setattr(mk, "_elsewhere", lambda device, stream: None)
    monkeypatch.setattr(mk, "_current_raw", lambda index: 0)
    logits = mk._logits
    monkeypatch.setattr(mk, "_logits", lambda t: (t.device, t.shape) if isinstance(t, torch.Tensor) else logits(t))
    cpu = torch.device("cpu")
    cache = types.SimpleNamespace(device=cpu, n_kv_heads=2, head_dim=64, workspaces={}, ref=None)
    for f, args, needed, optional in calls(cpu, cache, mk.Rope(64)):
        for name in needed + optional:
            for value in NO_TENSORS:
                # (a tensor that must be there and is None is refused by the library, where the binding does not look into it)
                if value is None and (name in optional or name not in ("q", "k", "v", "first", "logits", "noise", "path")):
                    continue
                refused(f, args, name, value)


@pytest.mark.gpu
def test_on_the_gpu():
    dev = torch.device("cuda", 0)
    k = [torch.zeros((2, 2, 8, 64), dtype=torch.bfloat16, device=dev)]
    for f, args, needed, optional in calls(dev, mk.Cache(k, [k[0].clone()]), mk.Rope(64)):
        for name in needed + optional:
            for value in NO_TENSORS:
                if value is not None or name in needed:
                    refused(f, args, name, value)
        f(**args)  # as it stands it is a call
    torch.cuda.synchronize()
