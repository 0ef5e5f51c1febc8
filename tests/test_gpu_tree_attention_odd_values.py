"""NaN and infinities in the v rows of drafted nodes where a block takes many
sequences one after another: they reach the rows that see them, in their own
columns, and no row of a sequence before or behind. On each kernel of
mk_tree_attention."""
import numpy as np
import pytest
import torch

from decode_megakernel_03_gb300 import mk
from tests import cache_ops_ref as ref
from tests.test_gpu_cache_ops import BF16, FP32, dev, ints, make_cache, make_parents

pytestmark = pytest.mark.gpu

# (nodes, D, type), 4 query heads to a kv-head: rows up to 16, 32, 128 and above
KERNELS = [(3, 64, BF16), (3, 128, BF16), (3, 64, FP32), (12, 64, BF16), (12, 128, BF16), (40, 64, BF16),
           (40, 128, BF16), (3, 128, FP32), (6, 64, FP32), (6, 128, FP32), (20, 64, FP32), (20, 128, FP32)]


@pytest.mark.parametrize("T,D,dtype", KERNELS)
@pytest.mark.parametrize("ends", [0.0, 0.7])
def test_odd_values_among_many_sequences(ends, T, D, dtype):
    """ends: the share of sequences whose context fills the cache, so that no node
    of theirs is there."""
    rng = np.random.default_rng(T + D)
    B, nkv, G, room = 500, 2, 4, 128
    k, v, table = make_cache(rng, B, room, nkv, D, 16)
    par = make_parents(rng, B, T, "odd")
    starts = rng.integers(0, room - T + 1, B)
    starts[rng.random(B) < ends] = room
    counts = rng.integers(1, T + 1, B)
    g = torch.Generator(device=dev()).manual_seed(3)
    q = torch.randn((B, T, nkv * G, D), generator=g, device=dev()).to(dtype)
    cache = mk.Cache(k, v, ints(table))
    args = (cache, 0, q, ints(starts), ints(par), ints(counts))
    clean = mk.tree_attention(*args).clone()
    assert clean.isfinite().all()
    want = clean.clone()
    for b in np.flatnonzero((rng.random(B) < 0.6) & (starts < room)):
        node, d = int(rng.integers(counts[b])), int(rng.integers(D))
        x = float(rng.choice([np.inf, -np.inf, np.nan]))
        s = starts[b] + node
        v[0][int(table[b, s // 16]), :, s % 16, d] = x
        rows = [t for t in range(counts[b]) if node in ref.family(par, b, t)]
        want[b, rows, :, d] = x
    assert (~want.isfinite()).any(dim=(1, 2, 3)).sum() > 50
    for _ in range(10):
        assert torch.equal(mk.tree_attention(*args).nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))
