"""What mk_tree_attention keeps of its values, against 64 bits, on each of its
kernels: an error by norm, which a lost part of a query or weight exceeds (the
elementwise bounds of test_gpu_cache_ops.py add up worst cases and cannot see
one). tests/test_precision_bounds.py shows that these bounds do see it."""
import numpy as np
import pytest
import torch

from decode_megakernel_03_gb300 import mk
from tests import cache_ops_ref as ref
from tests.test_gpu_cache_ops import BF16, FP32, dev, host, ints, make_cache, make_parents

pytestmark = pytest.mark.gpu

# Scores of randn values over 1 / sqrt(D) are of size 1, so that their fp32 sums (D
# products, 2^-24 each as they add up at random: sqrt(128) x 2^-24 = 2^-20.5) and the
# exponential (2^-22) leave weights off by about 2^-20.2 at worst, at random: 8e-7 of
# the output's norm. fp32's own rounding is 2^-24. So 1e-6, and a value of two bf16
# parts (2^-17) is beyond it.
FP32_BOUND = 1e-6
# bf16 calls: against the 64-bit output rounded to bf16. Weights of two parts are
# off by 2^-16 at most, so the output by less than 2^-17 of itself by norm, and an
# element differs only where that crosses a border between two bf16 values: a
# share 2^-17 / step of them, by a step (up to 2^-7), sqrt(2^-17 x 2^-7) = 2^-12 by
# norm. Twice that; weights of one part (2^-9) give 2^-9.
BF16_BOUND = 2.0**-11

# (nodes, heads, kv heads, D, type): rows of a kv-head pick the kernel
KERNELS = [(1, 4, 2, 64, BF16), (4, 8, 2, 128, BF16), (5, 32, 8, 64, BF16), (20, 8, 2, 128, BF16),
           (40, 16, 4, 64, BF16), (60, 8, 2, 128, BF16),
           (3, 4, 2, 64, FP32), (8, 4, 2, 64, FP32), (14, 4, 2, 64, FP32), (1, 4, 2, 128, FP32),
           (8, 8, 2, 128, FP32), (50, 8, 2, 64, FP32), (36, 8, 2, 128, FP32)]


@pytest.mark.parametrize("T,nh,nkv,D,dtype", KERNELS)
@pytest.mark.parametrize("starts", [[130, 700], [20003, 31]])
def test_error_by_norm(starts, T, nh, nkv, D, dtype):
    rng = np.random.default_rng(T + D)
    k, v, table = make_cache(rng, 2, max(starts) + T, nkv, D, 16)
    par = make_parents(rng, 2, T)
    g = torch.Generator(device=dev()).manual_seed(11)
    q = torch.randn((2, T, nh, D), generator=g, device=dev()).to(dtype)
    got = mk.tree_attention(mk.Cache(k, v, ints(table)), 0, q, ints(starts), ints(par))
    want = ref.attention(host(q), host(k[0]), host(v[0]), table, np.asarray(starts), par, None, D**-0.5)[0]
    if dtype == BF16:
        want = host(torch.from_numpy(want).to(BF16))
    for b in range(2):
        off = np.linalg.norm(host(got[b]) - want[b]) / np.linalg.norm(want[b])
        assert off <= (BF16_BOUND if dtype == BF16 else FP32_BOUND), f"sequence {b}: {off:.3g}"
