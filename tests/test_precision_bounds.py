"""The bounds that test_gpu_tree_attention_precision.py puts on mk_tree_attention hold
for its arithmetic as written out here, and not for the same with a part of the
queries or of the weights left out."""
import re
from pathlib import Path

import numpy as np
import pytest
import torch

HERE = Path(__file__).parent


def bound(name):
    text = (HERE / "test_gpu_tree_attention_precision.py").read_text()
    return float(eval(re.search(rf"^{name} = (.+)$", text, re.M).group(1)))


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16).double().numpy()


def parts(x, n):
    """x (of fp32) as the sum of n bf16 parts, each the rounded rest."""
    out, rest = np.zeros_like(x), x.copy()
    for _ in range(n):
        p = bf16(rest)
        out, rest = out + p, rest - p
    return out


def case(n, d, seed):
    r = np.random.default_rng(seed)
    k, v = bf16(r.standard_normal((n, d))), bf16(r.standard_normal((n, d)))
    return r.standard_normal((6, d)).astype(np.float32).astype(np.float64), k, v


def attend(q, k, v, q_parts, w_parts):
    s = parts(q, q_parts) @ k.T / np.sqrt(q.shape[1])
    w = np.exp(s - s.max(-1, keepdims=True))
    return (parts(w.astype(np.float32).astype(np.float64), w_parts) @ v) / w.sum(-1, keepdims=True)


def by_norm(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("n,d", [(130, 64), (2540, 128), (20003, 64)])
def test_fp32_bound_sees_a_lost_part(n, d):
    q, k, v = case(n, d, n)
    exact = attend(q, k, v, 9, 9)
    assert by_norm(attend(q, k, v, 3, 3), exact) <= bound("FP32_BOUND")
    for q_parts, w_parts in ((2, 3), (3, 2), (3, 1), (1, 3)):
        assert by_norm(attend(q, k, v, q_parts, w_parts), exact) > bound("FP32_BOUND"), (q_parts, w_parts)


@pytest.mark.parametrize("n,d", [(130, 64), (2540, 128), (20003, 64)])
def test_bf16_bound_sees_a_lost_part(n, d):
    q, k, v = case(n, d, n + 1)
    q = bf16(q)
    exact = bf16(attend(q, k, v, 1, 9))
    assert by_norm(bf16(attend(q, k, v, 1, 2)), exact) <= bound("BF16_BOUND")
    assert by_norm(bf16(attend(q, k, v, 1, 1)), exact) > bound("BF16_BOUND")
