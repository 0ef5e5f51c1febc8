"""Attention over contexts so long that a block's part of one is many thousands of products: what
the sums lose on the way must not grow with the length. The pages of a long context are those of a
short one over and over, so that the 64-bit form needs the short one only."""
import pytest
import torch

from decode_megakernel_03_gb300 import mk

pytestmark = pytest.mark.gpu

POOL, PAGE, B, NKV = 8192, 64, 19, 8

# The matrix unit truncates as it accumulates: a product of 16 keys may lose 2^-22 of what has been
# summed before it. Both parts of a tile's weights are 16 such products, so that 32 tiles lose at most
# 32 x 16 x 2^-22 = 2^-13 of their sum where all values have one sign. Sums that are joined by rounded
# adds lose nothing on the average. So the outputs' mean, which has no rounding left in it (2^-9 at
# random, over 10^5 outputs and more), is held to twice that.
MEAN_BOUND = 2.0**-12
# By norm, values of both signs: against the 64-bit output rounded to bf16, as in
# test_gpu_tree_attention_precision.py, at any length.
NORM_BOUND = 2.0**-11


def case(op, keys, T, nh, D, mean):
    """(the call's outputs, the exact ones rounded to bf16) of three of the sequences."""
    g = torch.Generator(device="cuda").manual_seed(keys + T)
    new = lambda *s: torch.randn(s, generator=g, device="cuda")
    k = new(POOL // PAGE, NKV, PAGE, D).bfloat16()
    v = (new(POOL // PAGE, NKV, PAGE, D) * (0.3 if mean else 1) + mean).bfloat16()
    q = new(B, T, nh, D).bfloat16()
    entries = (keys + T + PAGE - 1) // PAGE
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = (torch.arange(entries, device="cuda", dtype=torch.int32) % (POOL // PAGE)).expand(B, -1).contiguous()
    cache, starts, roots = mk.Cache([k], [v], table), ints([keys] * B), ints([[-1] * T] * B)
    if op == "tree":
        out = mk.tree_attention(cache, 0, q, starts, roots)
    else:
        out = mk.prefix_attention(cache, 0, q, ints([0]), ints([keys]), starts, roots)
    times = torch.full((POOL,), keys // POOL, device="cuda", dtype=torch.float64)
    times[:keys % POOL] += 1
    flat = lambda x: x.transpose(0, 1).reshape(NKV, POOL, D).double()
    kk, vv, own = flat(k), flat(v), (keys + torch.arange(T, device="cuda")) % POOL
    got, want = [], []
    for b in (0, 7, B - 1):
        qq = q[b].reshape(T, NKV, nh // NKV, D).permute(1, 0, 2, 3).double()
        s = torch.einsum("htgd,hkd->htgk", qq, kk) * D**-0.5
        w = (s - s.amax(-1, keepdim=True)).exp()
        mine = w[:, torch.arange(T), :, own].permute(1, 0, 2)[..., None]  # a node sees itself, no other node
        w = w * times
        o = (torch.einsum("htgk,hkd->htgd", w, vv) + mine * vv[:, own][:, :, None]) / (w.sum(-1, keepdim=True) + mine)
        got.append(out[b].reshape(T, NKV, nh // NKV, D).permute(1, 0, 2, 3).double())
        want.append(o.bfloat16().double())
    return torch.stack(got), torch.stack(want)


# rows of a kv-head pick the kernel: 2, 8 and 16 the one for few rows, 32 one block of rows, 256 two; for
# a prefix the rows of all 19 sequences, 38, 152 and more
SHAPES = [("tree", 1, 16, 128), ("tree", 1, 64, 64), ("tree", 2, 64, 128), ("tree", 4, 64, 128), ("tree", 4, 64, 64),
          ("tree", 32, 64, 128), ("tree", 32, 64, 64), ("prefix", 1, 16, 128), ("prefix", 1, 64, 128),
          ("prefix", 1, 64, 64), ("prefix", 4, 64, 128)]


@pytest.mark.parametrize("op,T,nh,D", SHAPES)
@pytest.mark.parametrize("keys", [8192, 70001, 2**20 + 77])
def test_loss_does_not_grow(keys, op, T, nh, D):
    got, want = case(op, keys, T, nh, D, 0.0)
    off = ((got - want).norm() / want.norm()).item()
    assert off <= NORM_BOUND, f"{off:.3g}"
    got, want = case(op, keys, T, nh, D, 1.0)
    off = ((got - want).mean() / want.mean()).item()
    assert abs(off) <= MEAN_BOUND, f"{off:.3g}"


@pytest.mark.parametrize("way", ["rising", "falling", "first pages missing"])
@pytest.mark.parametrize("op,T,D", [("tree", 2, 128), ("tree", 4, 128), ("tree", 32, 64), ("tree", 32, 128), ("prefix", 4, 128),
                                    ("prefix", 4, 64)])
def test_reference_moves(op, T, D, way):
    """Scores that grow along the context (each part's largest is far above the last one's), fall, or begin
    behind the first 70 tiles."""
    keys, nh = 24576 - 64, 64
    seqs = 2 * B if T == 2 else B  # (the kernel for few rows has two blocks per SM)
    g = torch.Generator(device="cuda").manual_seed(T + D)
    new = lambda *s: torch.randn(s, generator=g, device="cuda")
    n = (keys + 64) // PAGE
    size = torch.linspace(0.1, 4, keys + 64, device="cuda")
    if way == "falling":
        size = size.flip(0)
    if way == "first pages missing":
        size[:] = 1
    k = (new(n, NKV, PAGE, D) * size.view(n, 1, PAGE, 1)).bfloat16()
    v = (new(n, NKV, PAGE, D) + 0.5).bfloat16()
    q = new(seqs, T, nh, D).bfloat16()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.arange(n, device="cuda", dtype=torch.int32)
    gone = 70 * 128 // PAGE if way == "first pages missing" else 0
    table[:gone] = -1
    cache, starts, roots = mk.Cache([k], [v], table.expand(seqs, n).contiguous()), ints([keys] * seqs), ints([[-1] * T] * seqs)
    if op == "tree":
        out = mk.tree_attention(cache, 0, q, starts, roots)
    else:  # (the sequences' own keys are the long part)
        out = mk.prefix_attention(cache, 0, q, ints([0]), ints([128]), starts, roots)
    flat = lambda x: x.transpose(0, 1).reshape(NKV, keys + 64, D).double()
    kk, vv = flat(k), flat(v)
    at, t = torch.arange(keys + 64, device="cuda"), torch.arange(T, device="cuda")
    seen = ((at < keys) & (at >= gone * PAGE)) | (at == keys + t[:, None])
    for b in (0, seqs - 1):
        qq = q[b].reshape(T, NKV, nh // NKV, D).permute(1, 0, 2, 3).double()
        s = torch.einsum("htgd,hkd->htgk", qq, kk) * D**-0.5
        w = torch.softmax(s.masked_fill(~seen[None, :, None], float("-inf")), -1)
        want = torch.einsum("htgk,hkd->htgd", w, vv).bfloat16().double()
        got = out[b].reshape(T, NKV, nh // NKV, D).permute(1, 0, 2, 3).double()
        off = ((got - want).norm() / want.norm()).item()
        assert off <= NORM_BOUND, f"{off:.3g}"
