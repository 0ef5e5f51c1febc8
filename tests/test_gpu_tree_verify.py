"""Verification by rejection sampling against its plain 64-bit form, and its distribution."""
import itertools
import math

import numpy as np
import pytest
import torch

from decode_megakernel_03_gb300 import mk
from tests import sampling_ref as ref

BF16, FP32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu

# A probability is the exponential of (l - top) / temperature (in powers of two: two roundings of
# at most 64, the exponential's own 2^-22), over a sum of V weights (up to 128 adds of a thread in
# a row, 2^-24 each, and a tree of 10): 64 x 2^-23 + 2^-22 + 140 x 2^-24 < 2^-16.3, the sum of a
# residual the same of what it adds and takes away. Comparisons closer than 2^-15 of what is
# compared may fall either way; the inputs below have none (test_inputs_are_clear).
CLEAR = 2.0**-15


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dtype)


def make(seed, B, T, V, dtype=FP32, draft=None, parents="tree", counts=None, temperature=False, luck=0.7):
    """Inputs on the host: a target that is a noisy form of the drafter, tokens drawn from the drafter."""
    rng = np.random.default_rng(seed)
    par = None
    if parents is not None:
        par = np.full((B, T), -1, np.int32)
        for t in range(1, T):
            par[:, t] = rng.integers(max(0, t - 4), t, B) if parents == "tree" else rng.integers(-2, t + 2, B)
    base = rng.normal(size=(B, T, V)) * 2
    q = np.exp(base - base.max(-1, keepdims=True))
    q /= q.sum(-1, keepdims=True)
    tokens = np.zeros((B, T), np.int32)
    for b, t in itertools.product(range(B), range(T)):
        up = max(0, t - 1) if par is None else max(0, min(int(par[b, t]), T - 1))
        tokens[b, t] = np.argmax(q[b, up] / rng.exponential(size=V))
        if draft is None and rng.random() < luck:  # a sure drafter is right about these
            base[b, up, tokens[b, t]] += 5
    logits = rounded(base + 0.7 * rng.normal(size=base.shape), dtype)
    return dict(logits=logits, tokens=tokens, uniform=rng.random((B, T)).astype(np.float32),
                noise=np.maximum(rng.exponential(size=(B, V)), 1e-30).astype(np.float32), parents=par, counts=counts,
                draft=None if draft is None else rounded(q, draft),
                temperature=(0.5 + rng.random(B)).astype(np.float32) if temperature else None)


def expected(a):
    f = lambda x: None if x is None else x.double().numpy()
    return ref.verify(f(a["logits"]), a["tokens"], a["uniform"].astype(float), a["noise"].astype(float), a["parents"],
                      a["counts"], f(a["draft"]), None if a["temperature"] is None else a["temperature"].astype(float))


def on_device(a):
    def move(x, name):
        if x is None:
            return None
        t = x if torch.is_tensor(x) else torch.from_numpy(np.asarray(x))
        return (t.to(torch.int32) if name in ("tokens", "parents", "counts") else t).cuda()
    return {n: move(x, n) for n, x in a.items()}


def call(d, **kw):
    return mk.tree_verify(d["logits"], d["tokens"], d["uniform"], d["noise"], d["parents"], d["counts"], d["draft"],
                          d["temperature"], **kw)


def check(a, want=None):
    d = on_device(a)
    got = call(d)
    want = want or expected(a)
    for g, w, name in zip(got, want, ("path", "accepted", "next")):
        assert np.array_equal(g.cpu().numpy(), w), name
    return d, got


CASES = [dict(seed=i, B=B, T=T, V=V, dtype=dtype, draft=draft, parents=parents, counts=counts, temperature=heat)
         for i, (B, T, V, dtype, draft, parents, counts, heat) in enumerate([
             (1, 1, 1, FP32, None, "tree", None, False), (2, 3, 2, FP32, FP32, "tree", None, False),
             (4, 2, 7, BF16, None, None, None, True), (4, 5, 100, FP32, FP32, None, [5, 0, 1, 9], False),
             (3, 16, 1000, BF16, BF16, "tree", None, True), (3, 16, 1000, FP32, None, "odd", [16, 3, -2], True),
             (2, 33, 4099, FP32, BF16, "tree", None, False), (2, 64, 513, BF16, FP32, "tree", [64, 40], True),
             (6, 64, 50, FP32, None, "tree", None, True), (5, 8, 9001, BF16, FP32, None, None, True),
             (2, 40, 31, FP32, FP32, "odd", None, False), (3, 7, 128256, BF16, FP32, "tree", None, True),
             (2, 5, 128256, FP32, None, None, None, False), (1, 6, 50257, FP32, FP32, None, None, True),
             (9, 12, 2048, BF16, BF16, "tree", None, False), (17, 4, 8192, BF16, None, "tree", None, True),
             (40, 3, 1001, FP32, FP32, None, None, True), (1, 300, 40, FP32, None, None, None, False),
             (1, 9, 70001, BF16, BF16, "tree", None, False), (150, 6, 300, FP32, BF16, "tree", None, True)])]


@pytest.mark.parametrize("kw", CASES, ids=lambda kw: str(kw["seed"]))
def test_inputs_are_clear(kw):
    path, accepted, last, near = expected(make(**kw))
    assert near.min() > CLEAR


def test_inputs_go_all_ways():
    taken = [expected(make(**kw))[1] for kw in CASES]
    assert sum((a == 1).sum() for a in taken) > 50 and sum((a == 2).sum() for a in taken) > 20
    assert sum((a > 4).sum() for a in taken) > 10


@gpu
@pytest.mark.parametrize("kw", CASES, ids=lambda kw: str(kw["seed"]))
def test_verify(kw):
    check(make(**kw))


@gpu
@pytest.mark.parametrize("dtype,draft", [(FP32, BF16), (BF16, FP32), (FP32, FP32), (BF16, BF16)])
@pytest.mark.parametrize("V", [1001, 1003, 1008])
def test_strided_rows(V, dtype, draft):
    """Rows inside wider ones, at odd offsets: alignments of every kind, and neighbours that play no part."""
    a = make(50, 3, 9, V, dtype, draft)
    want = expected(a)
    for shift, wide in ((0, V), (1, V + 7), (3, V + 13), (8, V + 24)):
        d = on_device(a)
        for name in ("logits", "draft", "noise"):
            x = d[name]
            big = torch.full((*x.shape[:-1], wide + shift), float("nan"), dtype=x.dtype, device="cuda")
            if shift == 0 and wide == V:
                continue
            big[..., shift:shift + V] = x
            d[name] = big[..., shift:shift + V]
        for g, w in zip(call(d), want):
            assert np.array_equal(g.cpu().numpy(), w)


def odd_inputs():
    """Values without a meaning of their own, each taken as the header says."""
    inf, nan = float("inf"), float("nan")
    a = make(60, 16, 4, 40, FP32, FP32, None)
    logits, draft = a["logits"], a["draft"]
    logits[0, 0] = -inf                               # no distribution: nothing accepted
    logits[1, 1] = nan                                # nor behind an accepted node
    a["uniform"][1, 1], draft[1, 0, a["tokens"][1, 1]] = 0, 0.0
    logits[2, 0, ::2], logits[2, 0, 1::3] = nan, -inf  # some of both
    logits[3, 0, [7, 9]] = inf                        # shared by the infinite ones
    a["temperature"] = np.ones(16, np.float32)
    a["temperature"][[4, 5, 6, 7]] = 0.0, -1.0, nan, 1e-30
    logits[4, :, 5] = logits[4, :, 30] = 50.0         # the first of the largest
    logits[5, 0, a["tokens"][5, 1]] = 60.0
    a["temperature"][8] = inf                         # all that are not -inf alike
    logits[8, 0, :10] = -inf
    a["uniform"][9, 1], a["uniform"][10, 1], a["uniform"][11, 1] = nan, -3.0, 7.0
    a["noise"][12, :30], a["noise"][13, 3], a["noise"][13, 5] = inf, nan, -1.0
    draft[14, 0, ::2], draft[14, 0, 1::4] = nan, -0.5
    a["tokens"][15, 1] = 40
    a["tokens"][15, 2] = -1
    return a


def test_odd_inputs_are_clear():
    path, accepted, last, near = expected(odd_inputs())
    assert near.min() > CLEAR
    assert last[0] == -1 and accepted[0] == 1 and last[1] == -1 and accepted[1] == 2 and last[4] == 5 and accepted[5] > 1


@gpu
def test_odd_values():
    check(odd_inputs())


def twins():
    """Siblings with the same token, a token that comes again after its rejection, and none left of the residual."""
    a = make(64, 4, 8, 12, FP32, FP32, "tree")
    a["parents"][:] = [-1, 0, 0, 0, 0, 0, 3, 6]
    a["tokens"][:, 2] = a["tokens"][:, 1]
    a["tokens"][:, 3] = a["tokens"][:, 1]
    a["uniform"][:, 1:5] = 0.97
    a["draft"][2] = torch.softmax(a["logits"][2] - 3, -1)  # p = q: always accepted
    return a


def test_twins_are_clear():
    near = expected(twins())[3]
    assert near[[0, 1, 3]].min() > CLEAR


@gpu
@pytest.mark.parametrize("draft", [True, False])
def test_twins(draft):
    a = twins()
    if not draft:
        a["draft"] = None
    want = expected(a)
    got = [x.cpu().numpy() for x in call(on_device(a))]
    for b in range(4):
        if want[3][b] > CLEAR:
            assert all(np.array_equal(g[b], w[b]) for g, w in zip(got, want))


@gpu
def test_nothing_left():
    """p is one token's and the drafts without probabilities have taken it out: next is sampled from p."""
    logits = torch.full((1, 3, 50), -100.0, device="cuda")
    logits[0, :, 7] = 100.0
    t = lambda x, d=torch.int32: torch.tensor([x], dtype=d, device="cuda")
    path, accepted, last = mk.tree_verify(logits, t([0, 7, 9]), t([0.0, 1.0, 1.0], FP32), torch.ones((1, 50), device="cuda"),
                                          t([-1, 0, 0]))
    assert path.tolist() == [[0, -1, -1]] and accepted.tolist() == [1] and last.tolist() == [7]


@gpu
@pytest.mark.parametrize("n,accepted", [(3000, [3000, 1, 2999]), (9000, [9000, 129, 4000])])
def test_long_chains(n, accepted):
    """Chains longer than a tree may be, of sure drafts."""
    V = 5
    rng = np.random.default_rng(n)
    tokens = torch.from_numpy(rng.integers(0, V, (3, n)).astype(np.int32)).cuda()
    logits = torch.zeros((3, n, V), device="cuda")
    logits[:, :-1].scatter_(2, tokens[:, 1:, None].long(), 40.0)
    for b, a in enumerate(accepted):
        if a < n:
            logits[b, a - 1] = 0
            logits[b, a - 1, (int(tokens[b, a]) + 1) % V] = 40.0
    path, acc, last = mk.tree_verify(logits, tokens, torch.rand((3, n), device="cuda"), torch.ones((3, V), device="cuda"))
    assert acc.tolist() == accepted
    at = torch.arange(n, device="cuda")
    assert torch.equal(path, torch.where(at < acc[:, None], at, -1).int())
    for b, a in enumerate(accepted):
        assert int(last[b]) == int(logits[b, a - 1].argmax())


@gpu
@pytest.mark.parametrize("draft", ["sampled", "sure"])
@pytest.mark.parametrize("parents", [[-1, 0, 1], [-1, 0, 0, 0, 1, 1], [-1, 0, 0, 2, 2, 2, 4]])
def test_distribution(parents, draft):
    """What a sequence says first and second is distributed as the target has it: 40960 samples of each, counts within
    6 standard deviations of the expected ones (a chance of 2e-9 each, from a fixed seed)."""
    V, B, T, rounds = 6, 1024, len(parents), 40
    g = torch.Generator(device="cuda").manual_seed(9)
    # the target's and the drafter's distribution depend on the last token alone
    target, drafter = (torch.softmax(1.5 * torch.randn((V, V), generator=g, device="cuda"), -1) for _ in range(2))
    par = torch.tensor(parents, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    first, second = torch.zeros(V, device="cuda"), torch.zeros(V, V, device="cuda")
    for _ in range(rounds):
        tokens = torch.zeros((B, T), dtype=torch.long, device="cuda")
        for t in range(1, T):
            p = drafter[tokens[:, parents[t]]]
            if draft == "sure":  # any rule that does not look at the random numbers: the likeliest ones in turn
                order = p.argsort(-1, descending=True)
                tokens[:, t] = order[:, sum(x == parents[t] for x in parents[:t])]
            else:
                tokens[:, t] = (p / torch.empty_like(p).exponential_(generator=g)).argmax(-1)
        path, accepted, last = mk.tree_verify(
            target[tokens].log(), tokens.int(), torch.rand((B, T), generator=g, device="cuda"),
            torch.empty((B, V), device="cuda").exponential_(generator=g), par,
            draft=drafter[tokens].contiguous() if draft == "sampled" else None)
        said = torch.cat([tokens.gather(1, path.clamp_min(0).long()), last[:, None].long()], 1)
        said.scatter_(1, accepted[:, None].long(), last[:, None].long())  # the accepted tokens, then the new one
        first += torch.bincount(said[:, 1], minlength=V)
        both = accepted > 1
        second.view(-1).add_(torch.bincount(said[both, 1] * V + said[both, 2], minlength=V * V))

    def near(seen, p):
        n = seen.sum(-1, keepdim=True)
        assert ((seen - n * p).abs() <= 6 * (n * p * (1 - p)).sqrt() + 1).all()
    near(first, target[0])
    near(second, target)
    # (a sure draft of one child is accepted as often as the target says its token: 0.089 x 40960 here)
    assert second.sum() > 3000


@gpu
def test_greedy_is_tree_accept():
    """At temperature 0, without draft probabilities, it is the greedy acceptance."""
    a = make(70, 8, 30, 999, FP32, None, "tree", luck=1.0)
    a["temperature"] = np.zeros(8, np.float32)
    d = on_device(a)
    path, accepted, last = call(d)
    _, want_path, want_accepted, want_last = mk.tree_accept(d["logits"], d["tokens"], d["parents"])
    assert torch.equal(path, want_path) and torch.equal(accepted, want_accepted) and torch.equal(last, want_last)
    assert accepted.max() > 2


@gpu
@pytest.mark.parametrize("kw", [dict(seed=80, B=3, T=12, V=30000, draft=FP32), dict(seed=81, B=40, T=6, V=5000, dtype=BF16)])
def test_streams_graphs_and_repeats(kw):
    d, first = check(make(**kw))
    same = lambda x: all(torch.equal(a, b) for a, b in zip(x, first))
    for _ in range(20):
        assert same(call(d))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = call(d, stream=side)
    side.synchronize()
    assert same(x)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(d))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for o in outs:
            for t in o:
                t.fill_(99)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(o) for o in outs)


@gpu
def test_as_many_sequences_as_there_may_be():
    a = make(90, 1024, 3, 33, FP32, FP32, "tree", counts=list(np.arange(1024) % 5 - 1))
    want = expected(a)
    got = [x.cpu().numpy() for x in call(on_device(a))]
    sure = want[3] > CLEAR
    assert sure.mean() > 0.99
    for g, w in zip(got, want):
        assert np.array_equal(g[sure], w[sure])


@gpu
def test_binding_refusals():
    z = lambda *s, d=FP32: torch.zeros(s, device="cuda", dtype=d)
    logits, tokens, uniform, noise = z(2, 3, 9), z(2, 3, d=torch.int32), z(2, 3), z(2, 9)
    call = mk.tree_verify
    bad = [lambda: call(logits.half(), tokens, uniform, noise), lambda: call(logits.cpu(), tokens, uniform, noise),
           lambda: call(logits[0], tokens, uniform, noise), lambda: call(logits, tokens.long(), uniform, noise),
           lambda: call(logits, tokens, uniform.double(), noise), lambda: call(logits, tokens, uniform[:1], noise),
           lambda: call(logits, tokens, uniform, noise[:, :8]), lambda: call(logits, tokens, uniform, noise.cpu()),
           lambda: call(logits, tokens, uniform, noise.bfloat16()), lambda: call(logits, tokens, uniform, z(2, 18)[:, ::2]),
           lambda: call(z(2, 3, 18)[..., ::2], tokens, uniform, noise),
           lambda: call(logits, tokens, uniform, noise, draft=z(2, 3, 8)), lambda: call(logits, tokens, uniform, noise, draft=logits.cpu()),
           lambda: call(logits, tokens, uniform, noise, draft=logits.half()),
           lambda: call(logits, tokens, uniform, noise, parents=tokens[:1]), lambda: call(logits, tokens, uniform, noise, counts=tokens[0]),
           lambda: call(logits, tokens, uniform, noise, temperature=z(3)), lambda: call(logits, tokens, uniform, noise, temperature=1.0)]
    for i, f in enumerate(bad):
        with pytest.raises(mk.MkError) as e:
            f()
        assert e.value.code == mk.MK_ERR_INVALID, i
    torch.cuda.synchronize()


@gpu
def test_long_sums_of_a_residual():
    """A block that has a whole row to itself (153 sequences) adds up 2048 equal values a thread, each of which serial
    sums in fp32 would round the same way (2^-15 of the sum in all). Thresholds 2^-16 on either side of the exact one
    fall on theirs: a sum loses 2^-18.5 here (adds of a tree of 32 or 8, of a warp, of its parts, each compensated or 2^-24)."""
    B, V = 153, 2**19
    logits = torch.zeros((B, 3, V), dtype=BF16, device="cuda")  # p = 2^-19, exactly
    draft = torch.full((B, 3, V), 2.0**-19 * (0.5 - 2.0**-15), device="cuda")  # r = 2^-20 (1 + 2^-14) of each
    tokens = torch.tensor([0, 5, 9], dtype=torch.int32, device="cuda").expand(B, 3).contiguous()
    draft[:, 0, 5], draft[:, 0, 9] = 0.5, 0.8 * 2.0**-19
    q, p = float(draft[0, 0, 9]), 2.0**-19
    left = (V - 2) * 2.0**-20 * (1 + 2.0**-14) + (p - q)
    limit = (p - q) / (q * left)  # child 9 is accepted below it
    uniform = torch.full((B, 3), 0.9, device="cuda")
    uniform[0::2, 2], uniform[1::2, 2] = limit * (1 - 2.0**-16), limit * (1 + 2.0**-16)
    path, accepted, last = mk.tree_verify(logits, tokens, uniform, torch.ones((B, V), device="cuda"),
                                          torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda").expand(B, 3).contiguous(), draft=draft)
    assert (accepted[0::2] == 2).all() and (path[0::2, 1] == 2).all() and (accepted[1::2] == 1).all()


@gpu
@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_long_sums_of_ascending_logits(dtype):
    """Each value of a thread is its largest so far: its sum is not taken to a new reference, rounded, each time."""
    B, V = 153, 2**22
    row = torch.arange(V, device="cuda") * 2.0**-37 if dtype == FP32 else torch.arange(V, device="cuda") // 16384 * 2.0**-15
    row = row.to(dtype)
    logits = row.expand(B, 2, V).contiguous()
    tokens = torch.tensor([0, V // 2], dtype=torch.int32, device="cuda").expand(B, 2).contiguous()
    limit = torch.softmax(row.double(), -1)[V // 2].item()
    uniform = torch.zeros((B, 2), device="cuda")
    uniform[0::2, 1], uniform[1::2, 1] = limit * (1 - 2.0**-16), limit * (1 + 2.0**-16)
    path, accepted, last = mk.tree_verify(logits, tokens, uniform, torch.ones((B, V), device="cuda"))
    assert (accepted[0::2] == 2).all() and (accepted[1::2] == 1).all()


@gpu
@pytest.mark.parametrize("V", [33000, 9000])
def test_any_number_of_sequences(V):
    """A sequence's outcome does not depend on how many there are, and with them on the blocks that each has."""
    a = make(100, 3, 6, V, BF16, FP32, "tree")
    want = expected(a)
    assert want[3].min() > CLEAR
    d = on_device(a)
    for B in (1, 2, 13, 14, 15, 16, 19, 20, 36, 37, 38, 39, 73, 74, 75, 76, 77, 152, 153, 305):
        at = torch.arange(B, device="cuda") % 3
        got = call({n: None if x is None else x[at].contiguous() for n, x in d.items()})
        for g, w in zip(got, want):
            assert np.array_equal(g.cpu().numpy(), w[at.cpu().numpy()]), B
