"""Sampled serving with drafts, the operators as a serving loop runs them: two prompts, several answers of each on
forked pages, drafted trees appended with normed heads, attended over the shared prefixes, verified by rejection
sampling, the accepted rows kept."""
import numpy as np
import pytest
import torch

from decode_megakernel_03_gb300 import mk, synth
from tests import cache_ops_ref as ref
from tests import sampling_ref
from tests.test_gpu_cache_ops import BF16, FP32, dev, host, ints, make_parents, norm

pytestmark = pytest.mark.gpu


class Model:
    """The tiny shape with a norm on each head of q and k, in torch; its rotary plan."""

    def __init__(self, seed):
        self.shape = synth.TINY
        self.w = synth.make_weights(self.shape, seed=seed, device=dev())
        g = torch.Generator(device=dev()).manual_seed(seed)
        D = self.shape.head_dim
        self.qn, self.kn = ([(1 + 0.2 * torch.randn(D, generator=g, device=dev())).to(BF16) for _ in range(self.shape.n_layers)]
                            for _ in range(2))
        self.rope = mk.Rope(D, theta=self.shape.rope_theta)

    def layers(self, x, attend):
        s, w = self.shape, self.w
        for l in range(s.n_layers):
            n = norm(x, w["attn_norm"][l].to(x.dtype), s.rms_eps)
            q, k, v = ((n @ w[m][l].to(x.dtype).T).view(*x.shape[:-1], -1, s.head_dim) for m in ("wq", "wk", "wv"))
            x = x + attend(l, q, k, v).reshape(*x.shape[:-1], -1) @ w["wo"][l].to(x.dtype).T
            n = norm(x, w["mlp_norm"][l].to(x.dtype), s.rms_eps)
            up = torch.nn.functional.silu(n @ w["wgate"][l].to(x.dtype).T) * (n @ w["wup"][l].to(x.dtype).T)
            x = x + up @ w["wdown"][l].to(x.dtype).T
        head = w["lm_head"] if w["lm_head"] is not None else w["embed"]
        return norm(x, w["final_norm"].to(x.dtype), s.rms_eps) @ head.to(x.dtype).T

    def serve(self, cache, tokens, starts, parents, first, prefix, counts=None):
        """Logits of every node, over the cache."""
        def attend(l, q, k, v):
            q = mk.norm_rope_append(self.rope, cache, l, q, k, v, self.qn[l], self.kn[l], starts, parents, counts,
                                    eps=self.shape.rms_eps)
            return mk.prefix_attention(cache, l, q, first, prefix, starts, parents, counts)
        return self.layers(self.w["embed"][tokens.long()].float(), attend)

    def whole(self, tokens):
        """Logits behind each token of one sequence, in 64 bits, without a cache."""
        s, n = self.shape, len(tokens)
        f, _ = ref.frequencies(s.head_dim, s.rope_theta)
        angle = torch.arange(n, device=dev(), dtype=torch.float64)[:, None, None] * torch.tensor(f, device=dev(), dtype=torch.float64)
        hidden = torch.ones((n, n), dtype=torch.bool, device=dev()).triu(1)

        def turn(x, w):
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s.rms_eps) * w.double()
            a, b = x.chunk(2, -1)
            return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)

        def attend(l, q, k, v):
            q, k = turn(q, self.qn[l]), turn(k, self.kn[l])
            r = s.n_heads // s.n_kv_heads
            k, v = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1)
            sc = torch.einsum("thd,shd->hts", q, k) / s.head_dim ** 0.5
            return torch.einsum("hts,shd->thd", torch.softmax(sc.masked_fill(hidden, -torch.inf), -1), v)
        return self.layers(self.w["embed"][torch.tensor(tokens, device=dev())].double(), attend)


@pytest.mark.parametrize("sampled", [True, False])
def test_rounds_over_forked_pages(sampled):
    model = Model(4)
    shape, bs, cap, T = model.shape, 16, 128, 9
    V, D = shape.vocab, shape.head_dim
    prompts = [synth.make_tokens(V, n, seed=5 + n).tolist() for n in (37, 20)]
    parent_of = [0, 0, 0, 1, 1]                    # answers 0 to 4 of prompts 0 and 1
    pages = mk.Pages(80, bs, 7, cap)               # sequences 0 to 4: answers, 5 and 6: the prompts
    k, v = ([torch.zeros((80, shape.n_kv_heads, bs, D), dtype=BF16, device=dev()) for _ in range(shape.n_layers)]
            for _ in range(2))

    def near(a, b):
        a, b = host(a), host(b)
        assert np.linalg.norm(a - b) <= 1e-2 * np.linalg.norm(b) and np.abs(a - b).max() <= 5e-2

    def cache_of(rows):
        return mk.Cache(k, v, ints(pages.table()[rows]))

    # the prompts, a chain of 64 nodes at most at a time (these are shorter)
    pages.resize([5, 6], [len(p) for p in prompts])
    said, last = [], []
    for i, p in enumerate(prompts):
        logits = model.serve(cache_of([5 + i]), ints([p]), ints([0]), None, ints([0]), ints([0]))
        near(logits[0, -1], model.whole(p)[-1])
        top = logits[0, -1].argsort(descending=True)
        for j in range(parent_of.count(i)):        # each answer begins with another token
            said.append(list(p))
            last.append(int(top[j]))
    pages.fork([5 + i for i in parent_of], range(5))
    pages.resize([5, 6], [0, 0])
    first, prefix = ints([0, 3]), ints([len(p) for p in prompts])
    rng = np.random.default_rng(1)
    g = torch.Generator(device=dev()).manual_seed(2)
    counts = [T, T, 4, T, 1]
    lengths = []
    for _ in range(4):
        starts = [len(s) for s in said]
        mk.cache_copy_blocks(mk.Cache(k, v), pages.resize(range(5), [n + T for n in starts]))
        cache = cache_of(range(5))
        parents = make_parents(rng, 5, T)
        tokens = np.zeros((5, T), np.int64)
        tokens[:, 0] = last
        # the drafter: the model itself, its logits with noise, and tokens drawn from that
        draft = torch.zeros((5, T, V), device=dev())
        for b in range(5):
            for t in range(T):
                if t > 0:
                    p = draft[b, parents[b, t]]
                    tokens[b, t] = int((p / torch.empty_like(p).exponential_(generator=g)).argmax())
                line = said[b] + [int(tokens[b, n]) for n in ref.family(parents, b, t)[::-1]]
                z = 2 * model.whole(line)[-1].float()
                draft[b, t] = torch.softmax(z + 0.3 * torch.randn(V, generator=g, device=dev()), -1)
        logits = model.serve(cache, ints(tokens), ints(starts), ints(parents), first, prefix, ints(counts))
        for b, t in ((0, 0), (0, T - 1), (1, 4), (2, 3), (3, T - 1), (4, 0)):
            line = said[b] + [int(tokens[b, n]) for n in ref.family(parents, b, t)[::-1]]
            near(logits[b, t], model.whole(line)[-1])
        uniform = torch.rand((5, T), generator=g, device=dev())
        noise = torch.empty((5, V), device=dev()).exponential_(generator=g)
        heat = torch.full((5,), 0.5, device=dev())
        path, accepted, nxt = mk.tree_verify(logits, ints(tokens), uniform, noise, ints(parents), ints(counts),
                                             draft if sampled else None, heat)
        want = sampling_ref.verify(host(logits), tokens, host(uniform), host(noise), parents, counts,
                                   host(draft) if sampled else None, host(heat))
        for b in range(5):
            if want[3][b] > 2.0**-15:
                assert path[b].tolist() == want[0][b].tolist() and int(accepted[b]) == want[1][b] and int(nxt[b]) == want[2][b]
        mk.cache_compact(cache, ints(starts), path, accepted)
        for b, a in enumerate(accepted.tolist()):
            said[b] += [int(tokens[b, n]) for n in path[b, :a].tolist()]
            last[b] = int(nxt[b])
            lengths.append(a)
        pages.resize(range(5), [len(s) for s in said])
    if sampled:  # (a sure drafter of random tokens is seldom right)
        assert max(lengths) > 2 and sum(lengths) > 30
    # what the cache holds now is what the answers say: one more token of each, from scratch
    starts = [len(s) for s in said]
    mk.cache_copy_blocks(mk.Cache(k, v), pages.resize(range(5), [n + 1 for n in starts]))
    logits = model.serve(cache_of(range(5)), ints([[t] for t in last]), ints(starts), None, first, prefix)
    for b in range(5):
        near(logits[b, 0], model.whole(said[b] + [last[b]])[-1])
