"""An operator's first call of a process may be one that is captured: what it asks the device and keeps
(shared memory allowed, clusters resident) is not work on the stream."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = """
import torch
from decode_megakernel_03_gb300 import mk
dev = "cuda"
new = lambda *s, d=torch.float32: torch.ones(s, dtype=d, device=dev)
ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
logits, tokens = torch.zeros((2, 2, 40000), device=dev), ints([0, 7], [0, 9])
logits[0, 0, 7], logits[:, 1, 5], logits[1, 0, 3] = 60.0, 60.0, 60.0
k = [new(2, 2, 20000, 128, d=torch.bfloat16)]
cache, rope = mk.Cache(k, [k[0].clone()]), mk.Rope(128)
q, kn = new(2, 1, 16, 128, d=torch.bfloat16), new(2, 1, 2, 128, d=torch.bfloat16)
starts, first, prefix = ints(19000, 18000), ints(0), ints(17000)
uniform, noise = new(2, 2) / 2, new(2, 40000)
def calls():
    a = mk.norm_rope_append(rope, cache, 0, q, kn, kn, None, None, starts)
    return (*mk.tree_verify(logits, tokens, uniform, noise), mk.rope_append(rope, cache, 0, a, kn, kn, starts),
            mk.tree_attention(cache, 0, a, starts), mk.prefix_attention(cache, 0, a, first, prefix, starts),
            *mk.tree_accept(logits, tokens))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = calls()
graph.replay()
torch.cuda.synchronize()
assert outs[1].tolist() == [2, 1] and outs[2].tolist() == [5, 3]
assert all(torch.equal(a, b) for a, b in zip(outs, calls()))
torch.cuda.synchronize()
print("done")
"""


def test_first_call_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr
