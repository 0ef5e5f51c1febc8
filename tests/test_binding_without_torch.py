"""The host-only half of the binding (schedules, page tables, rotary plans) needs no
torch: importing the module does not import it."""
import os
import subprocess
import sys

from decode_megakernel_03_gb300 import build as mkbuild

SCRIPT = """
import sys, types
sys.modules["torch"] = None  # an import of it raises
from decode_megakernel_03_gb300 import mk
shape = types.SimpleNamespace(n_layers=2, hidden=256, n_heads=4, n_kv_heads=2, head_dim=64, ffn=1024, vocab=4096,
                              tied=True, rms_eps=1e-5, rope_theta=10000.0)
instrs, offsets, targets = mk.schedule(shape, 1, 128, 152, [5])
assert len(instrs) and len(offsets) == 153
pages = mk.Pages(8, 4, 3, 16)
pages.resize([0], [6])
pages.fork([0], [1])
assert pages.resize([1], [7]).tolist() == [[1, 2, 2]] and pages.n_free() == 5
assert mk.Rope(64).struct.rotary_dim == 64
try:
    pages.resize([9], [1])
except mk.MkError as e:
    assert e.code == mk.MK_ERR_INVALID
else:
    raise AssertionError
print("done")
"""


def test_host_calls_without_torch():
    mkbuild.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr
