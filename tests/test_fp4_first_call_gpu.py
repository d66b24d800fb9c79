"""The 4-bit cache's operators whose first call of a process is captured into a graph."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import sys
import torch
import kv_norm_rope_gb300 as k

name = sys.argv[1]
nb, bs, n = 12, 16, 70
gen = torch.Generator(device="cuda").manual_seed(1)
randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
kv, w, q = randn(n, 512).bfloat16(), (1 + 0.1 * randn(512)).bfloat16(), randn(2, 1, 5, 512).bfloat16()
slots = torch.arange(n, device="cuda")
angles = randn(n, 32)
cos_sin = torch.cat([angles.cos(), angles.sin()], 1).contiguous()
table = torch.tensor([[0, 1, 2], [3, 4, 0]], dtype=torch.int32, device="cuda")
lens = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
new = torch.tensor([[8], [9]], dtype=torch.int32, device="cuda")
lse = randn(2, 1, 5)
cache = torch.randint(0, 4, (k.fp4_cache_bytes(nb, bs),), generator=gen, device="cuda", dtype=torch.uint8)
gain = randn(2, 48).abs()
workspace = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()


def call():
    c, weights = cache.clone(), gain.clone()
    out = torch.zeros_like(q)
    if name == "insert":
        k.qnorm_rope_kv_fp4_insert(None, kv, w, slots, cos_sin, slots, c, nb, bs, 1e-6)
        return c
    if name == "gather":
        rows = torch.zeros_like(kv)
        k.fp4_dequant_gather(c, nb, bs, slots, rows)
        return rows
    if name == "attention":
        k.fp4_attention(q, c, nb, bs, table, lens, 0.05, out, workspace=workspace)
        return out
    if name == "weights":
        k.fp4_attention_weights(q, c, nb, bs, table, lens, 0.05, lse, weights)
        return weights
    kept = torch.zeros(2, 16, dtype=torch.int32, device="cuda")
    k.fp4_evict(c, nb, bs, table, lens, weights, 16, 4, new, kept, torch.empty_like(lens),
                torch.zeros(2, 16, device="cuda"))
    return c


graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = call()
graph.replay()
torch.cuda.synchronize()
eager = call()
torch.cuda.synchronize()
assert torch.equal(captured.view(torch.uint8), eager.view(torch.uint8))
print("same")
"""


@pytest.mark.parametrize("name", ["insert", "gather", "attention", "weights", "evict"])
def test_first_call_inside_a_capture(name):
    done = subprocess.run([sys.executable, "-c", SCRIPT, name], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "same" in done.stdout, done.stderr[-2000:]
