"""The operators for drafted trees and rotary positions whose first call of a process is captured
into a graph."""
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
nb, bs = 12, 16
gen = torch.Generator(device="cuda").manual_seed(1)
randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
q = randn(2, 3, 5, 512).bfloat16()
table = torch.tensor([[0, 1, 2], [3, 4, 0]], dtype=torch.int32, device="cuda")
lens = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
tree = torch.tensor([[1, 3, 5], [1, 3, 7]], device="cuda")
store = k.STORE_BF16 if name.endswith("bf16") else k.STORE_FP8
if store == k.STORE_FP8:  # codes and exponents of moderate values
    cache = torch.randint(0, 64, (k.fp8_cache_bytes(nb, bs),), generator=gen, device="cuda", dtype=torch.uint8)
else:
    cache = randn(nb * bs * 512).bfloat16().view(torch.uint8)
path = torch.tensor([[0, 2, -1], [1, -1, -1]], dtype=torch.int32, device="cuda")
path_lens = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
positions = torch.arange(50, device="cuda")
frequencies = k.rope_frequencies(64)
angles = randn(50, 32)
cos_sin = torch.cat([angles.cos(), angles.sin()], 1).contiguous()
x = randn(50, 3, 96)
workspace = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()


def call():
    if name.startswith("attention"):
        out = torch.zeros_like(q)
        k.latent_attention(store, q, cache, nb, bs, table, lens, 0.05, out, tree=tree, workspace=workspace)
        return out
    if name == "keep":
        c, new = cache.clone(), torch.empty_like(lens)
        k.tree_keep(store, c, nb, bs, table, lens, path, path_lens, new)
        return c
    if name == "table":
        out = torch.zeros(50, 64, device="cuda")
        k.rope_table(frequencies, out, positions=positions)
        return out
    out = torch.zeros_like(x)
    k.rope_rows(x, positions, cos_sin, out=out, layout=k.ROPE_HALF)
    return out


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


@pytest.mark.parametrize("name", ["attention_fp8", "attention_bf16", "keep", "table", "rows"])
def test_first_call_inside_a_capture(name):
    done = subprocess.run([sys.executable, "-c", SCRIPT, name], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "same" in done.stdout, done.stderr[-2000:]
