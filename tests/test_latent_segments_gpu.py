"""Attention over the FP8 and bf16 caches where a CTA's run is made of segments of one tile: a
row's reference and its sum both come out of that tile, over two halves of the keys.

The scores all lie far below zero, so a half that took anything but the row's maximum (a sum is
1 or more) as its reference would have probabilities of 0.  Bounds as in test_latent_gpu.
"""
import numpy as np
import pytest

from tests.test_latent_gpu import STORES, Batch, bf16, bf16_bytes, random_tree, torch

pytestmark = pytest.mark.gpu


def _shifted(s, level):
    """Every score of the batch moved by -level: a dim that is 1 in all rows, and that q has alike."""
    at = 448 if s.store == "fp8" else 896  # byte of dim 448
    for b, n in enumerate(s.lens):
        for i in range(n):
            s.row(b, i)[0][at:at + 2] = bf16_bytes([1.0])
    s.refresh()
    q = s.q64.copy()
    q[..., 448] = -level / s.scale
    s.q, s.q64 = bf16(q)
    return s


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("lens,Q,H,trees", [
    ([33 + i % 32 for i in range(320)], 1, 64, False),  # one row tile a request, a tile each
    ([1 + i % 64 for i in range(200)], 3, 40, False),   # two row tiles, the second not full
    ([20 + i % 45 for i in range(150)], 9, 16, True),
    ([64], 1, 8, False),
])
def test_segments_of_one_tile(store, lens, Q, H, trees):
    rng = np.random.default_rng(len(lens))
    words = [random_tree(rng, Q) for _ in lens] if trees else None
    s = _shifted(Batch(store, lens, Q, H, 16, seed=len(lens) + Q, trees=words), 260.0)
    out, lse = s.attention()
    s.check(out, lse)
    out2, lse2 = torch.empty_like(out), None
    for _ in range(100):
        _, lse2 = s.attention(out=out2)
        assert torch.equal(out2, out) and torch.equal(lse2, lse)
