"""Attention over the FP8 and bf16 caches: what the bytes of a row, and values that are not finite,
do to the tokens that see it.  Bounds as in test_latent_gpu.
"""
import numpy as np
import pytest

from tests.test_latent_gpu import Batch, random_tree, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block,narrow", [(16, 0), (16, 1), (7, 0)])
@pytest.mark.parametrize("tree", [False, True])
def test_fp8_padding_byte_means_nothing(block, narrow, tree):
    """Byte 7 of a scale row belongs to no block of 64 codes."""
    rng = np.random.default_rng(block)
    Q, lens = 3, [1 + 2, 64, 200, 131]
    words = [random_tree(rng, Q) for _ in lens] if tree else None
    s = Batch("fp8", lens, Q, 24, block, seed=40, narrow=narrow, trees=words)
    want, wlse = s.attention()
    s.check(want, wlse)
    for b, n in enumerate(lens):
        for i in range(n):
            s.row(b, i)[1][7] = 255 if i % 2 else rng.integers(183, 256)
    s.refresh()
    out, lse = s.attention()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
