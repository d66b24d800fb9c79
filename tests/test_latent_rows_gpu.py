"""Attention over the FP8 and bf16 caches: what the bytes of a row, and values that are not finite,
do to the tokens that see it.  Bounds as in test_latent_gpu.
"""
import numpy as np
import pytest

from tests.test_latent_gpu import STORES, Batch, bf16, bf16_bytes, random_tree, torch

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


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("order", ["low first", "high first", "mixed"])
@pytest.mark.parametrize("n", [50, 300, 5000])
@pytest.mark.parametrize("score", [2.0 ** 127, 2e38, 3e30, 1.7e12, 1.1e9, 5e8, 3e7, 7e6])
def test_large_scores_of_either_sign(store, order, n, score):
    """Finite scores, the largest further apart than fp32 reaches: the low ones have a probability of 0."""
    s = Batch(store, [n], 2, 5, 16, seed=41)
    high = {"low first": np.arange(n) >= n // 2, "high first": np.arange(n) < n // 2,
            "mixed": np.arange(n) % 3 == 0}[order]
    high[-1] = False  # (the token before the last sees as many)
    for i in range(n):
        s.row(0, i)[0][-128:-126] = bf16_bytes([1.0 if high[i] else -1.0])
    s.refresh()
    q = np.zeros_like(s.q64)
    q[..., 448] = score
    s.q, s.q64 = bf16(q)
    s.scale = 1.0
    out, lse = s.attention()
    rows = s.rows[0][high]
    want, size = rows.mean(0), np.abs(rows).mean(0)
    # every p that is not 0 is 1: half a step of the output, and the roundings of fp32 sums
    assert np.all(np.abs(out[0].double().cpu().numpy() - want) <= np.abs(want) * 2.0 ** -8 + size * 2.0 ** -8)
    assert np.allclose(lse[0].double().cpu().numpy(), s.q64[0, 0, 0, 448] + np.log(high.sum()), rtol=2.0 ** -20, atol=0)
