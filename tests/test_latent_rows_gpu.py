"""Attention over the FP8 and bf16 caches: what the bytes of a row, and values that are not finite,
do to the tokens that see it.  Bounds as in test_latent_gpu.
"""
import numpy as np
import pytest

from tests.test_latent_gpu import BAD, STORES, Batch, bf16, bf16_bytes, dev, random_tree, spoil, torch

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


WHOLE = [("fp8", kind) for kind in BAD["fp8"]] + [("bf16", kind) for kind in BAD["bf16"]]


@pytest.mark.parametrize("store,kind", WHOLE)
@pytest.mark.parametrize("n,Q,H,window", [(300, 1, 4, 0), (300, 3, 40, 0), (3000, 2, 24, 0), (500, 3, 64, 400)])
def test_rows_not_finite_that_every_token_sees(store, kind, n, Q, H, window):
    """A row that is not finite in a tile that all tokens see whole: NaN for all of them (all dims and
    lse), whatever its scores' signs, and nothing for the other requests."""
    s = Batch(store, [n, 77, n], Q, H, 16, seed=42)
    spoil(s, 0, n - 200 if window else 10, kind)
    s.cache = dev(s.cache_np)
    for sinks in (None, torch.linspace(-3, 3, H, device=s.q.device)):
        out, lse = s.attention(window=window, sinks=sinks)
        assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
        s.check(out, lse, window, sinks, skip={(0, j) for j in range(Q)})


@pytest.mark.parametrize("store,kind", WHOLE)
@pytest.mark.parametrize("n", [200, 4000])
def test_padding_beside_context_rows_not_finite(store, kind, n):
    """In a tree, tokens that are padding give zeros although their row tile holds products of 0 and
    rows that are not finite; the others give NaN."""
    Q, H = 8, 9
    tree = [1, 0b11, 0, 0b1011, 0, 0, 0, 0]
    s = Batch(store, [n, n], Q, H, 16, seed=43, trees=[tree, [0] * Q])
    for b in (0, 1):
        spoil(s, b, 70, kind)
    s.cache = dev(s.cache_np)
    seeing, padding = [0, 1, 3], [2, 4, 5, 6, 7]
    for sinks in (None, torch.linspace(-3, 3, H, device=s.q.device)):
        out, lse = s.attention(sinks=sinks)
        assert torch.isnan(out[0, seeing]).all() and torch.isnan(lse[0, seeing]).all()
        assert bool((out[0, padding] == 0).all()) and bool((out[1] == 0).all())
        s.check(out, lse, 0, sinks, skip={(0, j) for j in seeing})
