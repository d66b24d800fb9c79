"""The 4-bit cache's attention weights at the ends of the number range.  Bounds as in test_fp4_gpu.py."""
import numpy as np
import pytest

from oracle import fp4
from tests.test_fp4_gpu import DEV, Batch, dev, k, torch

pytestmark = pytest.mark.gpu


def _set_rope(s, b, i, dim, value):
    data, _ = fp4.row_bytes(s.cache_np, s.block, s.table_np[b, i // s.block] * s.block + i % s.block)
    at = 224 + 2 * (dim - 448)
    data[at:at + 2] = torch.tensor([value]).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint8)


def _add_weights(s, lse, window=0):
    w = torch.full((len(s.lens), max(s.lens)), 0.25, device=DEV)
    k.fp4_attention_weights(s.q, s.cache, s.nb, s.block, s.table, s.lens_t, s.scale, lse, w, window=window)
    return w.double().cpu().numpy()


@pytest.mark.parametrize("kind", ["group", "large", "rope nan", "rope inf", "rope -inf"])
@pytest.mark.parametrize("n,Q,H,window", [(300, 3, 4, 0), (258, 3, 40, 0), (300, 3, 4, 100), (500, 3, 64, 200)])
def test_weights_of_rows_not_finite(kind, n, Q, H, window):
    """A token that sees such a row has no lse, and makes NaN of the keys that it sees and of no
    others; left out by an lse of -infinity, it adds nothing, not even to that row."""
    hit, bad = (Q - 1, n - 1) if window == 0 else (0, n - Q + 1 - window)
    s = Batch([n, 40], Q, H, 16, seed=54)
    data, scale = fp4.row_bytes(s.cache_np, 16, s.table_np[0, bad // 16] * 16 + bad % 16)
    if kind == "group":
        scale[9], data[9 * 16:10 * 16] = 255, 0
    elif kind == "large":
        scale[13] = 230
    else:
        _set_rope(s, 0, bad, 448 + 45, {"rope nan": np.nan, "rope inf": np.inf, "rope -inf": -np.inf}[kind])
    s.cache = dev(s.cache_np)
    out, lse = s.attention(window=window)
    assert torch.isnan(lse[0, hit]).all()
    w = _add_weights(s, lse, window)
    seen = fp4.visible(n, Q, hit, window, np.arange(n))
    assert np.isnan(w[0, :n][seen]).all()
    left = lse.clone()
    left[0, hit] = -float("inf")
    without = _add_weights(s, left, window)
    left64 = left.double().cpu().numpy()
    for b, m in enumerate(s.lens):
        add = fp4.weights(s.q64[b], s.rows[b], s.ok[b], m, s.scale, left64[b], window)
        reach = (np.abs(s.q64[b]).reshape(-1, 512) @ np.abs(s.rows[b]).T).max() * s.scale
        largest = np.abs(left64[b][np.isfinite(left64[b])]).max()
        bound = reach * 2.0 ** -15 + 2.0 ** -18 + largest * 2.0 ** -22 + Q * H * 2.0 ** -24
        close = np.abs(without[b, :m] - 0.25 - add) <= add * bound + (0.25 + add) * 2.0 ** -23
        assert np.all(close)
        if b == 0:
            assert np.array_equal(w[0, :n][~seen], without[0, :n][~seen])
