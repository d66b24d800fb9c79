"""The 4-bit cache's attention and attention weights at the ends of the number range: scores past
fp32's range, values near nothing, and rows that are not finite.  Bounds as in test_fp4_gpu.py;
besides, a value below 2^-46 may be taken as any other that small (dsv4kv.h)."""
import numpy as np
import pytest

from oracle import fp4
from tests.test_fp4_gpu import DEV, Batch, bf16, dev, k, torch

pytestmark = pytest.mark.gpu


def _set_rope(s, b, i, dim, value):
    data, _ = fp4.row_bytes(s.cache_np, s.block, s.table_np[b, i // s.block] * s.block + i % s.block)
    at = 224 + 2 * (dim - 448)
    data[at:at + 2] = torch.tensor([value]).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint8)


def _reread(s):
    s.cache = dev(s.cache_np)
    for b, n in enumerate(s.lens):
        s.rows[b], s.ok[b] = fp4.rows_of(s.cache_np, s.block, s.table_np[b], n)


def _add_weights(s, lse, window=0):
    w = torch.full((len(s.lens), max(s.lens)), 0.25, device=DEV)
    k.fp4_attention_weights(s.q, s.cache, s.nb, s.block, s.table, s.lens_t, s.scale, lse, w, window=window)
    return w.double().cpu().numpy()


def _close(got, want, size, ds):
    tol = np.abs(want) * 2.0 ** -8 + size * (2.0 ** -8 + 2 * ds[..., None])
    assert np.all(np.abs(got - want) <= tol + 1e-30)


@pytest.mark.parametrize("with_sinks", [False, True])
@pytest.mark.parametrize("n", [300, 6000])
def test_scores_that_overflow_to_minus_infinity(n, with_sinks):
    """Head 0 has such scores for the first third of the keys, which take no part; head 1 for all of
    them, and so has no value; head 2 for none.  (6000 keys lie in many runs, some without a sum.)"""
    s = Batch([n, 40], 1, 3, 16, seed=51)
    third = n // 3
    for i in range(n):
        _set_rope(s, 0, i, 448, 100.0 if i < third else 0.0)
        _set_rope(s, 0, i, 449, 100.0)
    _reread(s)
    q = s.q64.copy()
    q[0, 0, :2] = 0.0
    q[0, 0, 0, 448] = q[0, 0, 1, 449] = -3e38
    s.q, s.q64 = bf16(q)
    sinks = dev([0.5, -1.5, 2.0], np.float32) if with_sinks else None
    out, lse = s.attention(sinks=sinks)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    calm = s.q64[0].copy()
    calm[0, :2] = 0.0
    part = s.ok[0] & (np.arange(n) >= third)
    sinks64 = None if sinks is None else sinks.double().cpu().numpy()
    for h, ok in ((0, part), (2, s.ok[0])):
        want, wlse, size, reach = fp4.attention(calm[:, h:h + 1], s.rows[0], ok, n, s.scale, 0,
                                                None if sinks64 is None else sinks64[h:h + 1])
        ds = s.scale * reach * 2.0 ** -15 + 2.0 ** -18
        _close(got[0, :, h:h + 1], want, size, ds)
        assert np.all(np.abs(glse[0, :, h] - wlse[:, 0]) <= ds[:, 0] + np.abs(wlse[:, 0]) * 2.0 ** -22)
    assert np.all(got[0, 0, 1] == 0)
    if with_sinks:
        assert abs(glse[0, 0, 1] + 1.5) <= 2.0 ** -20
    else:
        assert np.isneginf(glse[0, 0, 1])
    if not with_sinks:
        w = _add_weights(s, lse)[0, :n]
        want = 0.25 + fp4.weights(calm[:, :1], s.rows[0], part, n, s.scale, glse[0, :, :1])
        want += fp4.weights(calm[:, 2:], s.rows[0], s.ok[0], n, s.scale, glse[0, :, 2:])
        reach = (np.abs(calm[0]) @ np.abs(s.rows[0]).T).max() * s.scale
        assert np.all(np.abs(w - want) <= want * (reach * 2.0 ** -15 + 2.0 ** -18))


@pytest.mark.parametrize("Q,H", [(1, 3), (2, 40)])
def test_values_near_nothing(Q, H):
    """Groups and rope dims from 2^-70 to 2^-40 beside ordinary ones, and a request of nothing else."""
    s = Batch([200, 90], Q, H, 16, seed=52)
    rng = np.random.default_rng(53)
    for b, n in enumerate(s.lens):
        for i in range(n):
            _, scale = fp4.row_bytes(s.cache_np, 16, s.table_np[b, i // 16] * 16 + i % 16)
            groups = slice(0, 5) if b == 0 else slice(0, 14)
            scale[groups] = rng.integers(57, 88, scale[groups].size)
            for dim in range(448, 460 if b == 0 else 512):
                _set_rope(s, b, i, dim, float(rng.standard_normal() * 2.0 ** rng.integers(-70, -40)))
    _reread(s)
    out, lse = s.attention()
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(s.lens):
        want, wlse, size, reach = fp4.attention(s.q64[b], s.rows[b], s.ok[b], n, s.scale)
        ds = s.scale * reach * 2.0 ** -15 + 2.0 ** -18
        tol = np.abs(want) * 2.0 ** -8 + size * (2.0 ** -8 + 2 * ds[..., None]) + 2.0 ** -46
        assert np.all(np.abs(got[b] - want) <= tol)
        assert np.all(np.abs(glse[b] - wlse) <= ds + np.abs(wlse) * 2.0 ** -22)
    w = _add_weights(s, lse)
    for b, n in enumerate(s.lens):
        add = fp4.weights(s.q64[b], s.rows[b], s.ok[b], n, s.scale, glse[b])
        reach = (np.abs(s.q64[b]).reshape(-1, 512) @ np.abs(s.rows[b]).T).max() * s.scale
        bound = reach * 2.0 ** -15 + 2.0 ** -18 + np.abs(glse[b]).max() * 2.0 ** -22 + Q * H * 2.0 ** -24
        assert np.all(np.abs(w[b, :n] - 0.25 - add) <= add * bound + (0.25 + add) * 2.0 ** -23)


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
