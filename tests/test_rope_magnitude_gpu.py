"""Rows turned by a table of a magnitude other than 1, and back.

Bounds: table entries are within 2^-23 of m (half a step, and what test_rope_gpu allows beside it); fp32
rows take two roundings of 2^-24 each way, of |a cos| + |b sin| <= 2 m max|x|.  There and back that
is below 16 * 2^-23 times max|x| times the magnitudes' product; bf16 adds half a step (2^-8) each way.
"""
import numpy as np
import pytest

from oracle import latent
from tests.test_latent_gpu import DEV, Batch, bf16, dev, k, torch

pytestmark = pytest.mark.gpu


def tables(magnitudes, positions=50, dim=32):
    out = []
    for m in magnitudes:
        t = torch.empty(positions, dim, device=DEV)
        k.rope_table(k.rope_frequencies(dim, 1000.0), t, magnitude=m)
        out.append(t)
    return out


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("m", [1.0, 1.05, 0.7, -3.0, 0.1 * np.log(40.0) + 1])
@pytest.mark.parametrize("dtype,step", [(torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)])
def test_there_and_back(half, m, dtype, step):
    layout = k.ROPE_HALF if half else k.ROPE_PAIRS
    there, back = tables([m, 1 / m])
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(37, 6, 48, generator=gen, device=DEV).to(dtype)
    at = torch.randint(0, 50, (37,), generator=gen, device=DEV)
    turned, again = torch.empty_like(x), torch.empty_like(x)
    k.rope_rows(x, at, there, out=turned, layout=layout)
    k.rope_rows(turned, at, back, out=again, layout=layout, inverse=True)
    most = float(x.abs().max())
    tol = 2 * most * (8 * 2.0 ** -23 + 2 * step)
    assert float((again.double() - x.double()).abs().max()) <= tol
    # by its own table it is the transpose: m^2 times as large
    k.rope_rows(turned, at, there, out=again, layout=layout, inverse=True)
    part = slice(16, 48)
    assert float((again[..., part].double() - m * m * x[..., part].double()).abs().max()) <= m * m * tol
    assert torch.equal(again[..., :16], x[..., :16])


def test_attention_output_turned_back():
    """Rows turned by a table of magnitude m: the output's trailing dims, turned back by 1 / m at the token's
    position, are the sums of the rows as they were, turned by the distance."""
    m, n, H = 1.25, 90, 6
    rng = np.random.default_rng(5)
    there, back = tables([m, 1 / m], positions=n, dim=64)
    s = Batch("bf16", [n], 1, H, 16, seed=6)
    plain = rng.standard_normal((n, 512))
    turned, values = bf16(plain)
    k.rope_rows(turned, torch.arange(n, device=DEV), there)
    for i, row in enumerate(turned.view(torch.int16).cpu().numpy().view(np.uint8)):
        s.row(0, i)[0][:] = row
    s.refresh()
    out, lse = s.attention()
    s.check(out, lse)
    got = out.clone().view(1, H, 512)
    k.rope_rows(got, dev([n - 1], np.int64), back, inverse=True)
    scores = s.scale * s.q64[0, 0] @ s.rows[0].T
    p = np.exp(scores - scores.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    frequencies = k.rope_frequencies(64, 1000.0)
    moved = np.stack([latent.rotate(values[i], latent.table_row(n - 1 - i, frequencies, 1.0), 448, False, True)
                      for i in range(n)])
    want, size = p @ moved, np.abs(p) @ np.abs(moved)
    reach = s.scale * (np.abs(s.q64[0, 0]) @ np.abs(s.rows[0]).T).max() * 2.0 ** -15
    # bf16 roundings of the turned rows, of p, of the output and of the turn back: 2^-8 each, of sums of
    # two terms |a| + |b| in the turned dims
    pairs = size.copy()
    pairs[:, 448:] += size[:, 448:].reshape(H, 32, 2)[..., ::-1].reshape(H, 64)
    wide = p @ np.abs(values)
    wide[:, 448:] += wide[:, 448:].reshape(H, 32, 2)[..., ::-1].reshape(H, 64)
    tol = (4 * 2.0 ** -8 + 2 * reach) * 2 * np.maximum(pairs, wide)
    assert np.all(np.abs(got[0].double().cpu().numpy() - want) <= tol)
