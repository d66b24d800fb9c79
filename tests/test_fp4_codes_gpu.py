"""The 4-bit insert's bytes, code for code, signs of zeros among them."""
import numpy as np
import pytest

from oracle import fp4
from tests.test_fp4_gpu import EPS, bf16, cos_sin_table, dev, k, torch

pytestmark = pytest.mark.gpu


def _rows(kind, T, rng):
    zeros = np.where(rng.random((T, 512)) < 0.5, -0.0, 0.0)
    if kind == "gaussian":
        return np.where(rng.random((T, 512)) < 0.2, zeros, rng.standard_normal((T, 512)))
    # a quarter of +-2 and the rest zeros: the mean square is 1, so the weights alone
    # say what is stored, and a weight of 1.25 puts values onto a border between two codes
    signs = np.where(rng.random((T, 512)) < 0.5, -2.0, 2.0)
    return np.where(np.arange(512) % 4 == 0, signs, zeros)


@pytest.mark.parametrize("kind,eps", [("gaussian", EPS), ("borders", 0.0)])
@pytest.mark.parametrize("T,H", [(33, 0), (21, 2)])
def test_insert_code_bytes(kind, eps, T, H):
    """A code's sign is the value's, a zero's included, whichever arithmetic decided the row."""
    rng = np.random.default_rng(41)
    kv, kv64 = bf16(_rows(kind, T, rng))
    weight = np.where(rng.random(512) < 0.5, 1.25, 0.75)
    weight[rng.random(512) < 0.1] = 0.0
    weight[rng.random(512) < 0.1] = -0.0
    weight[0] = 1.25
    w, w64 = bf16(weight)
    q = bf16(rng.standard_normal((T, H, 512)))[0] if H else None
    block, nb = 16, -(-T // 16)
    cache = torch.zeros(k.fp4_cache_bytes(nb, block), dtype=torch.uint8, device="cuda")
    positions = np.arange(T)
    k.qnorm_rope_kv_fp4_insert(q, kv, w, dev(positions, np.int64), dev(cos_sin_table(T)),
                               dev(np.arange(T), np.int64), cache, nb, block, eps)
    got = cache.cpu().numpy()
    for t in range(T):
        _, exps, codes = fp4.quantise(fp4.norm_rope(kv64[t], w64, cos_sin_table(T)[t], eps))
        data, scale = fp4.row_bytes(got, block, t)
        assert np.array_equal(scale[:14], (exps + 127).astype(np.uint8))
        assert np.array_equal(data[:224], fp4.pack(codes)), t
