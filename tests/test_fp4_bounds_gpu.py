"""The 4-bit cache's operators on the bounds-checked build: no access leaves its buffer, and the
bytes are the release build's."""
import random

import pytest

from tests.test_bounds_gpu import _release_and_checked
from tests.test_fp4_gpu import DEV, EPS, Batch, cos_sin_table, dev, error_word, k, np, torch

pytestmark = pytest.mark.gpu


def _same(fn):
    released, checked = _release_and_checked(fn)
    for name, value in released.items():
        assert torch.equal(value.view(torch.uint8), checked[name].view(torch.uint8)), name


@pytest.mark.parametrize("T,H,block", [(1, 0, 1), (39, 0, 7), (5000, 0, 64), (33, 3, 16), (700, 40, 27)])
def test_insert_and_reader(T, H, block):
    gen = torch.Generator(device=DEV).manual_seed(T)
    kv = torch.randn(T, 512, generator=gen, device=DEV).bfloat16()
    kv[:: 3, ::4] = 2.0  # some rows that are decided again
    w = torch.ones(512, device=DEV, dtype=torch.bfloat16)
    q0 = torch.randn(T, H, 512, generator=gen, device=DEV).bfloat16() if H else None
    nb = -(-T // block)
    slots = torch.randperm(nb * block, generator=gen, device=DEV)[:T]
    slots[::5] = -1
    slots[3::11] = nb * block
    positions = torch.arange(T, device=DEV) % 50
    positions[4::13] = 50

    def run():
        q = None if q0 is None else q0.clone()
        cache = torch.full((k.fp4_cache_bytes(nb, block),), 3, dtype=torch.uint8, device=DEV)
        rows, err = torch.zeros(T, 512, dtype=torch.bfloat16, device=DEV), error_word()
        k.qnorm_rope_kv_fp4_insert(q, kv, w, positions, dev(cos_sin_table(50)), slots, cache, nb, block, EPS,
                                   device_error=err)
        k.fp4_dequant_gather(cache, nb, block, slots, rows, device_error=err)
        out = dict(cache=cache, rows=rows, err=err)
        return out if q is None else dict(out, q=q)

    _same(run)


@pytest.mark.parametrize("seed", range(14))
def test_attention_weights_and_eviction(seed):
    rng = random.Random(seed)
    Q, H, block = rng.choice([1, 1, 3, 9]), rng.randint(1, 140), rng.choice([1, 5, 16, 64])
    lens = [rng.choice([0, rng.randint(1, 700), rng.randint(1, 40)]) for _ in range(rng.randint(1, 40))]
    if seed == 0:
        lens = [9000]
    window = rng.choice([0, 0, 1, 200])
    s = Batch(lens, Q, H, block, seed=seed, spare=80 * len(lens) // block + len(lens), stride=rng.randint(0, 3))
    B, n = len(lens), max(max(lens), 1)
    if seed % 3 == 1:
        s.lens_t[0] = s.W * block + 9  # a length past the table, and pages outside the cache
        s.table[-1, 0] = s.nb
        s.table[0, -1] = -5
    budget = rng.randint(1, 80)
    used = set(s.table_np[s.table_np >= 0].tolist())
    free = [p for p in range(s.nb) if p not in used]
    W2 = -(-budget // block)
    new = dev(np.array(free[:B * W2]).reshape(B, W2), np.int32)
    sinks = torch.zeros(H, device=DEV) if seed % 2 else None

    def run():
        err, cache = error_word(), s.cache.clone()
        out = torch.zeros(B, Q, H, 512, dtype=torch.bfloat16, device=DEV)
        lse, w = torch.zeros(B, Q, H, device=DEV), torch.ones(B, n, device=DEV)
        workspace = torch.empty(k.fp4_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)
        k.fp4_attention(s.q, cache, s.nb, block, s.table, s.lens_t, s.scale, out, lse=lse, sinks=sinks,
                        window=window, workspace=workspace, device_error=err)
        k.fp4_attention_weights(s.q, cache, s.nb, block, s.table, s.lens_t, s.scale, lse, w, window=window,
                                device_error=err)
        kept = torch.zeros(B, budget, dtype=torch.int32, device=DEV)
        new_lens, new_w = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, budget, device=DEV)
        k.fp4_evict(cache, s.nb, block, s.table, s.lens_t, w, budget, 0, new, kept, new_lens,
                    new_w, device_error=err)
        return dict(out=out, lse=lse, w=w, cache=cache, kept=kept, lens=new_lens, new_w=new_w, err=err)

    _same(run)


def test_requests_by_the_thousand():
    pages = Batch([64], 1, 1, 16, seed=3)
    N, H = 3000, 5
    gen = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randn(N, 1, H, 512, generator=gen, device=DEV).bfloat16()
    table = torch.randint(0, pages.nb, (N, 9), generator=gen, device=DEV, dtype=torch.int32)
    lens = torch.randint(0, 144, (N,), generator=gen, device=DEV, dtype=torch.int32)
    lens[::3] = 0

    def run():
        out, lse = torch.zeros_like(q), torch.zeros(N, 1, H, device=DEV)
        w = torch.zeros(N, 144, device=DEV)
        k.fp4_attention(q, pages.cache, pages.nb, 16, table, lens, 0.04, out, lse=lse)
        k.fp4_attention_weights(q, pages.cache, pages.nb, 16, table, lens, 0.04, lse, w)
        return dict(out=out, lse=lse, w=w)

    _same(run)
