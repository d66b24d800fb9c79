"""Attention over the FP8 and bf16 caches, the kept path and the rotary positions on the
bounds-checked build: no access leaves its buffer, and the bytes are the release build's."""
import numpy as np
import pytest

from tests.test_bounds_gpu import _release_and_checked
from tests.test_latent_gpu import DEV, STORES, Batch, dev, error_word, k, random_tree, torch

pytestmark = pytest.mark.gpu


def _same(fn):
    released, checked = _release_and_checked(fn)
    for name, value in released.items():
        assert torch.equal(value.view(torch.uint8), checked[name].view(torch.uint8)), name


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("seed", range(10))
def test_attention_and_kept_path(store, seed):
    rng = np.random.default_rng(seed)
    Q, H = int(rng.choice([1, 1, 3, 33, 64])), int(rng.integers(1, 140))
    block = int(rng.choice([1, 5, 16, 64]))
    lens = [int(rng.choice([0, rng.integers(1, 700), rng.integers(1, 40)])) for _ in range(rng.integers(1, 20))]
    if seed == 0:
        lens = [5000]
    trees = [random_tree(rng, Q) for _ in lens] if seed % 2 else None
    window = int(rng.choice([0, 0, 64, 200]))
    s = Batch(store, lens, Q, H, block, seed=seed, stride=int(rng.integers(0, 4)), trees=trees, narrow=seed % 2)
    if seed % 3 == 1:
        s.lens_t[0] = s.W * block + 9  # a length past the table, and pages outside the cache
        s.table[-1, 0] = s.nb
        s.table[0, -1] = -5
    sinks = torch.zeros(H, device=DEV) if seed % 2 else None
    path = dev(np.tile(np.arange(Q), (len(lens), 1)), np.int32)
    path[:, 0] = 0 if Q == 1 else 1
    path_lens = dev(rng.integers(0, 2, len(lens)), np.int32)

    def run():
        err, work = error_word(), torch.empty(k.latent_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)
        out, lse = s.attention(window, sinks, err=err, workspace=work)
        # the cache again at the same alignment, for what moves in it
        room = torch.empty(s.cache.numel() + 16, dtype=torch.uint8, device=DEV)
        cache = room[8 * s.narrow:8 * s.narrow + s.cache.numel()]
        cache.copy_(s.cache)
        new = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
        k.tree_keep(STORES[store], cache, s.nb, block, s.table, s.lens_t, path, path_lens, new, device_error=err)
        return dict(out=out, lse=lse, cache=cache.clone(), new=new, err=err)

    if store == "bf16" and s.narrow:
        with pytest.raises(k.Dsv4Error):
            run()
        s.narrow = 0
        s.refresh()
    _same(run)


@pytest.mark.parametrize("store", STORES)
def test_requests_by_the_thousand(store):
    """64000 requests, most of them idle, in the release build; 3000 in both."""
    pages = Batch(store, [64], 1, 1, 16, seed=3)
    gen = torch.Generator(device=DEV).manual_seed(4)

    def make(N, H):
        q = torch.randn(N, 1, H, 512, generator=gen, device=DEV).bfloat16()
        table = torch.zeros(N, 9, dtype=torch.int32, device=DEV)
        table[:, :4] = pages.table[0, torch.randint(0, 4, (N, 4), generator=gen, device=DEV)]
        lens = torch.randint(0, 64, (N,), generator=gen, device=DEV, dtype=torch.int32)
        lens[torch.rand(N, generator=gen, device=DEV) < (0.33 if N < 10000 else 0.99)] = 0
        return q, table, lens

    def attend(q, table, lens):
        out, lse = torch.ones_like(q), torch.zeros(q.shape[:3], device=DEV)
        k.latent_attention(STORES[store], q, pages.cache, pages.nb, 16, table, lens, 0.04, out, lse=lse)
        return dict(out=out, lse=lse)

    some = make(3000, 5)
    _same(lambda: attend(*some))
    q, table, lens = make(64000, 2)
    got, live = attend(q, table, lens), lens > 0
    assert not bool(got["out"][~live].any()) and bool(torch.isneginf(got["lse"][~live]).all())
    alone = attend(q[live].contiguous(), table[live].contiguous(), lens[live].contiguous())
    # runs are cut elsewhere, so sums are in another order: a rounding of the output to bf16 apart
    assert torch.allclose(got["out"][live].float(), alone["out"].float(), rtol=2 ** -7, atol=2 ** -7)
    assert torch.allclose(got["lse"][live], alone["lse"], rtol=2 ** -18, atol=2 ** -18)


@pytest.mark.parametrize("T,H,D,dim,offset,dtype", [
    (1, 1, 2, 2, 0, torch.float32), (50, 3, 100, 64, 20, torch.bfloat16), (700, 5, 512, 64, 448, torch.bfloat16),
    (3000, 8, 128, 128, 0, torch.float16), (3000, 7, 64, 32, 32, torch.float32), (9, 2, 65, 6, 59, torch.float16)])
def test_rotary_table_and_rows(T, H, D, dim, offset, dtype):
    gen = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, H, D, generator=gen, device=DEV).to(dtype)
    positions = torch.randint(-2, 60, (T,), generator=gen, device=DEV)

    def run():
        err, table = error_word(), torch.zeros(57, dim, device=DEV)
        k.rope_table(k.rope_frequencies(dim), table, device_error=err)
        out, back, half = torch.zeros_like(x), x.clone(), torch.zeros_like(x)
        k.rope_rows(x, positions, table, out=out, offset=offset, device_error=err)
        k.rope_rows(back, positions, table, offset=offset, inverse=True, device_error=err)
        k.rope_rows(x, positions, table, out=half, offset=offset, layout=k.ROPE_HALF, device_error=err)
        return dict(table=table, out=out, back=back, half=half, err=err)

    _same(run)
