"""Keeping an accepted path's rows on the GPU, against the byte-wise oracle: every byte of the
cache is compared."""
import numpy as np
import pytest

from oracle import latent
from tests.test_latent_gpu import DEV, dev, error_word, k, torch

pytestmark = pytest.mark.gpu

STORES = {"fp8": k.STORE_FP8, "bf16": k.STORE_BF16, "fp4": k.STORE_FP4, "indexer": k.STORE_INDEXER}


def run(store, block, lens, Q, paths, path_lens, seed=0, table=None, alias=False, narrow=0, stride=0, stream=None):
    """paths: int32 [B, Q].  Returns the flags after comparing everything else."""
    rng = np.random.default_rng(seed)
    B, slot = len(lens), sum(latent.SLOT[store])
    pages = [max(-(-max(n, 1) // block), 1) for n in lens]
    nb, W = sum(pages) + 2, max(pages)
    order, at = rng.permutation(nb), 0
    mine = np.full((B, W + stride), -1, np.int32)
    for b in range(B):
        mine[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    if table is not None:
        table(mine, nb)
    before = rng.integers(0, 256, nb * block * slot).astype(np.uint8)
    want, new, flagged = before.copy(), [], False
    for b, n in enumerate(lens):
        limit = W * block
        length, bad = latent.keep(want, store, block, mine[b], min(n, limit), Q, paths[b], int(path_lens[b]), nb)
        new.append(length)
        flagged = flagged or bad or n > limit
    room = torch.empty(before.size + 16, dtype=torch.uint8, device=DEV)
    cache = room[narrow:narrow + before.size]
    cache.copy_(torch.from_numpy(before))
    lens_t = dev(lens, np.int32)
    new_t = lens_t if alias else torch.full((B,), -9, dtype=torch.int32, device=DEV)
    err = error_word()
    k.tree_keep(STORES[store], cache, nb, block, dev(mine)[:, :W], lens_t, dev(paths, np.int32),
                dev(path_lens, np.int32), new_t, device_error=err, stream=stream)
    torch.cuda.synchronize()
    assert new_t.tolist() == new
    assert np.array_equal(cache.cpu().numpy(), want)
    assert int(err.item()) == (k.DEVERR_SLOT_RANGE if flagged else 0)


def random_paths(rng, B, Q):
    paths, lens = np.full((B, Q), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        lens[b] = rng.integers(0, Q + 1)
        paths[b, :lens[b]] = np.sort(rng.choice(Q, lens[b], replace=False))
    return paths, lens


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("Q,block", [(1, 16), (2, 1), (7, 5), (32, 64), (33, 27), (64, 16), (64, 1), (64, 64)])
def test_random_paths(store, Q, block):
    rng = np.random.default_rng(Q + block)
    B = 9
    lens = [int(rng.integers(Q, Q + 150)) for _ in range(B)]
    lens[2], lens[5] = 0, Q
    paths, path_lens = random_paths(rng, B, Q)
    run(store, block, lens, Q, paths, path_lens, seed=Q, alias=Q % 2 == 0, stride=block % 3)


@pytest.mark.parametrize("store", STORES)
def test_whole_and_empty_and_last_paths(store):
    """All drafted rows kept (nothing moves), none, every other one, the last one alone."""
    Q = 64
    paths = np.full((4, Q), -1, np.int32)
    paths[0] = np.arange(Q)
    paths[2, :32] = np.arange(1, 64, 2)
    paths[3, 0] = 63
    run(store, 16, [200, 64, 100, 129], Q, paths, [64, 0, 32, 1])


@pytest.mark.parametrize("store,narrow", [("fp8", 8), ("indexer", 4), ("indexer", 8), ("indexer", 0)])
@pytest.mark.parametrize("block", [2, 3])
def test_rows_off_16_byte_boundaries(store, narrow, block):
    rng = np.random.default_rng(narrow)
    paths, path_lens = random_paths(rng, 3, 20)
    run(store, block, [40, 20, 33], 20, paths, path_lens, narrow=narrow)


@pytest.mark.parametrize("store", ["fp8", "bf16"])
def test_wrong_paths_end_where_they_go_wrong(store):
    Q = 40
    good = np.arange(1, 33, dtype=np.int32)
    paths = np.tile(np.concatenate([good, np.full(8, -1)]).astype(np.int32), (9, 1))
    lens = np.full(9, 32, np.int32)
    paths[1, 5] = paths[1, 4]        # twice the same
    paths[2, 31] = 3                 # falls
    paths[3, 31] = 40                # past the drafted
    paths[4, 0] = -1                 # below them
    lens[5] = 41                     # longer than they are
    lens[6] = -2
    paths[7, 35:] = [36, 35, 37, 38, 39]
    paths[7, 32:35] = [33, 34, 36]   # stops between the two words of entries
    lens[7] = 40
    for one in range(9):
        run(store, 16, [150], Q, paths[one:one + 1], lens[one:one + 1], seed=one)
    run(store, 16, [150] * 9, Q, paths, lens)


def test_lengths_and_blocks_out_of_range():
    rng = np.random.default_rng(1)
    Q = 12
    paths, path_lens = random_paths(rng, 5, Q)
    path_lens[0], paths[0, :3] = 3, [2, 5, 9]
    run("fp8", 4, [11, 5, 60, 60, 0], Q, paths, path_lens)      # fewer keys than drafted tokens
    run("fp8", 4, [-3, 40, 60, 60, 0], Q, paths, path_lens)
    def spoil(table, nb):
        table[0, 13], table[1, 14], table[2, 12] = nb, -1, 2 ** 31 - 1
    paths, path_lens = np.tile(np.arange(1, Q + 1), (3, 1)), np.full(3, Q - 1, np.int32)
    paths[:, Q - 1] = -1
    run("bf16", 4, [60, 60, 60], Q, paths, path_lens, table=spoil)
    run("bf16", 4, [60, 58, 59], Q, paths, path_lens, table=lambda t, nb: None)


def test_length_past_the_table():
    err, Q = error_word(), 4
    cache = torch.arange(32 * 1024, device=DEV).to(torch.uint8)
    before = cache.clone().view(32, 1024)
    new = torch.zeros(1, dtype=torch.int32, device=DEV)
    k.tree_keep(k.STORE_BF16, cache, 2, 16, dev([[1, 0]], np.int32), dev([99], np.int32), dev([[1, 3, -1, -1]], np.int32),
                dev([2], np.int32), new, device_error=err)
    after = cache.view(32, 1024)
    # 32 keys: the last four are slots 12..15 of block 0
    assert new.tolist() == [30] and int(err.item()) == k.DEVERR_SLOT_RANGE
    assert torch.equal(after[12], before[13]) and torch.equal(after[13], before[15])
    untouched = torch.ones(32, dtype=torch.bool)
    untouched[12:14] = False
    assert torch.equal(after[untouched.to(DEV)], before[untouched.to(DEV)])


def test_many_requests_on_another_stream():
    rng = np.random.default_rng(5)
    B, Q = 700, 24
    lens = [int(n) for n in rng.integers(Q, 90, B)]
    paths, path_lens = random_paths(rng, B, Q)
    run("indexer", 16, lens, Q, paths, path_lens, stream=torch.cuda.Stream())


def test_offsets_past_4_gib():
    slot, block = 1024, 64
    nb = 5 * 10 ** 9 // (slot * block)
    cache = torch.zeros(nb * block, slot, dtype=torch.uint8, device=DEV)
    last = (nb - 1) * block
    cache[last + 10] = 7
    cache[last + 13] = 9
    new = torch.zeros(1, dtype=torch.int32, device=DEV)
    k.tree_keep(k.STORE_BF16, cache, nb, block, dev([[nb - 1]], np.int32), dev([14], np.int32),
                dev([[2, 5, -1, -1, -1, -1]], np.int32), dev([2], np.int32), new)
    assert new.tolist() == [10]
    assert bool((cache[last + 8] == 7).all()) and bool((cache[last + 9] == 9).all())
    assert int(cache.any(1).sum()) == 4


def test_in_a_graph_and_before_the_next_step():
    """Verify, keep, go on, in one graph: the lengths that the next attention reads are the new ones."""
    Q, H, block, nb = 8, 4, 16, 12
    gen = torch.Generator(device=DEV).manual_seed(3)
    first = torch.randn(nb * block, 512, generator=gen, device=DEV).to(torch.bfloat16)
    q = torch.randn(1, Q, H, 512, generator=gen, device=DEV).to(torch.bfloat16)
    table = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)[None]
    path = dev([[0, 2, 6, -1, -1, -1, -1, -1]], np.int32)
    path_lens, start = dev([3], np.int32), dev([100], np.int32)
    lens, cache = start.clone(), first.clone()
    out, lse = torch.empty(1, 1, H, 512, dtype=torch.bfloat16, device=DEV), torch.empty(1, 1, H, device=DEV)

    def step():
        cache.copy_(first)
        lens.copy_(start)
        k.tree_keep(k.STORE_BF16, cache, nb, block, table, lens, path, path_lens, lens)
        k.latent_attention(k.STORE_BF16, q[:, :1].contiguous(), cache, nb, block, table, lens, 0.05, out, lse=lse)

    step()
    torch.cuda.synchronize()
    eager = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager) and lens.tolist() == [95]
    keys = [int(table[0, i // block]) * block + i % block for i in list(range(92)) + [92, 94, 98]]
    rows = first[keys].double()
    s = 0.05 * (q[0, 0].double() @ rows.T)
    want = torch.softmax(s, 1) @ rows
    size = torch.softmax(s, 1) @ rows.abs()
    assert bool(((out[0, 0].double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2.0 ** -7.9).all())
