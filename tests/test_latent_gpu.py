"""Attention over the FP8 and bf16 caches on the GPU, for chains and trees, against its 64-bit
definition (oracle/latent.py).

Bounds, fixed from the arithmetic: an fp32 score of 512 terms is off by at most scale * sum|q||k| *
2^-15 (512 roundings of 2^-24 each); probabilities are rounded to bf16 (half a step, 2^-8)
before the product with the rows, and the output once more; lse to 2^-22 of itself beside
the score's error.
"""
import numpy as np
import pytest

from oracle import latent

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kv_norm_rope_gb300 as k  # noqa: E402

DEV = torch.device("cuda:0")
STORES = {"fp8": k.STORE_FP8, "bf16": k.STORE_BF16}


def dev(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x, dtype)).to(DEV)


def bf16(x):
    """float array -> (bf16 tensor on the GPU, the float64 values it holds)"""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


def bf16_bytes(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint8)


def error_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def random_tree(rng, q_len, drafted=None):
    """Words of a random tree of `drafted` tokens, zeros behind them."""
    words = []
    for j in range(q_len if drafted is None else drafted):
        parent = int(rng.integers(max(0, j - 5), j)) if j else None
        words.append(1 << j | (words[parent] if j else 0))
    return words + [0] * (q_len - len(words))


def words_tensor(trees):
    return dev(np.array(trees, np.uint64).view(np.int64).reshape(len(trees), -1))


class Batch:
    """Requests over shuffled pages of random rows; everything that no request reads is 0xff (NaN)."""

    def __init__(self, store, lens, Q, H, block=16, seed=0, stride=0, gain=1.0, trees=None, spare=3, narrow=0):
        rng = np.random.default_rng(seed)
        self.store, self.lens, self.Q, self.H, self.block = store, lens, Q, H, block
        B = len(lens)
        pages = [-(-n // block) for n in lens]
        self.nb, self.W = sum(pages) + spare, max(max(pages), 1)
        order = rng.permutation(self.nb)
        table = np.full((B, self.W + stride), -1, np.int32)
        slot = sum(latent.SLOT[store])
        cache = np.full(self.nb * block * slot, 255, np.uint8)
        at = 0
        for b, n in enumerate(lens):
            table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        self.table_np, self.cache_np, self.rng = table, cache, rng
        for b, n in enumerate(lens):
            for i in range(n):
                data, scale = self.row(b, i)
                if store == "bf16":
                    data[:] = bf16_bytes(rng.standard_normal(512))
                else:
                    codes = rng.integers(0, 256, 448)
                    data[:448] = np.where(codes & 127 == 127, 0, codes)  # no NaN; subnormal codes among them
                    scale[:7], scale[7] = rng.integers(116, 121, 7), 0
                    data[448:] = bf16_bytes(rng.standard_normal(64) * 2)
        self.trees = trees
        self.tree = None if trees is None else words_tensor(trees)
        self.q, self.q64 = bf16(rng.standard_normal((B, Q, H, 512)) * gain)
        self.scale = 512.0 ** -0.5
        self.table = dev(table)[:, :self.W]
        self.lens_t = dev(lens, np.int32)
        self.narrow = narrow
        self.refresh()

    def row(self, b, i):
        return latent.row_bytes(self.cache_np, self.store, self.block,
                                self.table_np[b, i // self.block] * self.block + i % self.block)

    def refresh(self):
        """After the cache image changed: the device's copy (8 bytes past a 16-byte boundary if narrow)."""
        if self.narrow:
            room = torch.empty(self.cache_np.size + 16, dtype=torch.uint8, device=DEV)
            self.cache = room[8:8 + self.cache_np.size]
            self.cache.copy_(torch.from_numpy(self.cache_np))
        else:
            self.cache = dev(self.cache_np)
        self.rows, self.ok = [], []
        for b, n in enumerate(self.lens):
            rows, ok = latent.rows_of(self.cache_np, self.store, self.block, self.table_np[b], n, self.nb)
            self.rows.append(rows)
            self.ok.append(ok)

    def attention(self, window=0, sinks=None, lse=True, stream=None, err=None, out=None, workspace=None):
        B = len(self.lens)
        out = torch.full((B, self.Q, self.H, 512), 9.0, dtype=torch.bfloat16, device=DEV) if out is None else out
        lse = torch.full((B, self.Q, self.H), 9.0, device=DEV) if lse else None
        k.latent_attention(STORES[self.store], self.q, self.cache, self.nb, self.block, self.table, self.lens_t,
                           self.scale, out, lse=lse, sinks=sinks, window=window, tree=self.tree, stream=stream,
                           device_error=err, workspace=workspace)
        return out, lse

    def check(self, out, lse, window=0, sinks=None, lens=None, skip=()):
        out = out.double().cpu().numpy()
        sinks64 = None if sinks is None else sinks.double().cpu().numpy()
        for b, n in enumerate(self.lens if lens is None else lens):
            tree = None if self.trees is None else self.trees[b]
            want, wlse, size, reach = latent.attention(self.q64[b], self.rows[b][:n], self.ok[b][:n], n, self.scale,
                                                       window, sinks64, tree)
            ds = self.scale * reach * 2.0 ** -15 + 2.0 ** -18
            tol = np.abs(want) * 2.0 ** -8 + size * (2.0 ** -8 + 2 * ds[..., None]) + 1e-30
            got = None if lse is None else lse[b].double().cpu().numpy()
            for j in range(self.Q):
                if (b, j) in skip:
                    continue
                off = np.abs(out[b, j] - want[j])
                assert np.all(off <= tol[j]), (b, j, np.max(off - tol[j]))
                if got is not None:
                    empty = np.isneginf(wlse[j])
                    assert np.array_equal(np.isneginf(got[j]), empty)
                    off = np.abs(got[j][~empty] - wlse[j][~empty])
                    assert np.all(off <= ds[j][~empty] + np.abs(wlse[j][~empty]) * 2.0 ** -22)


CASES = [
    # lens, Q, H, block
    ([1], 1, 1, 16),
    ([5, 0, 2], 1, 8, 1),
    ([63, 64, 65], 1, 16, 64),
    ([127, 128, 129, 1], 1, 3, 27),
    ([64, 700], 1, 64, 64),
    ([300], 1, 65, 16),
    ([200, 333], 1, 128, 64),
    ([40], 1, 200, 5),
    ([3, 130, 1], 4, 8, 16),
    ([150, 2], 5, 13, 7),
    ([260, 90], 16, 24, 64),
    ([70], 70, 3, 64),
    ([1500], 2, 20, 128),
    ([17] * 40, 1, 8, 16),
    ([0, 0], 2, 4, 16),
]


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("lens,Q,H,block", CASES)
def test_attention(store, lens, Q, H, block):
    s = Batch(store, lens, Q, H, block, seed=len(lens) + Q + H)
    err = error_word()
    out, lse = s.attention(err=err)
    s.check(out, lse)
    assert int(err.item()) == 0


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("lens,Q,H,block", [CASES[1], CASES[3], CASES[8], CASES[9], CASES[10], CASES[12]])
@pytest.mark.parametrize("window", [1, 3, 63, 64, 100, 5000])
def test_window(store, lens, Q, H, block, window):
    s = Batch(store, lens, Q, H, block, seed=window)
    out, lse = s.attention(window=window)
    s.check(out, lse, window)


TREES = [
    # lens, Q, H, block, window
    ([1], 1, 1, 16, 0),
    ([7, 0, 3], 7, 8, 1, 0),          # a request shorter than its drafted tokens
    ([64, 65, 128, 200], 16, 3, 27, 0),
    ([300, 90], 16, 64, 64, 0),
    ([500], 61, 5, 16, 100),
    ([64, 130], 64, 2, 64, 64),
    ([1000, 64], 64, 20, 5, 0),
    ([333, 12, 90], 5, 128, 16, 5),
    ([40, 700], 33, 7, 64, 650),
    ([90] * 30, 6, 4, 16, 20),
]


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("lens,Q,H,block,window", TREES)
def test_tree(store, lens, Q, H, block, window):
    rng = np.random.default_rng(Q + len(lens))
    trees = [random_tree(rng, Q, Q if b % 2 == 0 else int(rng.integers(0, Q + 1))) for b in range(len(lens))]
    s = Batch(store, lens, Q, H, block, seed=Q, trees=trees)
    err = error_word()
    out, lse = s.attention(window=window, err=err)
    s.check(out, lse, window)
    assert int(err.item()) == 0


@pytest.mark.parametrize("store", STORES)
def test_tree_words_of_any_kind(store):
    """Words that no tree has: no own bit, every bit, bits past the last token, the sign bit alone."""
    Q = 9
    trees = [[0, 1, 2, (1 << 64) - 1, 1 << 63, 1 << 8, 0b101, 1 << 9, 0],
             [1 << i for i in range(Q)],
             [0] * Q]
    sinks = torch.linspace(-3, 3, 10, device=DEV)
    for window, sink in ((0, None), (9, sinks), (30, sinks)):
        s = Batch(store, [100, 60, 50], Q, 10, 16, seed=3, trees=trees)
        out, lse = s.attention(window=window, sinks=sink)
        s.check(out, lse, window, sink)
        assert bool((out[2] == 0).all())
    s = Batch(store, [64], 64, 3, 16, seed=4, trees=[[1 << 63] + [(1 << 64) - 1] * 62 + [1 << 63 | 1]])
    out, lse = s.attention()
    s.check(out, lse)


@pytest.mark.parametrize("store", STORES)
def test_chain_given_as_a_tree(store):
    Q = 12
    s = Batch(store, [400, 12, 77], Q, 16, 16, seed=5)
    out, lse = s.attention()
    s.check(out, lse)
    s.tree = words_tensor([[(2 << j) - 1 for j in range(Q)]] * 3)
    out, lse = s.attention()
    s.check(out, lse)  # against the chain's definition


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("lens,Q,H,block", [CASES[1], CASES[8], CASES[14], CASES[6]])
def test_sinks(store, lens, Q, H, block):
    s = Batch(store, lens, Q, H, block, seed=4)
    sinks = torch.linspace(-8, 8, H, device=DEV)
    out, lse = s.attention(sinks=sinks, window=50)
    s.check(out, lse, 50, sinks)
    sinks = torch.full((H,), -float("inf"), device=DEV)  # a sink that takes nothing
    out, lse = s.attention(sinks=sinks)
    s.check(out, lse)
    # a sink far above every score leaves nothing for the keys
    sinks = torch.full((H,), 300.0, device=DEV)
    out, lse = s.attention(sinks=sinks)
    s.check(out, lse, 0, sinks)


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("Q,H,narrow", [(1, 4, 0), (3, 40, 1)])
@pytest.mark.parametrize("order", ["rising", "falling", "spike"])
def test_scores_far_apart(store, Q, H, narrow, order):
    """Scores from -400 to 400 along the keys: the running maximum moves in every tile, or the
    first tile's is never reached again, or one key takes everything."""
    n = 1100
    s = Batch(store, [n], Q, H, 16, seed=11, narrow=narrow if store == "fp8" else 0)
    rng = np.random.default_rng(12)
    way = rng.integers(0, 2, 64) * 2 - 1.0
    level = {"rising": np.linspace(-1, 1, n), "falling": np.linspace(1, -1, n),
             "spike": np.where(np.arange(n) == 700, 1.0, -1.0)}[order]
    for i in range(n):
        data, scale = s.row(0, i)
        if store == "fp8":
            scale[:7] = 112
        data[-128:] = bf16_bytes(way * level[i] * 12)
    s.refresh()
    q = s.q64.copy()
    q[..., 448:] = way * 12 * np.linspace(0.5, 1, H)[None, None, :, None]
    s.q, s.q64 = bf16(q)
    out, lse = s.attention()
    s.check(out, lse)


@pytest.mark.parametrize("store", STORES)
def test_a_nan_in_q_stays_in_its_row(store):
    s = Batch(store, [30, 200], 1, 2, 16, seed=13)
    q = s.q64.copy()
    q[0] = 0.0
    s.q, s.q64 = bf16(q)
    out, lse = s.attention()
    s.check(out, lse)
    q[0, 0, 1, 3] = np.nan
    s.q, _ = bf16(q)
    out, lse = s.attention()
    assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(lse[0, 0, 1])
    assert torch.isfinite(out[0, 0, 0]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("store", STORES)
def test_scores_far_below_zero(store):
    """Every score of a row hugely negative: the softmax is of their differences alone."""
    s = Batch(store, [300], 1, 4, 16, seed=25)
    for i in range(300):
        s.row(0, i)[0][-128:-126] = bf16_bytes([1.0])
    s.refresh()
    q = np.zeros_like(s.q64)
    q[..., 448] = -np.exp2(np.array([10.0, 40.0, 80.0, 110.0]))  # the same score for every key
    s.q, s.q64 = bf16(q)
    out, lse = s.attention()
    got = out.double().cpu().numpy()[0, 0]
    want, size = s.rows[0].mean(0), np.abs(s.rows[0]).mean(0)
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + size * 2.0 ** -7)
    assert np.allclose(lse[0, 0].double().cpu().numpy(), s.scale * q[0, 0, :, 448] + np.log(300), rtol=2.0 ** -20, atol=0)


BAD = {"fp8": ["code", "exponent", "large", "rope nan", "rope inf", "rope -inf", "all"],
       "bf16": ["nan", "inf", "-inf", "all"]}


def spoil(s, b, i, kind):
    data, scale = s.row(b, i)
    if kind == "all":
        data[:], scale[:] = 255, 255
    elif kind == "code":
        data[200] = 0xff
    elif kind == "exponent":
        scale[3] = 255
    elif kind == "large":
        scale[6] = 183
    else:
        at = data.size - 2 * 45 if kind.startswith("rope") else 2 * 100
        data[at:at + 2] = bf16_bytes([float(kind.replace("rope ", ""))])


@pytest.mark.parametrize("store,kind", [(s, kind) for s in STORES for kind in BAD[s]])
@pytest.mark.parametrize("n,Q,H,window", [(300, 3, 4, 0), (258, 3, 40, 0), (300, 3, 4, 100), (500, 3, 64, 200)])
def test_rows_not_finite(store, kind, n, Q, H, window):
    """A row that is not finite makes NaN of the tokens that see it and of no others."""
    bad = n - 1 if window == 0 else n - Q + 1 - window  # seen by the last token alone, or the first
    s = Batch(store, [n, 40], Q, H, 16, seed=26)
    spoil(s, 0, bad, kind)
    s.cache = dev(s.cache_np)
    out, lse = s.attention(window=window)
    hit = Q - 1 if window == 0 else 0
    assert torch.isnan(out[0, hit]).all() and torch.isnan(lse[0, hit]).all()
    s.check(out, lse, window, skip={(0, hit)})


@pytest.mark.parametrize("store", STORES)
def test_drafted_rows_of_padding_and_siblings_not_finite(store):
    """Drafted keys that some or no token sees hold NaN: those that see them alone get it."""
    Q, n = 8, 150
    tree = [1, 0b11, 0b101, 0b1011, 0b10101, 0, 0, 0]
    s = Batch(store, [n, n], Q, 9, 16, seed=27, trees=[tree, tree])
    c = n - Q
    for i in (4, 5, 6, 7):
        spoil(s, 0, c + i, "all")
    s.cache = dev(s.cache_np)
    out, lse = s.attention()
    assert torch.isnan(out[0, 4]).all() and torch.isnan(lse[0, 4]).all()
    s.check(out, lse, skip={(0, 4)})
    assert bool((out[:, 5:] == 0).all()) and bool(torch.isneginf(lse[:, 5:]).all())


@pytest.mark.parametrize("store", STORES)
def test_bad_pages_and_lengths(store):
    """A block outside the cache takes no part and is flagged; so is a length past the table."""
    s = Batch(store, [300, 100, 50], 1, 8, 16, seed=14)
    s.table_np[0, 3] = s.nb
    s.table_np[0, 18] = -7          # the last, partly filled block of request 0
    s.table_np[1, :] = 2 ** 31 - 1  # no valid block at all
    s.table = dev(s.table_np)
    s.refresh()
    err = error_word()
    out, lse = s.attention(err=err)
    s.check(out, lse)
    assert int(err.item()) == k.DEVERR_SLOT_RANGE
    s = Batch(store, [304, 100, 50], 1, 8, 16, seed=15)
    s.lens_t = dev([19 * 16 + 5, 100, -4], np.int32)
    err = error_word()
    out, lse = s.attention(err=err)
    s.check(out, lse, lens=[304, 100, 0])
    assert int(err.item()) == k.DEVERR_SLOT_RANGE


def test_fp8_rows_at_the_ends_of_their_range():
    """Exponent bytes from 49 (values around 2^-78) to 182 (below 2^64), subnormal codes and large ones."""
    for e, gain in ((55, 2.0 ** 60), (90, 2.0 ** 30), (127, 1.0), (160, 2.0 ** -30), (182, 2.0 ** -50)):
        s = Batch("fp8", [150], 2, 6, 16, seed=e, gain=gain)
        for i in range(150):
            data, scale = s.row(0, i)
            scale[:7] = e
            data[448:] = bf16_bytes(s.rng.standard_normal(64) * 2.0 ** (e - 127))
        s.refresh()
        s.scale = float(np.float32(1.0 / (gain * 2.0 ** (e - 127) * 200 * 22)))
        out, lse = s.attention()
        s.check(out, lse)


@pytest.mark.parametrize("store,block,narrow", [("fp8", 1, 0), ("fp8", 7, 1), ("fp8", 16, 1), ("fp8", 27, 0), ("bf16", 7, 0)])
def test_rows_off_16_byte_boundaries(store, block, narrow):
    s = Batch(store, [200, 31], 3, 24, block, seed=block, narrow=narrow)
    out, lse = s.attention()
    s.check(out, lse)


def _ragged(count, seed):
    rng = np.random.default_rng(seed)
    lens = np.where(rng.random(count) < 0.2, 0, rng.integers(1, 60, count))
    lens[rng.choice(count, 5, replace=False)] = rng.integers(200, 900, 5)
    return [int(n) for n in lens]


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("count,Q,H", [(25, 1, 70), (160, 2, 3), (511, 1, 2), (513, 1, 2), (300, 1, 130)])
def test_many_short_requests_among_longer_ones(store, count, Q, H):
    """Runs of several requests, some of them idle, and requests over several runs."""
    s = Batch(store, _ragged(count, count), Q, H, 16, seed=27)
    out, lse = s.attention()
    s.check(out, lse)
    again, _ = s.attention()
    assert torch.equal(out, again)


@pytest.mark.parametrize("store", STORES)
def test_strided_table_and_other_stream(store):
    s = Batch(store, [90, 200], 2, 8, 16, seed=16, stride=5)
    assert not s.table.is_contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = s.attention(stream=side)
    side.synchronize()
    s.check(out, lse)
    ws = torch.empty(k.latent_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)
    out2 = torch.empty_like(out)
    k.latent_attention(STORES[store], s.q, s.cache, s.nb, s.block, s.table, s.lens_t, s.scale, out2, workspace=ws,
                       stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, out2)


@pytest.mark.parametrize("store", STORES)
def test_in_a_graph_follows_new_lengths_and_trees(store):
    """Captured once; replayed after the lengths and the trees changed on the device."""
    rng = np.random.default_rng(17)
    s = Batch(store, [700, 300], 6, 16, 16, seed=17, trees=[random_tree(rng, 6), random_tree(rng, 6)])
    out = torch.zeros(2, 6, 16, 512, dtype=torch.bfloat16, device=DEV)
    s.attention(out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, lse = s.attention(out=out)
    for lens in ([700, 300], [650, 0], [1, 299]):
        s.lens_t.copy_(dev(lens, np.int32))
        s.trees = [random_tree(rng, 6), random_tree(rng, 6, 4)]
        s.tree.copy_(words_tensor(s.trees))
        g.replay()
        torch.cuda.synchronize()
        s.check(out, lse, lens=lens)


@pytest.mark.parametrize("store", STORES)
def test_two_streams_at_once_with_a_workspace_each(store):
    batches = [Batch(store, [900, 40 * i + 30], 2, 24, 16, seed=30 + i) for i in range(2)]
    alone = [s.attention()[0] for s in batches]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(o) for o in alone]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, stream, out in zip(batches, streams, outs):
            s.attention(stream=stream, out=out, lse=False)
    torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("store", STORES)
def test_same_bits_again(store):
    s = Batch(store, [3000, 1, 777], 2, 40, 64, seed=18)
    first, lse = s.attention()
    for _ in range(3):
        out, lse2 = s.attention()
        assert torch.equal(out, first) and torch.equal(lse, lse2)


@pytest.mark.parametrize("store", STORES)
def test_offsets_past_4_gib(store):
    """Pages at the far end of a cache of 5 GB."""
    slot = sum(latent.SLOT[store])
    block, nb = 64, 5 * 10 ** 9 // (64 * slot)
    s = Batch(store, [500], 1, 8, block, seed=19)
    cache = torch.zeros(nb * block * slot, dtype=torch.uint8, device=DEV)
    far = nb - s.nb
    cache[far * block * slot:] = s.cache
    s.cache, s.nb = cache, nb
    s.table = s.table + far
    out, lse = s.attention()
    s.check(out, lse)


@pytest.mark.parametrize("store", STORES)
def test_leaves_what_is_not_its_own(store):
    """Rows behind the batch's last, and a workspace's bytes behind its size, stay as they were."""
    s = Batch(store, [70, 5], 2, 3, 16, seed=20)
    room = torch.full((3, 2, 3, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    n = k.latent_attention_workspace_bytes()
    ws = torch.full((n + 64,), 77, dtype=torch.uint8, device=DEV)
    out, lse = s.attention(out=room[:2], workspace=ws)
    s.check(out, lse)
    assert bool((room[2] == 7).all()) and bool((ws[n:] == 77).all())


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    store = "fp8" if seed % 2 else "bf16"
    tree = seed % 4 >= 2
    Q = int(rng.integers(1, 30)) if tree else int(rng.choice([1, 1, 2, 9, 100]))
    H, block = int(rng.choice([1, 5, 16, 33, 64, 128])), int(rng.choice([1, 5, 16, 64]))
    lens = [int(rng.choice([0, rng.integers(1, 40), rng.integers(1, 600)])) for _ in range(int(rng.integers(1, 12)))]
    window = int(rng.choice([0, 0, 1, 70, 300]))
    if tree and window:
        window = max(window, Q)
    trees = [random_tree(rng, Q, int(rng.integers(0, Q + 1))) for _ in lens] if tree else None
    s = Batch(store, lens, Q, H, block, seed=seed, trees=trees, stride=int(rng.integers(0, 3)))
    sinks = dev(rng.standard_normal(H), np.float32) if rng.random() < 0.5 else None
    out, lse = s.attention(window=window, sinks=sinks)
    s.check(out, lse, window, sinks)
