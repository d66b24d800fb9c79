"""The table, the insert, tree attention, the rotation back and the kept path, one after the other
as a server that drafts tokens uses them."""
import numpy as np
import pytest

from oracle import latent
from tests.test_latent_gpu import DEV, STORES, dev, error_word, k, random_tree, torch, words_tensor

pytestmark = pytest.mark.gpu

BLOCK, EPS, SCALE, POSITIONS = 16, 1e-6, 512.0 ** -0.5, 400


def cos_sin_table(err):
    table = torch.empty(POSITIONS, 64, device=DEV)
    k.rope_table(k.rope_frequencies(64, 10000.0, k.ROPE_YARN, 4.0, 64.0), table, magnitude=1.05, device_error=err)
    return table


def cache_of(store, nb):
    size = k.fp8_cache_bytes(nb, BLOCK) if store == "fp8" else k.bf16_cache_bytes(nb, BLOCK)
    return torch.full((size,), 255, dtype=torch.uint8, device=DEV)  # NaN wherever nothing is inserted


class Server:
    """Two caches for the same requests: one that drafts trees, one that takes the accepted tokens alone."""

    def __init__(self, store, lens, Q, H, seed):
        self.store, self.Q, self.H, self.B = store, Q, H, len(lens)
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.err = error_word()
        self.cos_sin = cos_sin_table(self.err)
        self.W = -(-(max(lens) + 3 * Q) // BLOCK)
        self.nb = self.B * self.W + 1
        self.table_np = self.rng.permutation(self.nb)[:self.B * self.W].reshape(self.B, self.W).astype(np.int32)
        self.table = dev(self.table_np)
        self.w = (1 + 0.1 * self.randn(512)).bfloat16()
        self.drafting, self.plain = cache_of(store, self.nb), cache_of(store, self.nb)
        kv = self.randn(sum(lens), 512).bfloat16()
        at = [(b, i) for b, n in enumerate(lens) for i in range(n)]
        for cache in (self.drafting, self.plain):
            self.insert(cache, None, kv, at, [i for _, i in at])
        self.lens = list(lens)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=DEV)

    def insert(self, cache, q, kv, at, positions):
        slots = dev([int(self.table_np[b, i // BLOCK]) * BLOCK + i % BLOCK if i >= 0 else -1 for b, i in at], np.int64)
        k.insert(STORES[self.store], q, kv, self.w, dev(positions, np.int64), self.cos_sin, slots, cache, self.nb,
                 BLOCK, EPS, device_error=self.err)

    def attend(self, cache, q, lens, tree=None):
        out = torch.empty_like(q)
        k.latent_attention(STORES[self.store], q, cache, self.nb, BLOCK, self.table, lens, SCALE, out, tree=tree,
                           device_error=self.err)
        return out


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("Q,H,lens", [(1, 3, [5]), (7, 16, [1, 40, 129]), (33, 4, [64, 17]), (64, 2, [100])])
def test_drafted_steps(store, Q, H, lens):
    s = Server(store, lens, Q, H, seed=Q)
    for step in range(2):
        trees = [random_tree(s.rng, Q, Q - b % 2 * (Q // 3)) for b in range(s.B)]
        depth = [[max(bin(word).count("1"), 1) - 1 for word in words] for words in trees]
        positions = [s.lens[b] + depth[b][j] for b in range(s.B) for j in range(Q)]
        q, kv = s.randn(s.B * Q, H, 512).bfloat16(), s.randn(s.B * Q, 512).bfloat16()
        # the tokens of padding are not inserted: their slots hold NaN
        at = [(b, s.lens[b] + j if trees[b][j] else -1) for b in range(s.B) for j in range(Q)]
        s.insert(s.drafting, q, kv, at, positions)
        q = q.view(s.B, Q, H, 512)
        lens_t = dev([n + Q for n in s.lens], np.int32)
        out = s.attend(s.drafting, q, lens_t, words_tensor(trees))

        # against the definition, over the cache's bytes
        image, q64, out64 = s.drafting.cpu().numpy(), q.double().cpu().numpy(), out.double().cpu().numpy()
        for b in range(s.B):
            n = s.lens[b] + Q
            rows, ok = latent.rows_of(image, store, BLOCK, s.table_np[b], n, s.nb)
            want, _, size, reach = latent.attention(q64[b], rows, ok, n, SCALE, tree=trees[b])
            ds = SCALE * reach * 2.0 ** -15 + 2.0 ** -18
            assert np.all(np.abs(out64[b] - want) <= np.abs(want) * 2.0 ** -8 + size * (2.0 ** -8 + 2 * ds[..., None]))

        # the output's trailing dims turned back by its token's angles
        turned = out.clone()
        k.rope_rows(turned.view(-1, H, 512), dev(positions, np.int64), s.cos_sin, inverse=True, device_error=s.err)
        angles = s.cos_sin.double().cpu().numpy()[positions].reshape(s.B, Q, 1, 64)
        even, odd = out64[..., 448::2], out64[..., 449::2]
        cos, sin = angles[..., :32], angles[..., 32:]
        want = np.stack([even * cos + odd * sin, odd * cos - even * sin], -1).reshape(s.B, Q, H, 64)
        # one rounding to bf16, and before it three to fp32, of the two products' size at most
        size = np.repeat(np.abs(even) * np.abs(cos) + np.abs(odd) * np.abs(sin) +
                         np.abs(odd) * np.abs(cos) + np.abs(even) * np.abs(sin), 2, -1)
        got = turned.double().cpu().numpy()
        assert np.array_equal(got[..., :448], out64[..., :448])
        assert np.all(np.abs(got[..., 448:] - want) <= np.abs(want) * 2.0 ** -8 + size * 2.0 ** -21)

        # a random token's path is accepted; the other cache gets those tokens one after the other
        path, path_lens = np.full((s.B, Q), -1, np.int32), np.zeros(s.B, np.int32)
        for b in range(s.B):
            live = [j for j in range(Q) if trees[b][j]]
            word = trees[b][int(s.rng.choice(live))]
            kept = [j for j in range(Q) if word >> j & 1]
            path[b, :len(kept)], path_lens[b] = kept, len(kept)
            s.insert(s.plain, None, kv.view(s.B, Q, 512)[b, kept].contiguous(),
                     [(b, s.lens[b] + i) for i in range(len(kept))], [s.lens[b] + i for i in range(len(kept))])
        k.tree_keep(STORES[store], s.drafting, s.nb, BLOCK, s.table, lens_t, dev(path), dev(path_lens), lens_t,
                    device_error=s.err)
        s.lens = [n + int(kept) for n, kept in zip(s.lens, path_lens)]
        assert lens_t.tolist() == s.lens
        drafted, plain = s.drafting.cpu().numpy(), s.plain.cpu().numpy()
        for b, n in enumerate(s.lens):
            for i in range(n):
                slot = int(s.table_np[b, i // BLOCK]) * BLOCK + i % BLOCK
                for one, other in zip(latent.row_bytes(drafted, store, BLOCK, slot),
                                      latent.row_bytes(plain, store, BLOCK, slot)):
                    assert np.array_equal(one, other), (b, i)

        # and a token decoded over either is the same
        q = s.randn(s.B, 1, H, 512).bfloat16()
        one, other = (s.attend(cache, q, lens_t) for cache in (s.drafting, s.plain))
        assert torch.equal(one.view(torch.int16), other.view(torch.int16))
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("store", STORES)
def test_two_graphs_that_share_a_workspace(store):
    """A graph for drafted trees and one for single tokens, replayed in turn on one stream."""
    s = Server(store, [300, 20, 77], 5, 6, seed=9)
    trees = words_tensor([random_tree(s.rng, 5) for _ in range(s.B)])
    kv = s.randn(s.B * 5, 512).bfloat16()
    s.insert(s.drafting, None, kv, [(b, s.lens[b] + j) for b in range(s.B) for j in range(5)],
             [s.lens[b] for b in range(s.B) for _ in range(5)])
    lens = dev([n + 5 for n in s.lens], np.int32)
    work = torch.empty(k.latent_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)
    wide, one = s.randn(s.B, 5, 6, 512).bfloat16(), s.randn(s.B, 1, 6, 512).bfloat16()
    calls = []
    for q, tree in ((wide, trees), (one, None)):
        out = torch.zeros_like(q)

        def call(q=q, tree=tree, out=out):
            k.latent_attention(STORES[store], q, s.drafting, s.nb, BLOCK, s.table, lens, SCALE, out, tree=tree,
                               workspace=work)
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        calls.append((graph, out, q, tree))
    for turn in range(3):
        for graph, out, q, tree in calls:
            q.copy_(s.randn(*q.shape))
            graph.replay()
        for graph, out, q, tree in calls:
            assert torch.equal(out.view(torch.int16), s.attend(s.drafting, q, lens, tree).view(torch.int16))


def test_example_runs():
    from examples import tree_decode
    lens, x = tree_decode.main(steps=12, batch=3, heads=16, seed=0)
    assert all(n >= 12 for n in lens) and bool(torch.isfinite(x).all())


def test_arguments_on_the_host_are_refused():
    """Before anything is launched, and naming the one that is not on the device."""
    q = torch.zeros(2, 1, 3, 512, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(k.fp8_cache_bytes(4, 16), dtype=torch.uint8, device=DEV)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)

    def attend(**kw):
        a = dict(q=q, cache=cache, table=table, lens=lens, out=torch.empty_like(q)) | kw
        k.latent_attention(k.STORE_FP8, a["q"], a["cache"], 4, 16, a["table"], a["lens"], 1.0, a["out"],
                           lse=kw.get("lse"), tree=kw.get("tree"))

    attend()
    for name, t in dict(cache=cache, table=table, lens=lens, out=q, lse=torch.zeros(2, 1, 3),
                        tree=torch.ones(2, 1, dtype=torch.int64)).items():
        with pytest.raises(ValueError, match=dict(cache="kv_cache", table="block_table", lens="seq_lens").get(name, name)):
            attend(**{name: t.cpu()})
    with pytest.raises(ValueError, match="host"):
        attend(q=q.cpu())
    path = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    for at in range(3):
        moved = [t.cpu() if i == at else t for i, t in enumerate((table, lens, path))]
        with pytest.raises(ValueError, match="CUDA|host"):
            k.tree_keep(k.STORE_FP8, cache, 4, 16, moved[0], moved[1], moved[2], lens, lens)
    x, positions = torch.zeros(3, 2, 8, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    cos_sin = torch.zeros(4, 8, device=DEV)
    for call in (lambda: k.rope_rows(x, positions.cpu(), cos_sin), lambda: k.rope_rows(x, positions, cos_sin.cpu()),
                 lambda: k.rope_rows(x, positions, cos_sin, out=x.cpu()), lambda: k.rope_rows(x.cpu(), positions, cos_sin),
                 lambda: k.rope_table((1.0, 0.5), torch.zeros(3, 4, device=DEV), positions=positions.cpu())):
        with pytest.raises(ValueError, match="CUDA|host"):
            call()
    torch.cuda.synchronize()


def test_host_threads_on_streams_of_their_own():
    """Four threads that each run all of it, from the same inputs, against a serial run."""
    import threading

    servers = [Server("fp8" if i % 2 else "bf16", [70 + i, 9], 6, 5, seed=20 + i) for i in range(4)]
    words = words_tensor([random_tree(s.rng, 6) for s in servers for _ in range(2)]).view(4, 2, 6)
    queries = [s.randn(2, 6, 5, 512).bfloat16() for s in servers]
    rows = [s.randn(12, 512).bfloat16() for s in servers]
    images = [s.drafting.clone() for s in servers]

    def run(i):
        s = servers[i]
        cache = images[i].clone()
        at = [(b, s.lens[b] + j) for b in range(2) for j in range(6)]
        positions = [s.lens[b] + j for b in range(2) for j in range(6)]
        q = queries[i].clone()
        s.insert(cache, q.view(12, 5, 512), rows[i], at, positions)
        lens = dev([n + 6 for n in s.lens], np.int32)
        out = s.attend(cache, q, lens, words[i])
        k.rope_rows(out.view(12, 5, 512), dev(positions, np.int64), s.cos_sin, inverse=True)
        path, path_lens = dev(np.array([[1, 3, 5, -1, -1, -1]] * 2), np.int32), dev([3, 2], np.int32)
        k.tree_keep(STORES[s.store], cache, s.nb, BLOCK, s.table, lens, path, path_lens, lens)
        return out, cache, lens

    serial = [run(i) for i in range(4)]
    torch.cuda.synchronize()
    found = [[] for _ in range(4)]

    def worker(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                found[i].append(run(i))
        stream.synchronize()

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(4):
        assert len(found[i]) == 5
        for got in found[i]:
            for one, other in zip(got, serial[i]):
                assert torch.equal(one.view(torch.uint8), other.view(torch.uint8)), i


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("lens", [[333, 390], [333, 700]])
def test_a_chunk_of_a_prompt(store, lens):
    """Hundreds of new tokens of a request at once, as a prompt's chunk, in a window too.  (Rows past the
    400 positions of the table are not inserted: the tokens that see their slots get NaN.)"""
    s = Server(store, lens, 1, 1, seed=31)
    assert int(s.err.item()) == (k.DEVERR_POS_RANGE if max(lens) > POSITIONS else 0)
    Q, H = 150, 5
    lens = dev(s.lens, np.int32)
    q = s.randn(2, Q, H, 512).bfloat16()
    image, q64 = s.drafting.cpu().numpy(), q.double().cpu().numpy()
    for window in (0, 90):
        out = torch.empty_like(q)
        k.latent_attention(STORES[store], q, s.drafting, s.nb, BLOCK, s.table, lens, SCALE, out, window=window)
        out = out.double().cpu().numpy()
        for b, n in enumerate(s.lens):
            rows, ok = latent.rows_of(image, store, BLOCK, s.table_np[b], n, s.nb)
            want, _, size, reach = latent.attention(q64[b], rows, ok, n, SCALE, window)
            ds = SCALE * reach * 2.0 ** -15 + 2.0 ** -18
            near = np.abs(out[b] - want) <= np.abs(want) * 2.0 ** -8 + size * (2.0 ** -8 + 2 * ds[..., None])
            assert np.all(near | (np.isnan(want) & np.isnan(out[b])))
            assert np.array_equal(np.isnan(want), np.isnan(out[b])) and (n > POSITIONS or not np.isnan(want).any())
