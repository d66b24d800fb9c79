"""The 4-bit cache's operators on the GPU against their 64-bit definitions (oracle/fp4.py).

Bounds, fixed from the arithmetic:
 * codes and exponents follow the exact values, so they are compared without one; rope
   dims and q are one bf16 rounding (half a step, 2^-8 of the value) after fp32 arithmetic
   good to 2^-18;
 * an fp32 score of 512 terms is off by at most scale * sum|q||k| * 2^-15 (512 roundings of
   2^-24 each); probabilities are rounded to bf16 (2^-8) before the product with the rows,
   and the output once more;
 * the reader, the eviction and every integer are exact.
"""
import numpy as np
import pytest

from oracle import fp4

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kv_norm_rope_gb300 as k  # noqa: E402

DEV = torch.device("cuda:0")
EPS = 1e-6


def bf16(x):
    """float array -> (bf16 tensor on the GPU, the float64 values it holds)"""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


def dev(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x, dtype)).to(DEV)


def as_bf16(x):
    """float64 values as bf16 holds them: past its largest is infinity"""
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def error_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- insert and reader

def cos_sin_table(n):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def check_insert(kv, w, H=0, eps=EPS, block=7, seed=0, slots=None, positions=None, max_pos=50):
    rng = np.random.default_rng(seed)
    T = kv.shape[0]
    nb = -(-2 * max(T, 1) // block)
    if slots is None:
        slots = rng.permutation(nb * block)[:T]
        slots[rng.random(T) < 0.1] = -1
    positions = rng.integers(0, max_pos, T) if positions is None else positions
    table = cos_sin_table(max_pos)
    kv_t, kv64 = bf16(kv)
    w_t, w64 = bf16(w)
    q_t, q64 = bf16(rng.standard_normal((T, H, 512))) if H else (None, None)
    poison = rng.integers(0, 256, nb * block * 368).astype(np.uint8)
    cache, err = dev(poison), error_word()
    k.qnorm_rope_kv_fp4_insert(q_t, kv_t, w_t, dev(positions, np.int64), dev(table), dev(slots, np.int64),
                               cache, nb, block, eps, device_error=err)
    torch.cuda.synchronize()
    got = cache.cpu().numpy()
    untouched = np.ones(got.size, bool)
    flags = 0
    for t in range(T):
        if not 0 <= positions[t] < max_pos:
            flags |= k.DEVERR_POS_RANGE
            if H:
                assert np.array_equal(q_t[t].double().cpu().numpy(), q64[t])
            continue
        cs = table[positions[t]]
        for h in range(H):
            want = fp4.norm_rope(q64[t, h], None, cs, eps)
            off = np.abs(q_t[t, h].double().cpu().numpy() - want)
            assert np.all(off <= np.abs(want) * (2.0 ** -8 + 2.0 ** -18) + 1e-30)
        if slots[t] >= nb * block:
            flags |= k.DEVERR_SLOT_RANGE
        if not 0 <= slots[t] < nb * block:
            continue
        v = fp4.norm_rope(kv64[t], w64, cs, eps)
        held, exps, codes = fp4.quantise(v)
        data, scale = fp4.row_bytes(got, block, slots[t])
        for part in fp4.row_bytes(untouched, block, slots[t]):
            part[:] = False
        assert np.array_equal(scale[:14], (exps + 127).astype(np.uint8)) and not scale[14:].any()
        assert np.array_equal(fp4.unpack(data, scale)[:448], held, equal_nan=True)
        tail = fp4.bf16_to_f64(data[224:].view(np.uint16))
        want = v[448:]
        # the pair's rotation in fp32: bounded by the pair's size
        size = np.abs(want) * (2.0 ** -8 + 2.0 ** -18) + 1e-30
        assert np.all((np.abs(tail - want) <= size) | (np.isnan(tail) & np.isnan(want)))
    assert np.array_equal(got[untouched], poison[untouched])
    assert int(err.item()) == flags
    # the reader, against the bytes
    ask = np.concatenate([np.asarray(slots, np.int64), [-3, nb * block, 0]])
    out, err = torch.full((ask.size, 512), 7.0, dtype=torch.bfloat16, device=DEV), error_word()
    k.fp4_dequant_gather(cache, nb, block, dev(ask), out, device_error=err)
    out = out.double().cpu().numpy()
    for t, s in enumerate(ask):
        want = np.zeros(512) if not 0 <= s < nb * block else fp4.unpack(*fp4.row_bytes(got, block, s))
        assert np.array_equal(out[t], as_bf16(want), equal_nan=True)
    assert int(err.item()) == k.DEVERR_SLOT_RANGE


@pytest.mark.parametrize("T,H,block", [(1, 0, 1), (1, 3, 16), (2, 1, 5), (3, 64, 64), (5, 0, 64), (37, 2, 27),
                                       (200, 0, 64), (130, 7, 3)])
def test_insert_and_gather(T, H, block):
    rng = np.random.default_rng(T * 100 + H)
    kv = rng.standard_normal((T, 512)) * np.where(rng.random((T, 512)) < 0.01, 30, 1)
    check_insert(kv, 1 + 0.1 * rng.standard_normal(512), H, block=block, seed=T)


def test_insert_every_row_count_layout():
    """Past one wave of warps, so that the persistent layout runs (KV rows alone and with q)."""
    rng = np.random.default_rng(3)
    for T, H in ((4000, 0), (900, 6)):
        T0 = T
        kv = np.tile(rng.standard_normal((100, 512)), (-(-T0 // 100), 1))[:T0]
        w = 1 + 0.1 * rng.standard_normal(512)
        kv_t, kv64 = bf16(kv)
        w_t, w64 = bf16(w)
        q, q64 = bf16(rng.standard_normal((T0, H, 512))) if H else (None, None)
        block, nb = 64, -(-T0 // 64)
        cache = torch.zeros(k.fp4_cache_bytes(nb, block), dtype=torch.uint8, device=DEV)
        pos = np.tile(np.arange(50), -(-T0 // 50))[:T0]
        k.qnorm_rope_kv_fp4_insert(q, kv_t, w_t, dev(pos, np.int64), dev(cos_sin_table(50)),
                                   dev(np.arange(T0), np.int64), cache, nb, block, EPS)
        got = cache.cpu().numpy()
        # rows repeat every 100 tokens, and so do their bytes
        first = [b"".join(x.tobytes() for x in fp4.row_bytes(got, block, t)) for t in range(100)]
        for t in range(T0):
            assert b"".join(x.tobytes() for x in fp4.row_bytes(got, block, t)) == first[t % 100]
        for t in range(0, 100, 9):
            held, _, _ = fp4.quantise(fp4.norm_rope(kv64[t], w64, cos_sin_table(50)[pos[t]], EPS))
            assert np.array_equal(fp4.unpack(*fp4.row_bytes(got, block, t))[:448], held)
        if H:
            out = q.double().cpu().numpy()
            for t in range(0, T0, 97):
                for h in range(H):
                    want = fp4.norm_rope(q64[t, h], None, cos_sin_table(50)[pos[t]], EPS)
                    assert np.all(np.abs(out[t, h] - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -18) + 1e-30)


def test_insert_at_borders():
    """Rows whose values fall exactly on borders between codes and between exponents (the
    mean square is exactly 1 and eps 0), and a hair beside them."""
    rows = []
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for scale in (1.0, 0.5, 2.0):
        x = np.zeros(512)
        x[:448] = np.tile(ties, 56) * scale * rng_signs(448)
        # fill up to a sum of squares of 512 * 4^j with the rope dims
        rows.append(x)
    out = []
    for x in rows:
        total = (x * x).sum()
        want = 512.0 * 4.0 ** np.ceil(np.log2(total / 512) / 2 + 1e-9)
        rest = want - total
        y = x.copy()
        for i in range(448, 512):  # greedy squares of bf16 values
            v = np.floor(np.sqrt(rest) * 16) / 16
            v = float(np.float32(v))
            t = torch.tensor(v).to(torch.bfloat16).double().item()
            if t * t > rest:
                t = np.nextafter(t, 0)
                t = torch.tensor(t * 0.99).to(torch.bfloat16).double().item()
            y[i], rest = t, rest - t * t
        out.append(y)
    base = np.array(out)
    near = np.repeat(base, 3, 0)
    near[1::3, 448] *= 1.01
    near[2::3, 448] *= 0.99
    check_insert(near, np.ones(512), eps=0.0, slots=np.arange(9), positions=np.zeros(9, np.int64))
    # constant rows: r = 1 / |c| exactly, every value 1
    const = np.ones((4, 512)) * np.array([1.0, 0.5, 2.0 ** -30, 2.0 ** 20])[:, None]
    for wv in (1.0, 1.25, 2.5, 0.75, 3.0, 6.0):
        check_insert(const, np.full(512, wv), eps=0.0, slots=np.arange(4))


def rng_signs(n):
    return np.where(np.random.default_rng(1).random(n) < 0.5, -1.0, 1.0)


def test_insert_extremes():
    rng = np.random.default_rng(8)
    kv = rng.standard_normal((8, 512))
    kv[0] *= 2.0 ** -70          # squares are subnormal
    kv[1] *= 2.0 ** -100
    kv[2, :] = 0.0
    kv[2, 5] = 1.0               # one element makes the row
    kv[3] *= 2.0 ** 50
    kv[4, 32:64] *= 2.0 ** -90   # a group far below its row
    kv[5, :448] = 0.0
    check_insert(kv, np.ones(512), eps=0.0, slots=np.arange(8))
    w = np.where(rng.random(512) < 0.3, 0.0, rng.standard_normal(512) * 8)
    w = np.where(np.abs(w) < 2.0 ** -9, 0.0, w)
    check_insert(kv, w, eps=1e-6, slots=np.arange(8))


def test_insert_zero_row_without_eps_reads_nan():
    kv = np.zeros((1, 512))
    check_insert(kv, np.ones(512), eps=0.0, slots=np.arange(1))


def test_insert_flags():
    rng = np.random.default_rng(9)
    slots = np.array([0, 1000, -1, 3, 4, 10 ** 12])
    check_insert(rng.standard_normal((6, 512)), np.ones(512), H=2, slots=slots,
                 positions=np.array([0, 1, 2, 50, -1, 3]))


def test_gather_every_code_and_scale():
    """Random bytes: each of the 256 scale bytes, over all codes."""
    rng = np.random.default_rng(10)
    nb, block = 20, 3
    raw = rng.integers(0, 256, nb * block * 368).astype(np.uint8)
    for s in range(60):
        data, scale = fp4.row_bytes(raw, block, s)
        scale[:14] = np.arange(14 * s, 14 * s + 14) % 256
        data[224:].view(np.uint16)[:] &= 0x7F7F  # finite rope dims
    out = torch.empty(60, 512, dtype=torch.bfloat16, device=DEV)
    k.fp4_dequant_gather(dev(raw), nb, block, dev(np.arange(60)), out)
    got = out.double().cpu().numpy()
    for s in range(60):
        want = fp4.unpack(*fp4.row_bytes(raw, block, s))
        assert np.array_equal(got[s], as_bf16(want), equal_nan=True)


# ---------------------------------------------------------------- attention

class Batch:
    """Random requests over a shuffled cache whose unused slots hold 0xff (NaN rope dims)."""

    def __init__(self, lens, Q, H, block, seed=0, spare=2, gain=1.0, stride=0):
        rng = np.random.default_rng(seed)
        self.lens, self.Q, self.H, self.block = list(lens), Q, H, block
        B = len(lens)
        self.W = max(1, -(-max(lens) // block))
        pages = [-(-n // block) for n in lens]
        self.nb = sum(pages) + spare
        order = rng.permutation(self.nb)
        table = np.full((B, self.W + stride), -1, np.int32)
        cache = np.full(self.nb * block * 368, 255, np.uint8)
        at = 0
        self.rows, self.ok = [], []
        for b, n in enumerate(lens):
            table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
            for i in range(n):
                data, scale = fp4.row_bytes(cache, block, table[b, i // block] * block + i % block)
                data[:224] = rng.integers(0, 256, 224)
                scale[:14], scale[14:] = rng.integers(124, 128, 14), 0
                tail = torch.from_numpy(rng.standard_normal(64).astype(np.float32) * 2).to(torch.bfloat16)
                data[224:] = tail.view(torch.int16).numpy().view(np.uint8)
        self.table_np, self.cache_np = table, cache
        for b, n in enumerate(lens):
            rows, ok = fp4.rows_of(cache, block, table[b], n)
            self.rows.append(rows)
            self.ok.append(ok)
        self.q, self.q64 = bf16(rng.standard_normal((B, Q, H, 512)) * gain)
        self.scale = 512.0 ** -0.5
        self.table = dev(table)[:, :self.W]
        self.cache = dev(cache)
        self.lens_t = dev(lens, np.int32)

    def attention(self, window=0, sinks=None, lse=True, stream=None, err=None, out=None):
        B = len(self.lens)
        out = torch.full((B, self.Q, self.H, 512), 9.0, dtype=torch.bfloat16, device=DEV) if out is None else out
        lse = torch.full((B, self.Q, self.H), 9.0, device=DEV) if lse else None
        k.fp4_attention(self.q, self.cache, self.nb, self.block, self.table, self.lens_t, self.scale, out,
                        lse=lse, sinks=sinks, window=window, stream=stream, device_error=err)
        return out, lse

    def check(self, out, lse, window=0, sinks=None, lens=None):
        out = out.double().cpu().numpy()
        sinks64 = None if sinks is None else sinks.double().cpu().numpy()
        for b, n in enumerate(lens or self.lens):
            want, wlse, size, reach = fp4.attention(self.q64[b], self.rows[b][:n], self.ok[b][:n], n, self.scale,
                                                    window, sinks64)
            ds = self.scale * reach * 2.0 ** -15 + 2.0 ** -18
            tol = np.abs(want) * 2.0 ** -8 + size * (2.0 ** -8 + 2 * ds[..., None])
            assert np.all(np.abs(out[b] - want) <= tol + 1e-30), (b, np.max(np.abs(out[b] - want) - tol))
            if lse is not None:
                got = lse[b].double().cpu().numpy()
                empty = np.isneginf(wlse)
                assert np.array_equal(np.isneginf(got), empty)
                off = np.abs(got[~empty] - wlse[~empty])
                assert np.all(off <= ds[~empty] + np.abs(wlse[~empty]) * 2.0 ** -22)


CASES = [
    # lens, Q, H, block
    ([1], 1, 1, 16),
    ([5, 0, 2], 1, 8, 1),
    ([127, 128, 129], 1, 16, 64),
    ([255, 256, 257, 1], 1, 3, 27),
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


@pytest.mark.parametrize("lens,Q,H,block", CASES)
def test_attention(lens, Q, H, block):
    s = Batch(lens, Q, H, block, seed=len(lens) + Q + H)
    err = error_word()
    out, lse = s.attention(err=err)
    s.check(out, lse)
    assert int(err.item()) == 0


@pytest.mark.parametrize("lens,Q,H,block", [CASES[1], CASES[3], CASES[8], CASES[9], CASES[10], CASES[12]])
@pytest.mark.parametrize("window", [1, 3, 100, 128, 5000])
def test_attention_window(lens, Q, H, block, window):
    s = Batch(lens, Q, H, block, seed=window)
    out, lse = s.attention(window=window)
    s.check(out, lse, window)


@pytest.mark.parametrize("lens,Q,H,block", [CASES[1], CASES[8], CASES[14], CASES[6]])
def test_attention_sinks(lens, Q, H, block):
    s = Batch(lens, Q, H, block, seed=4)
    sinks = torch.linspace(-8, 8, H, device=DEV)
    out, lse = s.attention(sinks=sinks, window=50)
    s.check(out, lse, 50, sinks)
    sinks = torch.full((H,), -float("inf"), device=DEV)  # a sink that takes nothing
    plain, _ = s.attention()
    out, lse = s.attention(sinks=sinks)
    s.check(out, lse)
    # a sink far above every score leaves nothing for the keys
    sinks = torch.full((H,), 300.0, device=DEV)
    out, lse = s.attention(sinks=sinks)
    s.check(out, lse, 0, sinks)


@pytest.mark.parametrize("order", ["rising", "falling", "spike"])
def test_attention_scores_far_apart(order):
    """Scores from -400 to 400 along the keys: the running maximum moves in every tile, or the
    first tile's is never reached again, or one key takes everything."""
    n, H = 1100, 4
    s = Batch([n], 1, H, 16, seed=11)
    rng = np.random.default_rng(12)
    way = rng.integers(0, 2, 64) * 2 - 1.0
    level = {"rising": np.linspace(-1, 1, n), "falling": np.linspace(1, -1, n),
             "spike": np.where(np.arange(n) == 700, 1.0, -1.0)}[order]
    cache = s.cache_np
    for i in range(n):
        data, scale = fp4.row_bytes(cache, 16, s.table_np[0, i // 16] * 16 + i % 16)
        scale[:14] = 120
        tail = torch.from_numpy((way * level[i] * 12).astype(np.float32)).to(torch.bfloat16)
        data[224:] = tail.view(torch.int16).numpy().view(np.uint8)
    s.cache = dev(cache)
    s.rows[0], s.ok[0] = fp4.rows_of(cache, 16, s.table_np[0], n)
    q = s.q64.copy()
    q[..., 448:] = way * 12 * np.linspace(0.5, 1, H)[None, None, :, None]
    s.q, s.q64 = bf16(q)
    out, lse = s.attention()
    s.check(out, lse)


def _ragged(count, seed):
    rng = np.random.default_rng(seed)
    lens = np.where(rng.random(count) < 0.2, 0, rng.integers(1, 60, count))
    lens[rng.choice(count, 5, replace=False)] = rng.integers(200, 900, 5)
    return [int(n) for n in lens]


@pytest.mark.parametrize("count,Q,H", [(25, 1, 70), (160, 2, 3), (511, 1, 2), (513, 1, 2), (300, 1, 130)])
def test_many_short_requests_among_longer_ones(count, Q, H):
    """Runs of several requests, some of them idle, and requests over several runs."""
    lens = _ragged(count, count)
    s = Batch(lens, Q, H, 16, seed=27)
    out, lse = s.attention()
    s.check(out, lse)
    again, _ = s.attention()
    assert torch.equal(out, again)


@pytest.mark.parametrize("count,Q,H", [(25, 1, 70), (160, 2, 3), (513, 1, 2)])
def test_weights_of_many_short_requests(count, Q, H):
    check_weights(Batch(_ragged(count, count), Q, H, 16, seed=28))


def test_attention_values_of_the_lowest_kind():
    """Scores that overflow to -infinity are masked; a row of them alone has no value."""
    s = Batch([30, 200], 1, 2, 16, seed=13)
    q = s.q64.copy()
    q[0] = 0.0
    s.q, s.q64 = bf16(q)
    out, lse = s.attention()
    s.check(out, lse)
    # a NaN in q stays in its own row
    q[0, 0, 1, 3] = np.nan
    s.q, _ = bf16(q)
    out, lse = s.attention()
    assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(lse[0, 0, 1])
    assert torch.isfinite(out[0, 0, 0]).all() and torch.isfinite(out[1]).all()


def test_attention_scores_far_below_zero():
    """Every score of a row hugely negative: the softmax is of their differences alone."""
    s = Batch([300], 1, 4, 16, seed=25)
    q = s.q64.copy()
    q[...] = 0.0
    cache = s.cache_np
    for i in range(300):
        data, _ = fp4.row_bytes(cache, 16, s.table_np[0, i // 16] * 16 + i % 16)
        data[224:226] = torch.tensor([1.0]).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint8)
    s.cache = dev(cache)
    s.rows[0], s.ok[0] = fp4.rows_of(cache, 16, s.table_np[0], 300)
    q[..., 448] = -np.exp2(np.array([10.0, 40.0, 80.0, 110.0]))  # the same score for every key
    s.q, s.q64 = bf16(q)
    out, lse = s.attention()
    got = out.double().cpu().numpy()[0, 0]
    want = s.rows[0].mean(0)
    size = np.abs(s.rows[0]).mean(0)
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + size * 2.0 ** -7)
    assert np.allclose(lse[0, 0].double().cpu().numpy(), s.scale * q[0, 0, :, 448] + np.log(300), rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("kind", ["group", "large", "rope nan", "rope inf", "rope -inf"])
@pytest.mark.parametrize("n,Q,H,window", [(300, 3, 4, 0), (258, 3, 40, 0), (300, 3, 4, 100), (500, 3, 64, 200)])
def test_attention_rows_not_finite(kind, n, Q, H, window):
    """A row that is not finite makes NaN of the tokens that see it and of no others."""
    bad = [n - 1] if window == 0 else [n - Q + 1 - window]  # seen by the last token alone, or the first
    s = Batch([n, 40], Q, H, 16, seed=26)
    cache = s.cache_np
    for i in bad:
        data, scale = fp4.row_bytes(cache, 16, s.table_np[0, i // 16] * 16 + i % 16)
        if kind == "group":
            scale[9], data[9 * 16:10 * 16] = 255, 0
        elif kind == "large":
            scale[13] = 230
        else:
            value = {"rope nan": np.nan, "rope inf": np.inf, "rope -inf": -np.inf}[kind]
            tail = torch.tensor([value]).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint8)
            data[224 + 2 * 45:226 + 2 * 45] = tail
    s.cache = dev(cache)
    out, lse = s.attention(window=window)
    hit = Q - 1 if window == 0 else 0
    assert torch.isnan(out[0, hit]).all() and torch.isnan(lse[0, hit]).all()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, length in enumerate(s.lens):
        rows = s.rows[b].copy()
        want, wlse, size, reach = fp4.attention(s.q64[b], rows, s.ok[b], length, s.scale, window)
        ds = s.scale * reach * 2.0 ** -15 + 2.0 ** -18
        for j in range(Q):
            if b == 0 and j == hit:
                continue
            tol = np.abs(want[j]) * 2.0 ** -8 + size[j] * (2.0 ** -8 + 2 * ds[j][:, None])
            assert np.all(np.abs(out[b, j] - want[j]) <= tol + 1e-30)
            assert np.all(np.abs(lse[b, j] - wlse[j]) <= ds[j] + np.abs(wlse[j]) * 2.0 ** -22)


def test_attention_bad_pages_and_lengths():
    """A block outside the cache takes no part and is flagged; so is a length past the table."""
    s = Batch([300, 100, 50], 1, 8, 16, seed=14)
    table = s.table_np.copy()
    table[0, 3] = s.nb
    table[0, 18] = -7          # the last, partly filled block of request 0
    table[1, :] = 2 ** 31 - 1  # no valid block at all
    s.table = dev(table)
    for b in range(2):
        s.rows[b], s.ok[b] = fp4.rows_of(s.cache_np, 16, table[b], s.lens[b], s.nb)
    err = error_word()
    out, lse = s.attention(err=err)
    s.check(out, lse)
    assert int(err.item()) == k.DEVERR_SLOT_RANGE
    s = Batch([300, 100, 50], 1, 8, 16, seed=15)
    s.lens_t = dev([19 * 16 + 5, 100, -4], np.int32)
    cache, table = s.cache_np, s.table_np
    for i in range(300, 304):  # the table's last slots hold finite rows
        data, scale = fp4.row_bytes(cache, 16, table[0, i // 16] * 16 + i % 16)
        data[:], scale[:] = 0, 0
    s.cache = dev(cache)
    s.rows[0], s.ok[0] = fp4.rows_of(cache, 16, table[0], 304)
    err = error_word()
    out, lse = s.attention(err=err)
    s.check(out, lse, lens=[304, 100, 0])
    assert int(err.item()) == k.DEVERR_SLOT_RANGE


def test_attention_strided_table_and_other_stream():
    s = Batch([90, 200], 2, 8, 16, seed=16, stride=5)
    assert not s.table.is_contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = s.attention(stream=side)
    side.synchronize()
    s.check(out, lse)
    ws = torch.empty(k.fp4_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)
    out2 = torch.empty_like(out)
    k.fp4_attention(s.q, s.cache, s.nb, s.block, s.table, s.lens_t, s.scale, out2, workspace=ws,
                    stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, out2)


def test_attention_in_a_graph_follows_new_lengths():
    """Captured once; replayed after the lengths and the table changed on the device."""
    s = Batch([700, 300], 1, 16, 16, seed=17)
    out = torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16, device=DEV)
    s.attention(out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, lse = s.attention(out=out)
    for lens in ([700, 300], [650, 0], [1, 299]):
        s.lens_t.copy_(dev(lens, np.int32))
        g.replay()
        torch.cuda.synchronize()
        s.check(out, lse, lens=lens)


def test_attention_same_bits_again():
    s = Batch([3000, 1, 777], 2, 40, 64, seed=18)
    first, lse = s.attention()
    for _ in range(3):
        out, lse2 = s.attention()
        assert torch.equal(out, first) and torch.equal(lse, lse2)


def test_attention_offsets_past_4_gib():
    """Pages at the far end of a cache of 4.6 GB."""
    block, nb = 64, 195000
    s = Batch([500], 1, 8, block, seed=19)
    cache = torch.zeros(nb * block * 368, dtype=torch.uint8, device=DEV)
    far = nb - s.nb
    cache[far * block * 368:] = s.cache
    s.cache, s.nb = cache, nb
    s.table = s.table + far
    out, lse = s.attention()
    s.check(out, lse)


# ---------------------------------------------------------------- weights

def check_weights(s, window=0, stride=3, lens=None):
    out, lse = s.attention(window=window)
    B, n = len(s.lens), max(max(s.lens), 1)
    start = np.random.default_rng(20).random((B, n + stride)).astype(np.float32)
    whole = dev(start)
    w, err = whole[:, :n], error_word()
    k.fp4_attention_weights(s.q, s.cache, s.nb, s.block, s.table, s.lens_t, s.scale, lse, w, window=window,
                            device_error=err)
    got = whole.double().cpu().numpy()
    lse64 = lse.double().cpu().numpy()
    for b, m in enumerate(s.lens):
        add = fp4.weights(s.q64[b], s.rows[b], s.ok[b], m, s.scale, lse64[b], window)
        reach = 0.0
        if m:
            reach = (np.abs(s.q64[b]).reshape(-1, 512) @ np.abs(s.rows[b]).T).max()
        want = start[b, :m].astype(np.float64) + add
        tol = add * (s.scale * reach * 2.0 ** -15 + 2.0 ** -18 + np.abs(lse64[b][np.isfinite(lse64[b])]).max(initial=0) * 2.0 ** -22)
        tol = tol + want * 2.0 ** -23 + add * s.Q * s.H * 2.0 ** -24
        assert np.all(np.abs(got[b, :m] - want) <= tol)
        assert np.array_equal(got[b, m:], start[b, m:].astype(np.float64))
    return err


@pytest.mark.parametrize("lens,Q,H,block", CASES)
def test_weights(lens, Q, H, block):
    assert int(check_weights(Batch(lens, Q, H, block, seed=21)).item()) == 0


@pytest.mark.parametrize("window", [1, 3, 100, 128])
def test_weights_window(window):
    for c in (CASES[1], CASES[8], CASES[10]):
        check_weights(Batch(*c, seed=22), window)


def test_weights_same_bits_and_bad_pages():
    s = Batch([2000, 3], 3, 50, 64, seed=23)
    _, lse = s.attention()
    runs = []
    for _ in range(3):
        w = torch.ones(2, 2000, device=DEV)
        k.fp4_attention_weights(s.q, s.cache, s.nb, s.block, s.table, s.lens_t, s.scale, lse, w)
        runs.append(w)
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])
    # a row too narrow for its request: what it has is served
    err, w = error_word(), torch.ones(2, 2100, device=DEV)
    k.fp4_attention_weights(s.q, s.cache, s.nb, s.block, s.table, s.lens_t, s.scale, lse, w[:, :1500],
                            device_error=err)
    assert int(err.item()) == k.DEVERR_SLOT_RANGE
    assert torch.equal(w[0, :1500], runs[0][0, :1500]) and bool((w[0, 1500:] == 1).all())
    s = Batch([300, 100], 1, 8, 16, seed=24)
    table = s.table_np.copy()
    table[0, 5] = -1
    s.table = dev(table)
    s.rows[0], s.ok[0] = fp4.rows_of(s.cache_np, 16, table[0], 300, s.nb)
    assert int(check_weights(s).item()) == k.DEVERR_SLOT_RANGE


# ---------------------------------------------------------------- eviction

def check_evict(lens, budget, recent, block=16, w=None, seed=0, alias=False, stride=0):
    rng = np.random.default_rng(seed)
    B = len(lens)
    W, W2 = max(1, -(-max(lens) // block)), -(-budget // block)
    nb = B * (W + W2) + 1
    order = rng.permutation(nb)
    table = order[:B * W].reshape(B, W).astype(np.int32)
    new = order[B * W:B * (W + W2)].reshape(B, W2).astype(np.int32)
    image = rng.integers(0, 256, nb * block * 368).astype(np.uint8)
    if w is None:
        w = np.round(rng.exponential(2.0, (B, max(max(lens), 1))), 1).astype(np.float32)
    padded = np.concatenate([w, np.full((B, stride), 7, np.float32)], 1)
    cache, err = dev(image), error_word()
    lens_t = dev(lens, np.int32)
    new_lens = lens_t if alias else torch.full((B,), -5, dtype=torch.int32, device=DEV)
    kept = torch.full((B, budget), -9, dtype=torch.int32, device=DEV)
    nw = torch.full((B, budget), 5.0, device=DEV)
    k.fp4_evict(cache, nb, block, dev(table), lens_t, dev(padded)[:, :w.shape[1]], budget, recent, dev(new),
                kept, new_lens, nw, device_error=err)
    got = cache.cpu().numpy()
    want = image.copy()
    for b, n in enumerate(lens):
        keep = fp4.evict(w[b], n, budget, recent)
        assert new_lens[b].item() == len(keep)
        assert kept[b].tolist() == keep + [-1] * (budget - len(keep))
        assert np.array_equal(nw[b].cpu().numpy(), np.concatenate([w[b][keep], np.zeros(budget - len(keep), np.float32)]),
                              equal_nan=True)
        for i, j in enumerate(keep):
            src = fp4.row_bytes(image, block, table[b, j // block] * block + j % block)
            dst = fp4.row_bytes(want, block, new[b, i // block] * block + i % block)
            for x, y in zip(src, dst):
                y[:] = x
    assert np.array_equal(got, want)
    assert int(err.item()) == 0


@pytest.mark.parametrize("lens,budget,recent,block", [
    ([1], 1, 0, 16), ([2], 1, 1, 1), ([40, 0, 7, 20], 20, 5, 7), ([5000, 1024, 1025, 3], 1024, 100, 64),
    ([3000], 1, 0, 64), ([3000], 2999, 2999, 27), ([3000, 10], 2999, 0, 64), ([700] * 30, 33, 8, 5),
    ([40000, 39999, 8192], 4097, 17, 64), ([100000], 8192, 1, 64)])
def test_evict(lens, budget, recent, block):
    check_evict(lens, budget, recent, block, seed=budget)


def test_evict_ties_and_odd_weights():
    rng = np.random.default_rng(30)
    n = 5000
    w = np.stack([
        np.zeros(n), np.full(n, 3.5), np.where(rng.random(n) < 0.5, -0.0, 0.0),
        np.where(rng.random(n) < 0.7, np.nan, 1.0), np.where(rng.random(n) < 0.01, np.inf, rng.integers(0, 3, n)),
        -rng.random(n), np.where(rng.random(n) < 0.5, -np.inf, np.nan), np.arange(n), np.arange(n)[::-1],
        rng.random(n) * 1e-42,
    ]).astype(np.float32)
    for budget, recent in ((100, 0), (1500, 33), (4999, 1)):
        check_evict([n] * 10, budget, recent, 16, w=w)


def test_evict_lens_in_place_strided_weights():
    check_evict([300, 50, 64], 64, 8, 16, seed=31, alias=True, stride=9)


def test_evict_bad_pages_and_lengths():
    block, nb = 16, 20
    image = np.random.default_rng(32).integers(0, 256, nb * block * 368).astype(np.uint8)
    cache, err = dev(image), error_word()
    table = dev(np.array([[0, 1, 99], [4, -1, 6]]), np.int32)
    new = dev(np.array([[10, -3], [12, 13]]), np.int32)
    kept = torch.empty(2, 30, dtype=torch.int32, device=DEV)
    lens, nl, nw = dev([60, 40], np.int32), torch.empty(2, dtype=torch.int32, device=DEV), torch.empty(2, 30, device=DEV)
    w = torch.arange(96, device=DEV, dtype=torch.float32).view(2, 48)
    k.fp4_evict(cache, nb, block, table, lens, w, 30, 30, new, kept, nl, nw, device_error=err)
    assert int(err.item()) == k.DEVERR_SLOT_RANGE
    assert kept[0].tolist() == list(range(18, 48)) and kept[1].tolist() == list(range(10, 40))
    got, want = cache.cpu().numpy(), image.copy()
    tn, nn = table.cpu().numpy(), new.cpu().numpy()
    for b in range(2):
        for i, j in enumerate(kept[b].tolist()):
            s, d = tn[b, j // block], nn[b, i // block]
            if 0 <= s < nb and 0 <= d < nb:
                for x, y in zip(fp4.row_bytes(image, block, s * block + j % block),
                                fp4.row_bytes(want, block, d * block + i % block)):
                    y[:] = x
    assert np.array_equal(got, want)


def test_all_in_a_graph():
    """Insert, attention, weights and eviction captured as one graph, against eager calls."""
    rng = np.random.default_rng(33)
    s = Batch([60, 200], 1, 8, 16, seed=34, spare=30)
    used = set(s.table_np[s.table_np >= 0].tolist())
    free = [p for p in range(s.nb) if p not in used]
    new = dev(np.array(free[:10]).reshape(2, 5), np.int32)
    kv, _ = bf16(rng.standard_normal((2, 512)))
    weight, _ = bf16(np.ones(512))
    cs, pos = dev(cos_sin_table(256)), dev([59, 199], np.int64)
    slots = dev([s.table_np[b, (n - 1) // 16] * 16 + (n - 1) % 16 for b, n in enumerate(s.lens)], np.int64)
    ws = torch.empty(k.fp4_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)

    def buffers():
        return dict(q=s.q.clone(), cache=s.cache.clone(), out=torch.zeros(2, 1, 8, 512, dtype=torch.bfloat16, device=DEV),
                    lse=torch.zeros(2, 1, 8, device=DEV), w=torch.ones(2, 200, device=DEV),
                    kept=torch.zeros(2, 70, dtype=torch.int32, device=DEV), nl=torch.zeros(2, dtype=torch.int32, device=DEV),
                    nw=torch.zeros(2, 70, device=DEV))

    def step(b):
        k.qnorm_rope_kv_fp4_insert(b["q"][:, 0], kv, weight, pos, cs, slots, b["cache"], s.nb, 16, EPS)
        k.fp4_attention(b["q"], b["cache"], s.nb, 16, s.table, s.lens_t, s.scale, b["out"], lse=b["lse"], workspace=ws)
        k.fp4_attention_weights(b["q"], b["cache"], s.nb, 16, s.table, s.lens_t, s.scale, b["lse"], b["w"])
        k.fp4_evict(b["cache"], s.nb, 16, s.table, s.lens_t, b["w"], 70, 10, new, b["kept"], b["nl"], b["nw"])

    eager, captured = buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        step(captured)
    g.replay()
    torch.cuda.synchronize()
    for name in eager:
        assert torch.equal(eager[name].view(torch.uint8), captured[name].view(torch.uint8)), name


# ---------------------------------------------------------------- together

def test_example_runs_and_keeps_the_attention_of_what_stays():
    """The example's decoding loop: every step gives each request `heads` of attention in all,
    and an eviction keeps the weights of the rows that stay."""
    from examples import fp4_cache_decode
    lens, weights, x = fp4_cache_decode.main(steps=96, batch=3, heads=16, limit=64, budget=40, recent=8)
    assert lens == [48, 48, 48]  # 64, cut to 40, up to 64, cut to 40, and 8 more
    assert torch.isfinite(x).all() and bool((weights[:, 48:] == 0).all())
    # 96 steps of 16 heads, less what left with the evicted rows
    assert bool((weights.sum(1) <= 96 * 16 * (1 + 1e-3)).all()) and bool((weights.sum(1) > 8 * 16).all())


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    """Seeded random sizes through attention, weights and eviction."""
    rng = np.random.default_rng(1000 + seed)
    H, Q = int(rng.integers(1, 140)), int(rng.choice([1, 1, 2, 5, 9]))
    B, block = int(rng.integers(1, 7)), int(rng.choice([1, 3, 16, 27, 64, 200]))
    lens = [int(x) for x in rng.integers(0, int(rng.choice([5, 140, 600])), B)]
    window = int(rng.choice([0, 0, 1, 40, 300]))
    s = Batch(lens, Q, H, block, seed=seed, stride=int(rng.integers(0, 3)), gain=float(rng.choice([0.1, 1, 4])))
    sinks = dev(rng.standard_normal(H) * 3, np.float32) if rng.random() < 0.5 else None
    out, lse = s.attention(window=window, sinks=sinks)
    s.check(out, lse, window, sinks)
    check_weights(s, window, stride=int(rng.integers(0, 5)))
    n = max(max(lens), 1)
    budget = int(rng.integers(1, n + 3))
    check_evict(lens, budget, int(rng.integers(0, budget + 1)), block, seed=seed, alias=bool(rng.random() < 0.5))
