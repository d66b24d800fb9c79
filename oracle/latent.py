"""Attention over the FP8 and bf16 caches, the move of an accepted path and the rotary
positions, in 64 bits (numpy) or more (integers, mpmath-free).

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the definitions in
``include/dsv4kv.h``, element by element, with nothing of the library's.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .fp4 import bf16_to_f64

# bytes of a slot: its data row, and its scale row behind the block's data rows
SLOT = {"fp8": (576, 8), "bf16": (1024, 0), "fp4": (352, 16), "indexer": (128, 4)}


def row_bytes(cache: np.ndarray, store: str, block_size: int, slot: int):
    """Views of a slot's data and scale bytes in a flat cache image."""
    data_bytes, scale_bytes = SLOT[store]
    b, o = divmod(int(slot), block_size)
    base = b * block_size * (data_bytes + scale_bytes)
    data = base + o * data_bytes
    scale = base + block_size * data_bytes + o * scale_bytes
    return cache[data:data + data_bytes], cache[scale:scale + scale_bytes]


def e4m3(code: int) -> float:
    e, m = code >> 3 & 15, code & 7
    if code & 127 == 127:
        return math.nan
    v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
    return -v if code & 128 else v


E4M3 = np.array([e4m3(c) for c in range(256)])


def unpack(data: np.ndarray, scale: np.ndarray, store: str) -> np.ndarray:
    """A slot's 512 values from its bytes."""
    if store == "bf16":
        return bf16_to_f64(data.view(np.uint16))
    v = np.zeros(512)
    for b in range(7):
        v[64 * b:64 * b + 64] = np.ldexp(E4M3[data[64 * b:64 * b + 64]], int(scale[b]) - 127)
    v[448:] = bf16_to_f64(data[448:].view(np.uint16))
    return v


def rows_of(cache, store, block_size, table, n, num_blocks=None):
    """[n, 512] values of a request's first n keys, and which of them have a valid block."""
    out, ok = np.zeros((n, 512)), np.ones(n, bool)
    for i in range(n):
        b = int(table[i // block_size])
        if b < 0 or (num_blocks is not None and b >= num_blocks):
            ok[i] = False
            continue
        out[i] = unpack(*row_bytes(cache, store, block_size, b * block_size + i % block_size), store)
    return out, ok


def visible(n, q_len, j, window, tree=None):
    """The keys that token j of a request of n keys sees; tree: its tokens' words, or None."""
    c = n - q_len
    if tree is None:
        to = c + 1 + j
        return [i for i in range(max(0, to - window if window else 0), max(to, 0))]
    word = int(tree[j]) & (1 << q_len) - 1
    if word == 0:
        return []
    since = max(0, c + bin(word).count("1") - window) if window else 0
    return list(range(since, max(c, 0))) + [c + i for i in range(q_len) if word >> i & 1 and c + i >= 0]


def attention(q, rows, ok, n, scale, window=0, sinks=None, tree=None):
    """One request: q float64 [Q, H, 512], rows [n, 512].  Returns (out, lse, |p| . |rows|,
    the largest sum |q||k|): the last two are what error bounds go by."""
    Q, H, _ = q.shape
    out, size = np.zeros((Q, H, 512)), np.zeros((Q, H, 512))
    lse, reach = np.full((Q, H), -np.inf), np.zeros((Q, H))
    for j in range(Q):
        seen = np.array([i for i in visible(n, Q, j, window, tree) if ok[i]], int)
        s = scale * (q[j] @ rows[seen].T)
        if sinks is not None:
            s = np.concatenate([s, sinks[:, None]], 1)
        if s.shape[1] == 0:
            continue
        if seen.size:
            reach[j] = (np.abs(q[j]) @ np.abs(rows[seen]).T).max(1)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        total = p.sum(1, keepdims=True)
        lse[j] = (m + np.log(total))[:, 0]
        p = (p / total)[:, :seen.size]
        out[j] = p @ rows[seen]
        size[j] = p @ np.abs(rows[seen])
    return out, lse, size, reach


def keep(cache, store, block_size, table, n, q_len, path, path_len, num_blocks):
    """One request, on the image itself: (the new length, whether something was flagged)."""
    if n <= 0:
        return 0, False
    if n < q_len:
        return n, True
    c, kept, last, moves, flagged = n - q_len, 0, -1, [], False
    for i in range(max(0, path_len)):
        if i >= q_len or path[i] <= last or path[i] >= q_len:
            break
        last = int(path[i])
        kept += 1
        if last != i:
            moves.append((c + last, c + i))
    flagged = kept != path_len
    read = []
    for src, dst in moves:
        a, b = int(table[src // block_size]), int(table[dst // block_size])
        if not (0 <= a < num_blocks and 0 <= b < num_blocks):
            flagged = True
            continue
        data, scale = row_bytes(cache, store, block_size, a * block_size + src % block_size)
        read.append((b * block_size + dst % block_size, data.copy(), scale.copy()))
    for slot, data, scale in read:
        to_data, to_scale = row_bytes(cache, store, block_size, slot)
        to_data[:], to_scale[:] = data, scale
    return c + kept, flagged


# 2 pi to 200 bits, by Machin's formula for pi in integers
def _pi(bits: int) -> int:
    def arctan_inverse(x):
        total, term, k = 0, (1 << bits + 20) // x, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= x * x
            k += 1
        return total
    return 4 * (4 * arctan_inverse(5) - arctan_inverse(239)) >> 20


_PI = _pi(220)


def angle(position: int, frequency: float) -> float:
    """position * frequency modulo 2 pi in (-pi, pi], the product and the remainder exact."""
    x = (Fraction(position) * Fraction(frequency))
    fixed = (x.numerator << 220) // x.denominator
    fixed %= 2 * _PI
    if fixed > _PI:
        fixed -= 2 * _PI
    return float(Fraction(fixed, 1 << 220))


def table_row(position: int, frequencies, magnitude: float) -> np.ndarray:
    a = [angle(position, f) for f in frequencies]
    return magnitude * np.array([math.cos(x) for x in a] + [math.sin(x) for x in a])


def rotate(x: np.ndarray, cos_sin: np.ndarray, offset: int, half: bool, inverse: bool) -> np.ndarray:
    """Rows [..., width] turned by cos_sin [..., d]."""
    d = cos_sin.shape[-1]
    z = cos_sin[..., :d // 2] + 1j * cos_sin[..., d // 2:]
    if inverse:
        z = z.conj()
    i = np.arange(d // 2)
    first, second = (offset + i, offset + d // 2 + i) if half else (offset + 2 * i, offset + 2 * i + 1)
    turned = (x[..., first] + 1j * x[..., second]) * z
    out = x.copy()
    out[..., first], out[..., second] = turned.real, turned.imag
    return out
