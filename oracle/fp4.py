"""The operators of the 4-bit KV cache in 64 bits (numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the definitions in
``include/dsv4kv.h``, element by element, with nothing of the library's.
"""
from __future__ import annotations

import numpy as np

DATA_BYTES, SCALE_BYTES, SLOT_BYTES = 352, 16, 368
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
DIM_OF_NIBBLE = (0, 2, 4, 6, 1, 3, 5, 7)


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):  # signalling NaNs among the bits
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def exponent(amax: float) -> int:
    """The smallest s >= -127 with amax <= 6 * 2^s."""
    if amax == 0.0:
        return -127
    s = int(np.floor(np.log2(amax))) - 4
    while amax > np.ldexp(6.0, s):
        s += 1
    return max(s, -127)


def e2m1_rne(u: np.ndarray) -> np.ndarray:
    """Codes (without the sign bit) of the nearest magnitudes to |u|, ties to the even code."""
    d = np.abs(np.minimum(np.abs(u), 6.0)[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    hit = d == best  # one or two neighbours
    code = np.arange(8)
    even = np.where(hit & (code % 2 == 0), code, -1).max(-1)
    only = np.where(hit, code, -1).max(-1)
    return np.where(hit.sum(-1) == 2, even, only)


def quantise(v: np.ndarray):
    """[448] values -> (values as held, exponents [14], codes [448])."""
    held, codes, exps = np.zeros(448), np.zeros(448, np.int64), np.zeros(14, np.int64)
    for g in range(14):
        x = v[32 * g:32 * g + 32]
        if not np.all(np.isfinite(x)):
            exps[g] = 128
            held[32 * g:32 * g + 32] = np.nan
            continue
        s = exponent(np.abs(x).max())
        c = e2m1_rne(np.ldexp(x, -s))
        exps[g] = s
        codes[32 * g:32 * g + 32] = c + 8 * np.signbit(x)
        held[32 * g:32 * g + 32] = np.sign(x) * np.ldexp(MAGNITUDES[c], s)
    return held, exps, codes


def norm_rope(x: np.ndarray, w, cos_sin: np.ndarray, eps: float) -> np.ndarray:
    """One 512-wide row (float64) normalised, weighted (w may be None) and rotated."""
    with np.errstate(divide="ignore", invalid="ignore"):
        v = x * (1.0 / np.sqrt((x * x).sum() / 512.0 + np.float64(np.float32(eps))))
    if w is not None:
        v = v * w
    a, b = v[448::2].copy(), v[449::2].copy()
    c, s = cos_sin[:32].astype(np.float64), cos_sin[32:].astype(np.float64)
    v[448::2], v[449::2] = a * c - b * s, b * c + a * s
    return v


def row_bytes(cache: np.ndarray, block_size: int, slot: int):
    """Views of a slot's data and scale bytes in a flat cache image."""
    b, o = divmod(int(slot), block_size)
    base = b * block_size * SLOT_BYTES
    data = base + o * DATA_BYTES
    scale = base + block_size * DATA_BYTES + o * SCALE_BYTES
    return cache[data:data + DATA_BYTES], cache[scale:scale + SCALE_BYTES]


def pack(codes: np.ndarray) -> np.ndarray:
    """[448] codes -> 224 bytes."""
    out = np.zeros(224, np.uint8)
    for i in range(56):
        word = 0
        for n, d in enumerate(DIM_OF_NIBBLE):
            word |= int(codes[8 * i + d]) << (4 * n)
        out[4 * i:4 * i + 4] = np.frombuffer(word.to_bytes(4, "little"), np.uint8)
    return out


def unpack(data: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """A slot's 512 values from its bytes."""
    v = np.zeros(512)
    for i in range(56):
        word = int.from_bytes(data[4 * i:4 * i + 4].tobytes(), "little")
        for n, d in enumerate(DIM_OF_NIBBLE):
            c = (word >> (4 * n)) & 15
            e = int(scale[i // 4])
            m = MAGNITUDES[c & 7]
            if e == 255:
                v[8 * i + d] = np.nan if m == 0 else (-np.inf if c & 8 else np.inf)
            else:
                v[8 * i + d] = (-1.0 if c & 8 else 1.0) * np.ldexp(m, e - 127)
    v[448:] = bf16_to_f64(data[224:].view(np.uint16))
    return v


def rows_of(cache, block_size, table, n, num_blocks=None):
    """[n, 512] values of a request's first n keys, and which of them have a valid block."""
    out, ok = np.zeros((n, 512)), np.ones(n, bool)
    for i in range(n):
        b = int(table[i // block_size])
        if b < 0 or (num_blocks is not None and b >= num_blocks):
            ok[i] = False
            continue
        out[i] = unpack(*row_bytes(cache, block_size, b * block_size + i % block_size))
    return out, ok


def visible(n, q_len, j, window, i):
    to = n - q_len + 1 + j
    since = max(0, to - window) if window else 0
    return (i >= since) & (i < to)


def attention(q, rows, ok, n, scale, window=0, sinks=None):
    """One request: q float64 [Q, H, 512], rows [n, 512].  Returns (out, lse, |p| . |rows|,
    the largest sum |q||k|): the last two are what error bounds go by."""
    Q, H, _ = q.shape
    out, size = np.zeros((Q, H, 512)), np.zeros((Q, H, 512))
    lse = np.full((Q, H), -np.inf)
    reach = np.zeros((Q, H))
    i = np.arange(n)
    for j in range(Q):
        seen = np.flatnonzero(visible(n, Q, j, window, i) & ok)
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


def weights(q, rows, ok, n, scale, lse, window=0):
    """One request: what each of its n keys gets."""
    Q = q.shape[0]
    got = np.zeros(n)
    i = np.arange(n)
    for j in range(Q):
        seen = np.flatnonzero(visible(n, Q, j, window, i) & ok)
        for h in range(q.shape[1]):
            if lse[j, h] != -np.inf:
                got[seen] += np.exp(scale * (rows[seen] @ q[j, h]) - lse[j, h])
    return got


def evict(w, n, budget, recent):
    """One request: the indices it keeps."""
    if n <= budget:
        return list(range(n))
    w = [(-np.inf if np.isnan(x) else float(x) + 0.0) for x in w[:n - recent]]
    best = sorted(range(n - recent), key=lambda i: (-w[i], i))[:budget - recent]
    return sorted(best) + list(range(n - recent, n))
