"""Pins of the 64-bit definitions of the 4-bit cache (oracle/fp4.py), on the CPU."""
import numpy as np
import pytest

from oracle import fp4


def test_codes_at_and_beside_every_border():
    borders = [(0.25, 0, 1), (0.75, 1, 2), (1.25, 2, 3), (1.75, 3, 4), (2.5, 4, 5), (3.5, 5, 6), (5.0, 6, 7)]
    for b, below, above in borders:
        even = below if below % 2 == 0 else above
        got = fp4.e2m1_rne(np.array([np.nextafter(b, 0), b, np.nextafter(b, 9), -b]))
        assert list(got) == [below, even, above, even]
    assert list(fp4.e2m1_rne(np.array([0.0, 6.0, 7.9, -9.0]))) == [0, 7, 7, 7]


@pytest.mark.parametrize("k", range(-120, 121, 7))
def test_exponent_at_its_boundary(k):
    top = np.ldexp(6.0, k)
    assert fp4.exponent(top) == k
    assert fp4.exponent(np.nextafter(top, np.inf)) == k + 1
    assert fp4.exponent(np.nextafter(top, 0)) == k


def test_smallest_exponent():
    assert fp4.exponent(0.0) == -127
    assert fp4.exponent(2.0 ** -140) == -127


def test_a_word_written_by_hand():
    # dims 0..7 = 0.5, -1, 1.5, 2, -3, 4, 6, 0: codes 1 A 3 4 D 6 7 0; nibbles are dims 0 2 4 6 1 3 5 7
    codes = np.zeros(448, np.int64)
    codes[:8] = [0x1, 0xA, 0x3, 0x4, 0xD, 0x6, 0x7, 0x0]
    data = np.zeros(352, np.uint8)
    data[:224] = fp4.pack(codes)
    assert int.from_bytes(data[:4].tobytes(), "little") == 0x064A7D31
    scale = np.full(16, 127, np.uint8)
    scale[0] = 129
    assert list(fp4.unpack(data, scale)[:9]) == [2, -4, 6, 8, -12, 16, 24, 0, 0]


def test_quantise_round_trip_and_bound():
    rng = np.random.default_rng(5)
    v = rng.standard_normal(448) * np.exp(rng.standard_normal(448))
    held, exps, codes = fp4.quantise(v)
    step = np.ldexp(1.0, exps).repeat(32)
    assert np.all(np.abs(v) <= 6 * step)
    assert np.all(np.abs(held - v) <= step)  # half of the widest gap
    data = np.concatenate([fp4.pack(codes), np.zeros(128, np.uint8)])
    scale = np.concatenate([(exps + 127).astype(np.uint8), np.zeros(2, np.uint8)])
    assert np.array_equal(fp4.unpack(data, scale)[:448], held)
    again, exps2, codes2 = fp4.quantise(held)
    assert np.array_equal(again, held)


def test_attention_closed_forms():
    rng = np.random.default_rng(6)
    rows = rng.standard_normal((9, 512))
    ok = np.ones(9, bool)
    q = np.zeros((1, 2, 512))
    out, lse, _, _ = fp4.attention(q, rows, ok, 9, 0.1)
    assert np.allclose(out[0, 0], rows.mean(0)) and np.allclose(lse, np.log(9))
    # a sink as large as the nine scores' sum halves the output
    out, lse, _, _ = fp4.attention(q, rows, ok, 9, 0.1, sinks=np.log([9.0, 9.0]))
    assert np.allclose(out[0, 1], rows.mean(0) / 2) and np.allclose(lse, np.log(18))
    # a window of one sees the last key; with three tokens the first sees all but two
    q = rng.standard_normal((3, 1, 512))
    out, _, _, _ = fp4.attention(q, rows, ok, 9, 0.1, window=1)
    assert np.allclose(out[:, 0], rows[6:])
    out, lse, _, _ = fp4.attention(q[:, :, :] * 0, rows[:2], ok[:2], 2, 0.1)
    assert np.all(out[0] == 0) and lse[0, 0] == -np.inf and np.allclose(out[1, 0], rows[0])


def test_weights_sum_to_the_rows():
    rng = np.random.default_rng(7)
    rows, q = rng.standard_normal((20, 512)), rng.standard_normal((3, 4, 512))
    ok = np.ones(20, bool)
    _, lse, _, _ = fp4.attention(q, rows, ok, 20, 0.05)
    got = fp4.weights(q, rows, ok, 20, 0.05, lse)
    assert np.isclose(got.sum(), 12.0)
    assert got[19] < got.sum() / 3  # the last key is seen by one of three tokens


def test_evict_by_hand():
    w = np.array([5, 1, 5, np.nan, 2, 2, -0.0, 0.0, 9, 9], np.float32)
    assert fp4.evict(w, 10, 5, 2) == [0, 2, 4, 8, 9]  # the tie of 4 and 5 goes to 4
    assert fp4.evict(w, 10, 9, 1) == [0, 1, 2, 4, 5, 6, 7, 8, 9]
    assert fp4.evict(w, 10, 3, 3) == [7, 8, 9]
    assert fp4.evict(w, 4, 5, 2) == [0, 1, 2, 3]
