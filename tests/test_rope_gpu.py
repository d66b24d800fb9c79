"""The rotary table and the rotation of rows on the GPU against their definitions
(oracle/latent.py).

Bounds, fixed from the arithmetic:
 * table: the entry is one fp32 rounding of a sum of a pair of floats and a correction of at most
   0.025 * magnitude, off by a few roundings of 2^-24 each (4 * 0.025 * 2^-24 and 2^-33 turns of the
   angle: below 2^-27 of the magnitude).  The rounding is half a step of values up to the magnitude m:
   with 2^(e - 1) < m <= 2^e they are below 2^e, or 2^e itself, which is an fp32, so the step
   is 2^(e - 1) * 2^-23 and half of it 2^(e - 25);
 * rows: a product rounded once (2^-24), a fused multiply-add rounded once: 2^-23 of |a c| + |b s|,
   then half a step of the type (bf16 2^-8... relative 2^-9 of the next power, so 2^-8 covers it; fp16 2^-11).
"""
import math

import numpy as np
import pytest

from oracle import latent
from tests.test_latent_gpu import DEV, dev, error_word, k, torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp16": (torch.float16, 2.0 ** -11), "fp32": (torch.float32, 0.0)}


def check_table(out, positions, frequencies, magnitude=1.0, rows=None):
    got = out.double().cpu().numpy()
    for r in range(len(positions)) if rows is None else rows:
        want = latent.table_row(int(positions[r]), frequencies, magnitude)
        half_step = 2.0 ** (math.ceil(math.log2(abs(magnitude))) - 25)
        assert np.all(np.abs(got[r] - want) <= half_step + abs(magnitude) * 2.0 ** -27), (r, positions[r])


@pytest.mark.parametrize("dim", [2, 4, 6, 8, 30, 64, 128, 250, 256])
@pytest.mark.parametrize("n", [1, 2, 33, 500])
def test_table_of_a_range(dim, n):
    frequencies = k.rope_frequencies(dim)
    for first in (0, 1, 100003):
        out = torch.full((n + 1, dim), 9.0, device=DEV)
        k.rope_table(frequencies, out[:n], first=first)
        check_table(out, range(first, first + n), frequencies, rows=sorted({0, n // 2, n - 1}))
        assert bool((out[n] == 9).all())


@pytest.mark.parametrize("scaling,factor,magnitude", [(k.ROPE_LINEAR, 8.0, 1.0), (k.ROPE_NTK, 4.0, 0.7),
                                                      (k.ROPE_YARN, 40.0, 0.1 * math.log(40.0) + 1), (k.ROPE_PLAIN, 1.0, -2.5)])
def test_table_of_positions(scaling, factor, magnitude):
    frequencies = k.rope_frequencies(64, 10000.0, scaling, factor, 4096.0)
    rng = np.random.default_rng(1)
    positions = np.concatenate([rng.integers(0, 2 ** 32, 300), [0, 2 ** 32 - 1, 2 ** 31, 1], rng.integers(0, 2 ** 20, 200)])
    out = torch.empty(positions.size, 64, device=DEV)
    k.rope_table(frequencies, out, positions=dev(positions, np.int64), magnitude=magnitude)
    check_table(out, positions, frequencies, magnitude)


def test_table_at_every_arc_and_its_ends():
    """One pair whose angle is a chosen part of a turn: arcs' middles, borders and points."""
    turns = np.concatenate([np.arange(0, 256) / 256.0, np.arange(0, 256) / 256.0 + 2.0 ** -20,
                            np.arange(1, 257) / 256.0 - 2.0 ** -20])
    for i in range(0, turns.size, 128):
        part = list(2 * math.pi * turns[i:i + 128])
        out = torch.empty(4, 256, device=DEV)
        k.rope_table(part, out)
        check_table(out, range(4), part)
        assert bool((out[0, :128] == 1).all()) and bool((out[0, 128:] == 0).all())


def test_table_misaligned_and_strangely_sized():
    room = torch.full((1 + 37 * 64 + 5,), 9.0, device=DEV)
    out = room[1:1 + 37 * 64].view(37, 64)
    frequencies = k.rope_frequencies(64)
    k.rope_table(frequencies, out, first=7)
    check_table(out, range(7, 44), frequencies)
    assert room[0] == 9 and bool((room[-5:] == 9).all())
    k.rope_table([0.0, 65535.9, 1e-30], out.view(-1)[:12].view(2, 6), first=2 ** 32 - 2)
    check_table(out.view(-1)[:12].view(2, 6), [2 ** 32 - 2, 2 ** 32 - 1], [0.0, 65535.9, 1e-30])


def test_table_positions_out_of_range():
    err = error_word()
    out = torch.full((4, 8), 9.0, device=DEV)
    k.rope_table(k.rope_frequencies(8), out, positions=dev([3, -1, 2 ** 32, 5], np.int64), device_error=err)
    assert int(err.item()) == k.DEVERR_POS_RANGE
    assert bool((out[1:3] == 9).all())
    check_table(out, [3, 0, 0, 5], k.rope_frequencies(8), rows=[0, 3])


def test_table_is_what_the_inserts_take():
    """The fused step with a table of this library and with one made in numpy."""
    T, H = 40, 3
    gen = torch.Generator(device=DEV).manual_seed(2)
    q0 = torch.randn(T, H, 512, generator=gen, device=DEV).to(torch.bfloat16)
    kv = torch.randn(T, 512, generator=gen, device=DEV).to(torch.bfloat16)
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    positions, slots = torch.arange(T, device=DEV) * 7, torch.arange(T, device=DEV)
    mine = torch.empty(300, 64, device=DEV)
    k.rope_table(k.rope_frequencies(64), mine)
    a = np.arange(300)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    rows = []
    for table in (mine, dev(np.concatenate([np.cos(a), np.sin(a)], 1), np.float32)):
        q, cache = q0.clone(), torch.zeros(4 * 16, 512, dtype=torch.bfloat16, device=DEV)
        k.qnorm_rope_kv_bf16_insert(q, kv, w, positions, table, slots, cache, 4, 16, 1e-6)
        rows.append((q.float(), cache.float()))
    for x, y in zip(*rows):
        # entries differ by a step of 2^-24 at most: the bf16 outputs by a step here and there
        assert bool(((x - y).abs() <= 2.0 ** -7 * y.abs() + 2.0 ** -20).all())


# ---------------------------------------------------------------- rows

def check_rows(kind, T, H, width, offset, dim, half, inverse, in_place, make=None, seed=0, max_position=60):
    dtype, step = TYPES[kind]
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cos_sin = torch.empty(max_position, dim, device=DEV)
    k.rope_table(k.rope_frequencies(dim, 100.0), cos_sin)
    positions = torch.randint(0, max_position, (T,), generator=gen, device=DEV)
    x = torch.randn(T, H, width, generator=gen, device=DEV).to(dtype)
    if make is not None:
        x = make(x)
    before = x.double().cpu().numpy()
    out = x if in_place else torch.full((T, H, width), 9.0, device=DEV).to(dtype)
    k.rope_rows(x, positions, cos_sin, out=None if in_place else out, offset=offset, inverse=inverse,
                layout=k.ROPE_HALF if half else k.ROPE_PAIRS)
    angles = cos_sin.double().cpu().numpy()[positions.cpu().numpy()][:, None]
    want = latent.rotate(before, angles, offset, half, inverse)
    got = out.double().cpu().numpy()
    part = before[..., offset:offset + dim]
    i = np.arange(dim)
    partner = (i + dim // 2) % dim if half else i ^ 1
    size = np.ones_like(before)
    size[..., offset:offset + dim] = np.abs(part) + np.abs(part[..., partner])  # |c|, |s| <= 1
    tol = np.abs(want) * step + size * 2.0 ** -23 * (1 + step) + 2.0 ** -25 * (kind == "fp16")
    rest = np.ones(width, bool)
    rest[offset:offset + dim] = False
    assert np.array_equal(got[..., rest], before[..., rest])
    assert np.all(np.abs(got - want)[..., ~rest] <= tol[..., ~rest])
    return x, out


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,H,width,offset,dim", [
    (1, 1, 2, 0, 2), (3, 2, 64, 0, 64), (5, 7, 512, 448, 64), (33, 4, 128, 0, 64), (20, 3, 192, 128, 64),
    (9, 5, 96, 16, 48), (7, 3, 70, 3, 30), (4, 2, 33, 1, 32), (300, 8, 64, 32, 32), (2, 128, 256, 0, 256),
    (17, 1, 600, 100, 250), (6, 2, 40, 0, 40),
])
def test_rows(kind, half, in_place, T, H, width, offset, dim):
    check_rows(kind, T, H, width, offset, dim, half, inverse=(T + H) % 2 == 1, in_place=in_place, seed=T)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("half", [False, True])
def test_rows_by_the_ten_thousand(kind, half):
    """Enough rows for four a thread at once, an odd number of them."""
    check_rows(kind, 8191, 11, 64, 0, 32, half, False, False)
    check_rows(kind, 40001, 3, 16, 0, 16, half, True, True)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_strided(kind, in_place):
    def heads_outside(x):  # [H, T, D] seen as [T, H, D]
        return x.transpose(0, 1).contiguous().transpose(0, 1)

    def part_of_wider(x):
        room = torch.zeros(x.shape[0], x.shape[1] + 2, x.shape[2] + 24, dtype=x.dtype, device=DEV)
        room[:, 1:-1, 8:-16] = x
        return room[:, 1:-1, 8:-16]

    def off_by_one(x):
        room = torch.zeros(x.numel() + 1, dtype=x.dtype, device=DEV)
        room[1:] = x.reshape(-1)
        return room[1:].view(x.shape)

    for make in (heads_outside, part_of_wider, off_by_one):
        for half in (False, True):
            check_rows(kind, 19, 5, 64, 32, 32, half, False, in_place, make=make)
    if not in_place:
        check_rows(kind, 19, 5, 64, 32, 32, False, False, False, make=lambda x: x[:, :1].expand(-1, 5, -1))
        check_rows(kind, 19, 5, 64, 32, 32, True, True, False, make=lambda x: x[:1].expand(19, -1, -1))


def test_rows_leave_their_surroundings():
    room = torch.full((10, 6, 80), 5.0, dtype=torch.bfloat16, device=DEV)
    x = room[2:8, 1:5, 8:72]
    before = room.clone()
    cos_sin = torch.empty(9, 16, device=DEV)
    k.rope_table(k.rope_frequencies(16), cos_sin)
    k.rope_rows(x, torch.arange(1, 7, device=DEV), cos_sin, offset=24)
    changed = room != before
    inside = torch.zeros_like(changed)
    inside[2:8, 1:5, 32:48] = True
    assert bool(changed.any()) and not bool((changed & ~inside).any())
    out = torch.full((6, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    k.rope_rows(x, torch.arange(1, 7, device=DEV), cos_sin, out=out)
    assert torch.equal(out[..., :48], x[..., :48])


def test_rows_positions_out_of_range_and_none():
    err = error_word()
    cos_sin = torch.empty(9, 16, device=DEV)
    k.rope_table(k.rope_frequencies(16), cos_sin)
    x = torch.randn(5, 3, 32, device=DEV)
    out = torch.full_like(x, 9.0)
    k.rope_rows(x, dev([0, 9, 4, -1, 2 ** 40], np.int64), cos_sin, out=out, device_error=err)
    assert int(err.item()) == k.DEVERR_POS_RANGE
    assert bool((out[[1, 3, 4]] == 9).all()) and torch.equal(out[0], x[0])
    k.rope_rows(x[:0], torch.zeros(0, dtype=torch.int64, device=DEV), cos_sin)
    flat = torch.randn(5, 32, device=DEV)
    three = flat.clone()[:, None]
    at = dev([0, 1, 2, 3, 4], np.int64)
    k.rope_rows(flat, at, cos_sin)
    k.rope_rows(three, at, cos_sin)
    assert torch.equal(flat, three[:, 0])


@pytest.mark.parametrize("half", [False, True])
def test_inverse_is_the_gradient(half):
    """Of sum(out * g) by x: the inverse of g, against differences (the map is linear, so a
    difference over a step of 1 is exact but for the roundings of two outputs)."""
    layout = k.ROPE_HALF if half else k.ROPE_PAIRS
    gen = torch.Generator(device=DEV).manual_seed(4)
    cos_sin = torch.empty(9, 8, device=DEV)
    k.rope_table(k.rope_frequencies(8, 50.0), cos_sin)
    x, g = (torch.randn(4, 2, 12, generator=gen, device=DEV) for _ in range(2))
    at = dev([0, 3, 8, 5], np.int64)
    grad = torch.empty_like(g)
    k.rope_rows(g, at, cos_sin, out=grad, offset=2, layout=layout, inverse=True)

    def loss(y):
        out = torch.empty_like(y)
        k.rope_rows(y, at, cos_sin, out=out, offset=2, layout=layout)
        return (out.double() * g.double()).sum()

    base = loss(x)
    for i in range(0, x.numel(), 5):
        step = torch.zeros_like(x)
        step.view(-1)[i] = 1.0
        # fp32 outputs of size up to 8, two that change with their partners: 4 roundings of 2^-21 and |g| <= 5
        assert abs(float(loss(x + step) - base - grad.view(-1)[i])) <= 4 * 8 * 2.0 ** -22 * 5
    # there and back: two roundings each way
    back = torch.empty_like(x)
    k.rope_rows(x, at, cos_sin, out=back, offset=2, layout=layout)
    k.rope_rows(back, at, cos_sin, offset=2, layout=layout, inverse=True)
    assert torch.allclose(back, x, rtol=0, atol=8 * 2.0 ** -21)


def test_special_values_stay_in_their_pair():
    cos_sin = torch.empty(4, 8, device=DEV)
    k.rope_table(k.rope_frequencies(8), cos_sin)
    x = torch.randn(2, 1, 8, device=DEV).to(torch.bfloat16)
    x[0, 0, 2], x[1, 0, 7] = float("nan"), float("inf")
    k.rope_rows(x, dev([1, 2], np.int64), cos_sin)
    assert torch.isnan(x[0, 0, 2:4]).all() and torch.isfinite(x[0, 0, [0, 1, 4, 5, 6, 7]]).all()
    assert not torch.isfinite(x[1, 0, 6:8]).any() and torch.isfinite(x[1, 0, :6]).all()


def test_in_a_graph_and_on_another_stream():
    cos_sin = torch.empty(500, 64, device=DEV)
    frequencies = k.rope_frequencies(64)
    x = torch.randn(40, 6, 512, device=DEV).to(torch.bfloat16)
    at = torch.arange(40, device=DEV)
    eager = torch.empty_like(x)
    k.rope_table(frequencies, cos_sin)
    k.rope_rows(x, at, cos_sin, out=eager)
    out, table = torch.zeros_like(x), torch.zeros_like(cos_sin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k.rope_table(frequencies, table)
        k.rope_rows(x, at, table, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager) and torch.equal(table, cos_sin)
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    k.rope_rows(x, at, cos_sin, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, eager)


def test_offsets_past_4_gib():
    """5 GB of bf16 rows, in place: the last ones are turned like a copy of them alone."""
    T, H = 40000, 122
    x = torch.zeros(T, H, 512, dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn(3, H, 512, device=DEV).to(torch.bfloat16)
    tail = x[-3:].clone()
    cos_sin = torch.empty(100, 64, device=DEV)
    k.rope_table(k.rope_frequencies(64), cos_sin)
    at = torch.arange(T, device=DEV) % 100
    k.rope_rows(x, at, cos_sin)
    k.rope_rows(tail, at[-3:].contiguous(), cos_sin)
    assert torch.equal(x[-3:], tail) and not bool(x[:-3].any())
