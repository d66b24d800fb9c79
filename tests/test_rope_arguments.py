"""Arguments of the rotary calls that only the host's arithmetic can tell apart, without a GPU."""
import random

import pytest

import kv_norm_rope_gb300 as k

torch = pytest.importorskip("torch")
if torch.cuda.is_available():  # pragma: no cover
    pytest.skip("the pointers are made up", allow_module_level=True)

A = 1 << 20  # a made-up device pointer: what is not refused ends for want of a GPU (ERR_CUDA)


def _rows(type=0, x=A, xt=1024, xh=128, out=1 << 62, ot=1024, oh=128, T=4, H=8, width=128, layout=0):
    return k.lib().dsv4_rope_rows(type, x, xt, xh, out, ot, oh, T, H, width, 0, 64, layout, 0, A, A, 16, None, None)


@pytest.mark.parametrize("kw,status", [
    # (2^31 - 2) * 2^31 + 128 elements: of 2 bytes 2^33 - 256 bytes short of 2^63, of 4 twice as many
    (dict(T=2**31 - 1, H=1, xt=2**31), k.ERR_CUDA), (dict(T=1, H=2**31 - 1, type=1, xh=2**31), k.ERR_CUDA),
    (dict(T=2**31 - 1, H=1, type=2, xt=2**31), k.ERR_SHAPE), (dict(T=2**31 - 1, H=1, type=2, ot=2**31), k.ERR_SHAPE),
    (dict(T=1, H=2**31 - 1, type=2, xh=2**31), k.ERR_SHAPE),
    (dict(T=2**31 - 1, H=1, type=2, xt=2**30), k.ERR_CUDA), (dict(T=2**31 - 1, H=1, type=2, xt=2**30 + 4), k.ERR_SHAPE),
    (dict(T=2**30, H=1, type=2, xt=2**31), k.ERR_CUDA), (dict(T=2**30 + 2, H=1, type=2, xt=2**31), k.ERR_SHAPE),
    (dict(), k.ERR_CUDA),
])
def test_bytes_of_rows_are_counted_in_64_bits(kw, status):
    assert _rows(**kw) == status


def _meet(d, T, H, width, ts, hs):
    """Whether rows [d + t ts + h hs, + width) and [t' ts + h' hs, + width) share an element."""
    starts = [t * ts + h * hs for t in range(T) for h in range(H)]
    taken = {a + i for a in starts for i in range(width)}
    return any(a + d + i in taken for a in starts for i in range(width))


def test_rows_that_overlap_their_input_are_refused():
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(600):
        T, H, width = rng.randint(1, 5), rng.randint(1, 5), rng.randint(2, 9)
        inner = width + rng.choice([0, 0, 1, 5, 2 * width])
        count = rng.choice([T, H])
        outer = (count - 1) * inner + width + rng.choice([0, 0, 1, 3, 20])
        ts, hs = (outer, inner) if count == H else (inner, outer)
        type = rng.randint(0, 2)
        size = 4 if type == 2 else 2
        for d in rng.sample(range(-150, 150), 20):
            if d == 0:
                continue
            # what strides of a single row are makes no difference
            xt, xh = (ts if T > 1 else rng.randint(0, 50)), (hs if H > 1 else rng.randint(0, 50))
            status = k.lib().dsv4_rope_rows(type, A, xt, xh, A + d * size, ts, hs, T, H, width, 0, 2, 0, 0, A, A, 16, None, None)
            meet = _meet(d, T, H, width, ts, hs)
            seen[meet] += 1
            assert status == (k.ERR_SHAPE if meet else k.ERR_CUDA), (type, T, H, width, ts, hs, d)
    assert min(seen.values()) > 1000


def test_far_rows_of_the_largest_sizes():
    for T, H in ((2**31 - 1, 1), (1, 2**31 - 1), (2**16 - 1, 2**15)):
        for out in (A + 2**40, 2**62, A + 2, A + 128 * 2):
            stride = min(128 * H, 2**31)  # (of one token: it makes no difference)
            status = _rows(T=T, H=H, xt=stride, ot=stride, out=out)
            ends = A + 2 * 128 * T * H
            assert status == (k.ERR_SHAPE if out < ends else k.ERR_CUDA), (T, H, out)
