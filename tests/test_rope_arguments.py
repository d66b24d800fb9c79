"""Arguments of the rotary calls that only the host's arithmetic can tell apart, without a GPU."""
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
