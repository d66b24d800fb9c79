"""Sizes at the ends of what the 4-bit cache's operators count in 32 bits, refused on the host
before CUDA is touched."""
import pytest

import kv_norm_rope_gb300 as k
from tests.test_fp4_api import _attention, _evict, _weights


def _accepted(status):
    """Past the checks of sizes and pointers: without a GPU the launch itself fails."""
    return status == k.ERR_CUDA


@pytest.mark.parametrize("call", [_attention, _weights])
def test_positions_of_a_launch_are_counted_in_32_bits(call):
    """The line that is dealt to the CTAs has two positions a row tile beside its tiles of keys."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the pointers are made up")
    # 65535 requests of 16 row tiles (1024 heads) and 2047 tiles of 128 keys: 2146402320 tiles,
    # 2148499440 positions
    size = dict(batch=65535, H=1024, bs=64, nb=1 << 20)
    for blocks, fits in ((2047 * 2, False), (2046 * 2, True)):
        status = call(width=blocks, stride=blocks, **size)
        assert _accepted(status) if fits else status == k.ERR_SHAPE, (blocks, status)


def test_rows_of_an_eviction_fit_its_grid():
    """A block moves 64 kept rows, and a grid has at most 2^31 - 1 blocks."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the pointers are made up")
    most = 2 ** 31 - 1
    width = 2 ** 31 // 64
    size = dict(batch=65535, recent=0, new_width=width, new_stride=width, budget=most)
    assert _evict(**size) == k.ERR_SHAPE
    assert _accepted(_evict(**dict(size, batch=64, budget=most)))
