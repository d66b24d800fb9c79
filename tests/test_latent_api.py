"""The attention over the FP8 and bf16 caches, the kept path and the rotary positions without a
GPU: sizes, host arithmetic, and every refusal comes before CUDA is touched."""
import ctypes
import math

import numpy as np
import pytest

import kv_norm_rope_gb300 as k
from oracle import latent

A = 1 << 20  # a made-up device pointer: every call below is refused, or returns early, on the host


def _attention(store=0, q=A, cache=A, nb=4, bs=64, table=A, stride=8, width=8, lens=A, batch=2, Q=1, H=8,
               scale=0.1, window=0, tree=None, sinks=None, out=A, lse=None, ws=A, ws_bytes=None, err=None):
    if ws_bytes is None:
        ws_bytes = k.latent_attention_workspace_bytes()
    return k.lib().dsv4_latent_attention(store, q, cache, nb, bs, table, stride, width, lens, batch, Q, H, scale,
                                         window, tree, sinks, out, lse, ws, ws_bytes, err, None)


_SHARED = [
    (dict(nb=0), k.ERR_SHAPE), (dict(bs=0), k.ERR_SHAPE), (dict(nb=2**32, bs=2), k.ERR_SHAPE),
    (dict(nb=2**31, bs=1), k.ERR_SHAPE), (dict(width=0), k.ERR_SHAPE),
    (dict(stride=7, width=8), k.ERR_SHAPE), (dict(batch=-1), k.ERR_SHAPE),
    (dict(batch=65536), k.ERR_SHAPE), (dict(width=2**25, stride=2**25, bs=64), k.ERR_SHAPE),
    (dict(store=4), k.ERR_VALUE), (dict(store=-1), k.ERR_VALUE),
    (dict(cache=None), k.ERR_NULL), (dict(table=None), k.ERR_NULL), (dict(lens=None), k.ERR_NULL),
    (dict(cache=A + 4), k.ERR_ALIGN), (dict(table=A + 2), k.ERR_ALIGN), (dict(store=1, cache=A + 8), k.ERR_ALIGN),
    (dict(lens=A + 2), k.ERR_ALIGN), (dict(err=A + 2), k.ERR_ALIGN), (dict(batch=0), k.OK),
]


@pytest.mark.parametrize("kw,status", _SHARED + [
    (dict(store=2), k.ERR_VALUE), (dict(store=3), k.ERR_VALUE),
    (dict(Q=0), k.ERR_SHAPE), (dict(H=0), k.ERR_SHAPE), (dict(window=-1), k.ERR_SHAPE),
    (dict(Q=2**20, H=2**20), k.ERR_SHAPE), (dict(Q=2**15, H=2**10, batch=65535), k.ERR_SHAPE),
    (dict(scale=0.0), k.ERR_VALUE), (dict(scale=-1.0), k.ERR_VALUE), (dict(scale=math.inf), k.ERR_VALUE),
    (dict(scale=math.nan), k.ERR_VALUE), (dict(scale=2.0**33), k.ERR_VALUE),
    (dict(tree=A, Q=65), k.ERR_SHAPE), (dict(tree=A, Q=8, window=7), k.ERR_SHAPE),
    (dict(tree=A + 4, Q=8), k.ERR_ALIGN),
    (dict(ws_bytes=0), k.ERR_SHAPE), (dict(ws=None), k.ERR_NULL), (dict(q=None), k.ERR_NULL),
    (dict(out=None), k.ERR_NULL), (dict(q=A + 8), k.ERR_ALIGN), (dict(out=A + 8), k.ERR_ALIGN),
    (dict(ws=A + 8), k.ERR_ALIGN), (dict(sinks=A + 2), k.ERR_ALIGN), (dict(lse=A + 2), k.ERR_ALIGN),
])
def test_attention_refusals(kw, status):
    assert _attention(**kw) == status


def _keep(store=0, cache=A, nb=4, bs=64, table=A, stride=8, width=8, lens=A, batch=2, Q=8, path=A, path_lens=A,
          new=A, err=None):
    return k.lib().dsv4_tree_keep(store, cache, nb, bs, table, stride, width, lens, batch, Q, path, path_lens, new,
                                  err, None)


@pytest.mark.parametrize("kw,status", _SHARED + [
    (dict(Q=0), k.ERR_SHAPE), (dict(Q=65), k.ERR_SHAPE), (dict(path=None), k.ERR_NULL),
    (dict(path_lens=None), k.ERR_NULL), (dict(new=None), k.ERR_NULL), (dict(path=A + 2), k.ERR_ALIGN),
    (dict(path_lens=A + 2), k.ERR_ALIGN), (dict(new=A + 2), k.ERR_ALIGN),
    (dict(store=2, cache=A + 8), k.ERR_ALIGN), (dict(store=3, cache=A + 2), k.ERR_ALIGN),
])
def test_keep_refusals(kw, status):
    assert _keep(**kw) == status


def test_positions_of_a_launch_are_counted_in_32_bits():
    """The line that is dealt to the CTAs has four positions a row tile beside its tiles of 64 keys."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the pointers are made up")
    # 65535 requests of 8 row tiles (512 heads): 2^31 - 1024 positions allow 4096 - 4 tiles
    size = dict(batch=65535, H=512, bs=64, nb=1 << 20)
    for blocks, fits in ((4093, False), (4091, True)):
        status = _attention(width=blocks, stride=blocks, **size)
        assert status == (k.ERR_CUDA if fits else k.ERR_SHAPE), (blocks, status)


# ---------------------------------------------------------------- frequencies

def _reference_frequencies(dim, theta, scaling, factor, original, fast, slow):
    if scaling == k.ROPE_NTK and dim > 2:
        theta = theta * factor ** (dim / (dim - 2))
    out = []
    if scaling == k.ROPE_YARN:
        index = lambda turns: dim / 2 * math.log(original / (2 * math.pi * turns)) / math.log(theta)
        low, high = max(0, math.floor(index(fast))), min(dim // 2 - 1, math.ceil(index(slow)))
    for i in range(dim // 2):
        f = theta ** (-2 * i / dim)
        if scaling == k.ROPE_LINEAR:
            f /= factor
        elif scaling == k.ROPE_YARN:
            r = 0.0 if i <= low else 1.0 if i >= high else (i - low) / (high - low)
            f = f * (1 - r) + f / factor * r
        out.append(f)
    return out


@pytest.mark.parametrize("dim", [2, 4, 64, 96, 256])
@pytest.mark.parametrize("scaling", [k.ROPE_PLAIN, k.ROPE_LINEAR, k.ROPE_NTK, k.ROPE_YARN])
@pytest.mark.parametrize("theta,factor,original", [(10000.0, 16.0, 65536.0), (500000.0, 40.0, 4096.0), (1.5, 1.0, 10.0)])
def test_frequencies(dim, scaling, theta, factor, original):
    got = k.rope_frequencies(dim, theta, scaling, factor, original)
    want = _reference_frequencies(dim, theta, scaling, factor, original, 32.0, 1.0)
    assert len(got) == dim // 2
    # a few operations in 64 bits, a power of up to 256 log theta among them
    assert np.allclose(got, want, rtol=1e-13, atol=0)


def test_yarn_keeps_fast_pairs_and_stretches_slow_ones():
    plain, yarn = k.rope_frequencies(64), k.rope_frequencies(64, 10000.0, k.ROPE_YARN, 16.0, 65536.0)
    assert yarn[0] == plain[0] and yarn[-1] == plain[-1] / 16.0
    ratio = np.array(yarn) / np.array(plain)
    assert np.all(np.diff(ratio) <= 1e-15) and ratio[0] == 1.0


_BUFFER = (ctypes.c_double * 128)()


@pytest.mark.parametrize("args,status", [
    ((0, 63, 1e4, 1.0, 0, 0, 0), k.ERR_SHAPE), ((0, 0, 1e4, 1.0, 0, 0, 0), k.ERR_SHAPE),
    ((0, 258, 1e4, 1.0, 0, 0, 0), k.ERR_SHAPE), ((4, 64, 1e4, 1.0, 0, 0, 0), k.ERR_VALUE),
    ((-1, 64, 1e4, 1.0, 0, 0, 0), k.ERR_VALUE), ((0, 64, 1.0, 1.0, 0, 0, 0), k.ERR_VALUE),
    ((0, 64, math.inf, 1.0, 0, 0, 0), k.ERR_VALUE), ((0, 64, math.nan, 1.0, 0, 0, 0), k.ERR_VALUE),
    ((1, 64, 1e4, 0.5, 0, 0, 0), k.ERR_VALUE), ((2, 64, 1e4, math.nan, 0, 0, 0), k.ERR_VALUE),
    ((3, 64, 1e4, 2.0, 0.0, 32, 1), k.ERR_VALUE), ((3, 64, 1e4, 2.0, 4096, 1, 1), k.ERR_VALUE),
    ((3, 64, 1e4, 2.0, 4096, 32, 0), k.ERR_VALUE), ((3, 64, 1e4, 2.0, 4096, 32, 1), k.OK),
])
def test_frequency_refusals(args, status):
    assert k.lib().dsv4_rope_frequencies(*args, _BUFFER) == status


def test_frequencies_need_room():
    assert k.lib().dsv4_rope_frequencies(0, 64, 1e4, 1.0, 0, 0, 0, None) == k.ERR_NULL


def _table(freq=(1.0, 0.5), dim=4, magnitude=1.0, positions=None, first=0, n=3, out=A, err=None):
    f = None if freq is None else (ctypes.c_double * len(freq))(*freq)
    return k.lib().dsv4_rope_table(f, dim, magnitude, positions, first, n, out, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=3), k.ERR_SHAPE), (dict(dim=0), k.ERR_SHAPE), (dict(dim=258), k.ERR_SHAPE), (dict(n=-1), k.ERR_SHAPE),
    (dict(first=-1), k.ERR_SHAPE), (dict(first=2**32 - 2), k.ERR_SHAPE), (dict(n=2**32 + 1), k.ERR_SHAPE),
    (dict(magnitude=math.nan), k.ERR_VALUE), (dict(magnitude=math.inf), k.ERR_VALUE), (dict(magnitude=1e-6), k.ERR_VALUE),
    (dict(magnitude=70000.0), k.ERR_VALUE), (dict(freq=(1.0, -0.5)), k.ERR_VALUE),
    (dict(freq=(1.0, math.nan)), k.ERR_VALUE), (dict(freq=(65536.0, 1.0)), k.ERR_VALUE), (dict(freq=None), k.ERR_NULL),
    (dict(out=None), k.ERR_NULL), (dict(out=A + 2), k.ERR_ALIGN), (dict(positions=A + 4), k.ERR_ALIGN),
    (dict(err=A + 2), k.ERR_ALIGN), (dict(n=0, out=None), k.OK),
])
def test_table_refusals(kw, status):
    assert _table(**kw) == status


def _rows(type=0, x=A, xt=1024, xh=128, out=A, ot=1024, oh=128, T=4, H=8, width=128, offset=64, dim=64, layout=0,
          inverse=0, positions=A, cos_sin=A, max_position=16, err=None):
    return k.lib().dsv4_rope_rows(type, x, xt, xh, out, ot, oh, T, H, width, offset, dim, layout, inverse, positions,
                                  cos_sin, max_position, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=63), k.ERR_SHAPE), (dict(dim=0), k.ERR_SHAPE), (dict(dim=258, width=512), k.ERR_SHAPE),
    (dict(width=0), k.ERR_SHAPE), (dict(width=65537), k.ERR_SHAPE), (dict(offset=-1), k.ERR_SHAPE),
    (dict(offset=65), k.ERR_SHAPE), (dict(T=-1), k.ERR_SHAPE), (dict(H=0), k.ERR_SHAPE), (dict(max_position=0), k.ERR_SHAPE),
    (dict(T=2**28, H=8), k.ERR_SHAPE), (dict(xt=-1), k.ERR_SHAPE), (dict(ot=2**31 + 1), k.ERR_SHAPE),
    (dict(out=2 * A, oh=127), k.ERR_SHAPE), (dict(out=2 * A, ot=1023), k.ERR_SHAPE), (dict(out=2 * A, oh=0), k.ERR_SHAPE),
    (dict(xh=0), k.ERR_SHAPE), (dict(type=3), k.ERR_VALUE), (dict(type=-1), k.ERR_VALUE), (dict(layout=2), k.ERR_VALUE),
    (dict(inverse=2), k.ERR_VALUE), (dict(x=None, out=2 * A), k.ERR_NULL), (dict(out=None), k.ERR_NULL),
    (dict(positions=None), k.ERR_NULL), (dict(cos_sin=None), k.ERR_NULL), (dict(x=A + 1, out=A + 1), k.ERR_ALIGN),
    (dict(type=2, x=A + 2, out=A + 2), k.ERR_ALIGN), (dict(positions=A + 4), k.ERR_ALIGN), (dict(cos_sin=A + 8), k.ERR_ALIGN),
    (dict(err=A + 2), k.ERR_ALIGN), (dict(T=0), k.OK),
])
def test_rows_refusals(kw, status):
    assert _rows(**kw) == status


# ---------------------------------------------------------------- the oracle

def test_oracle_codes():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, latent.E4M3, equal_nan=True)


def test_oracle_angles():
    for p in (0, 1, 12345, 2 ** 20 + 7):
        for f in (1.0, 0.1, 1e-4, 3.25):
            a = latent.angle(p, f)
            assert -math.pi <= a <= math.pi
            assert math.cos(a) == pytest.approx(math.cos(p * f), abs=2e-9)
            assert math.sin(a) == pytest.approx(math.sin(p * f), abs=2e-9)
    assert latent.angle(1, 2.0) == 2.0 and latent.angle(1, 6.5) == pytest.approx(6.5 - 2 * math.pi, rel=1e-14)


def test_oracle_visibility():
    assert latent.visible(10, 3, 0, 0) == list(range(8)) and latent.visible(10, 3, 2, 4) == [6, 7, 8, 9]
    assert latent.visible(2, 3, 0, 0) == [] and latent.visible(2, 3, 2, 0) == [0, 1]
    tree = [0b1, 0b11, 0b101, 0]
    assert latent.visible(10, 4, 2, 0, tree) == [0, 1, 2, 3, 4, 5, 6, 8]
    assert latent.visible(10, 4, 2, 4, tree) == [4, 5, 6, 8] and latent.visible(10, 4, 3, 0, tree) == []
    assert latent.visible(3, 4, 1, 0, tree) == [0]  # key c + 0 = -1 is none


# ---------------------------------------------------------------- the binding

def test_binding_refuses_tensors():
    torch = pytest.importorskip("torch")
    nb, bs, B = 3, 16, 2
    cache = torch.zeros(k.fp8_cache_bytes(nb, bs), dtype=torch.uint8)
    q = torch.zeros(B, 1, 4, 512, dtype=torch.bfloat16)
    table, lens = torch.zeros(B, 2, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    ws = torch.empty(k.latent_attention_workspace_bytes(), dtype=torch.uint8)

    def call(store=k.STORE_FP8, q=q, cache=cache, table=table, lens=lens, out=torch.empty_like(q), **kw):
        k.latent_attention(store, q, cache, nb, bs, table, lens, 0.1, out, workspace=ws, **kw)

    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(ValueError, match="batch, q_len"):
        call(q=q[0])
    with pytest.raises(TypeError, match="q"):
        call(q=q.float())
    with pytest.raises(ValueError, match="kv_cache"):
        call(cache=cache[:-1])
    with pytest.raises(ValueError, match="kv_cache"):
        call(store=k.STORE_BF16)
    with pytest.raises(TypeError, match="block_table"):
        call(table=table.long())
    with pytest.raises(ValueError, match="block_table"):
        call(table=table[:1])
    with pytest.raises(ValueError, match="out"):
        call(out=q[:1])
    with pytest.raises(ValueError, match="lse"):
        call(lse=torch.zeros(3))
    with pytest.raises(ValueError, match="sinks"):
        call(sinks=torch.zeros(3))
    with pytest.raises(TypeError, match="tree"):
        call(tree=torch.zeros(B, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="tree"):
        call(tree=torch.zeros(B, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="handle"):
        k.latent_attention(k.STORE_FP8, q, cache, nb, bs, table, lens, 0.1, q, stream=7)
    path = torch.zeros(B, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="batch, q_len"):
        k.tree_keep(k.STORE_FP8, cache, nb, bs, table, lens, path[0], lens, lens)
    with pytest.raises(ValueError, match="path_lens"):
        k.tree_keep(k.STORE_FP8, cache, nb, bs, table, lens, path, lens[:1], lens)
    with pytest.raises(ValueError, match="kv_cache"):
        k.tree_keep(k.STORE_FP8, cache[:-1], nb, bs, table, lens, path, lens, lens)
    with pytest.raises(ValueError, match="CUDA"):
        k.tree_keep(k.STORE_FP8, cache, nb, bs, table, lens, path, lens, lens)
    with pytest.raises(ValueError, match="out"):
        k.rope_table((1.0, 0.5), torch.zeros(3, 5))
    with pytest.raises(ValueError, match="positions"):
        k.rope_table((1.0, 0.5), torch.zeros(3, 4), positions=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        k.rope_table((1.0, 0.5), torch.zeros(3, 4))
    x, positions, cos_sin = torch.zeros(3, 2, 16), torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    with pytest.raises(TypeError, match="x"):
        k.rope_rows(x.double(), positions, cos_sin)
    with pytest.raises(TypeError, match="out"):
        k.rope_rows(x, positions, cos_sin, out=x.half())
    with pytest.raises(ValueError, match="one shape"):
        k.rope_rows(x, positions, cos_sin, out=x[:2])
    with pytest.raises(ValueError, match="positions"):
        k.rope_rows(x, positions[:2], cos_sin)
    with pytest.raises(ValueError, match="cos_sin_cache"):
        k.rope_rows(x, positions, cos_sin[0])
    with pytest.raises(ValueError, match="CUDA"):
        k.rope_rows(x, positions, cos_sin)
    with pytest.raises(k.Dsv4Error):
        k.rope_frequencies(63)


def test_no_cpu_fallback_without_a_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    assert _attention() == _keep() == _table() == _rows() == k.ERR_CUDA
