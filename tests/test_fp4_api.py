"""The 4-bit cache's entry points without a GPU: sizes, and every refusal comes before CUDA
is touched."""
import math

import pytest

import kv_norm_rope_gb300 as k

# fake device pointers: never dereferenced, because every call below is refused (or
# returns early) on the host
A = 1 << 20


def test_cache_bytes():
    assert k.fp4_cache_bytes(1024, 64) == 1024 * 64 * 368
    assert k.fp4_cache_bytes(0, 64) == 0 and k.fp4_cache_bytes(4, 0) == 0
    assert k.FP4_SLOT_BYTES == 368


def _insert(q=A, kv=A, w=A, pos=A, cs=A, max_pos=64, slot=A, cache=A, nb=4, bs=64, T=16, H=8,
            eps=1e-6, err=None):
    return k.lib().dsv4_qnorm_rope_kv_fp4_insert(q, kv, w, pos, cs, max_pos, slot, cache, nb, bs, T,
                                                 H, eps, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), k.ERR_SHAPE), (dict(H=-1), k.ERR_SHAPE), (dict(nb=0), k.ERR_SHAPE),
    (dict(bs=0), k.ERR_SHAPE), (dict(nb=2**32, bs=2), k.ERR_SHAPE), (dict(max_pos=0), k.ERR_SHAPE),
    (dict(eps=-1.0), k.ERR_VALUE), (dict(eps=math.nan), k.ERR_VALUE),
    (dict(q=None), k.ERR_NULL), (dict(kv=None), k.ERR_NULL), (dict(w=None), k.ERR_NULL),
    (dict(pos=None), k.ERR_NULL), (dict(cs=None), k.ERR_NULL), (dict(slot=None), k.ERR_NULL),
    (dict(cache=None), k.ERR_NULL),
    (dict(q=A + 8), k.ERR_ALIGN), (dict(cache=A + 8), k.ERR_ALIGN), (dict(slot=A + 4), k.ERR_ALIGN),
    (dict(err=A + 2), k.ERR_ALIGN), (dict(T=0), k.OK),
])
def test_insert_refusals(kw, status):
    assert _insert(**kw) == status


def _gather(cache=A, nb=4, bs=64, slots=A, n=5, out=A, err=None):
    return k.lib().dsv4_fp4_dequant_gather(cache, nb, bs, slots, n, out, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), k.ERR_SHAPE), (dict(nb=0), k.ERR_SHAPE), (dict(bs=0), k.ERR_SHAPE),
    (dict(nb=2**32, bs=2), k.ERR_SHAPE), (dict(cache=None), k.ERR_NULL),
    (dict(slots=None), k.ERR_NULL), (dict(out=None), k.ERR_NULL), (dict(cache=A + 8), k.ERR_ALIGN),
    (dict(out=A + 8), k.ERR_ALIGN), (dict(slots=A + 4), k.ERR_ALIGN), (dict(n=0), k.OK),
])
def test_gather_refusals(kw, status):
    assert _gather(**kw) == status


_SHARED = [
    (dict(nb=0), k.ERR_SHAPE), (dict(bs=0), k.ERR_SHAPE), (dict(nb=2**32, bs=2), k.ERR_SHAPE),
    (dict(nb=2**31, bs=1), k.ERR_SHAPE), (dict(width=0), k.ERR_SHAPE),
    (dict(stride=7, width=8), k.ERR_SHAPE), (dict(batch=-1), k.ERR_SHAPE),
    (dict(batch=65536), k.ERR_SHAPE), (dict(width=2**25, stride=2**25, bs=64), k.ERR_SHAPE),
    (dict(cache=None), k.ERR_NULL), (dict(table=None), k.ERR_NULL), (dict(lens=None), k.ERR_NULL),
    (dict(cache=A + 8), k.ERR_ALIGN), (dict(table=A + 2), k.ERR_ALIGN),
    (dict(lens=A + 2), k.ERR_ALIGN), (dict(err=A + 2), k.ERR_ALIGN), (dict(batch=0), k.OK),
]
_QUERY = [
    (dict(Q=0), k.ERR_SHAPE), (dict(H=0), k.ERR_SHAPE), (dict(window=-1), k.ERR_SHAPE),
    (dict(Q=2**20, H=2**20), k.ERR_SHAPE), (dict(Q=2**15, H=2**10, batch=65535), k.ERR_SHAPE),
    (dict(scale=0.0), k.ERR_VALUE), (dict(scale=-1.0), k.ERR_VALUE),
    (dict(scale=math.inf), k.ERR_VALUE), (dict(scale=math.nan), k.ERR_VALUE),
    (dict(scale=2.0**33), k.ERR_VALUE),
    (dict(q=None), k.ERR_NULL), (dict(q=A + 8), k.ERR_ALIGN),
]


def _attention(q=A, cache=A, nb=4, bs=64, table=A, stride=8, width=8, lens=A, batch=2, Q=1, H=8,
               scale=0.1, window=0, sinks=None, out=A, lse=None, ws=A, ws_bytes=None, err=None):
    if ws_bytes is None:
        ws_bytes = k.fp4_attention_workspace_bytes()
    return k.lib().dsv4_fp4_attention(q, cache, nb, bs, table, stride, width, lens, batch, Q, H, scale,
                                      window, sinks, out, lse, ws, ws_bytes, err, None)


@pytest.mark.parametrize("kw,status", _SHARED + _QUERY + [
    (dict(ws_bytes=0), k.ERR_SHAPE), (dict(ws=None), k.ERR_NULL), (dict(out=None), k.ERR_NULL),
    (dict(out=A + 8), k.ERR_ALIGN), (dict(ws=A + 8), k.ERR_ALIGN), (dict(sinks=A + 2), k.ERR_ALIGN),
    (dict(lse=A + 2), k.ERR_ALIGN),
])
def test_attention_refusals(kw, status):
    assert _attention(**kw) == status


def _weights(q=A, cache=A, nb=4, bs=64, table=A, stride=8, width=8, lens=A, batch=2, Q=1, H=8,
             scale=0.1, window=0, lse=A, w=A, w_stride=512, w_width=512, err=None):
    return k.lib().dsv4_fp4_attention_weights(q, cache, nb, bs, table, stride, width, lens, batch, Q, H,
                                              scale, window, lse, w, w_stride, w_width, err, None)


@pytest.mark.parametrize("kw,status", _SHARED + _QUERY + [
    (dict(w_width=-1), k.ERR_SHAPE), (dict(w_stride=511), k.ERR_SHAPE), (dict(lse=None), k.ERR_NULL),
    (dict(w=None), k.ERR_NULL), (dict(w=A + 2), k.ERR_ALIGN), (dict(lse=A + 2), k.ERR_ALIGN),
])
def test_weights_refusals(kw, status):
    assert _weights(**kw) == status


def _evict(cache=A, nb=4, bs=64, table=A, stride=8, width=8, lens=A, batch=2, w=A, w_stride=512,
           w_width=512, budget=100, recent=10, new=A, new_stride=2, new_width=2, kept=A, new_lens=A,
           new_w=A, err=None):
    return k.lib().dsv4_fp4_evict(cache, nb, bs, table, stride, width, lens, batch, w, w_stride, w_width,
                                  budget, recent, new, new_stride, new_width, kept, new_lens, new_w, err,
                                  None)


@pytest.mark.parametrize("kw,status", _SHARED + [
    (dict(budget=0, recent=0), k.ERR_SHAPE), (dict(recent=-1), k.ERR_SHAPE),
    (dict(recent=101), k.ERR_SHAPE), (dict(new_width=1), k.ERR_SHAPE),
    (dict(new_width=0), k.ERR_SHAPE), (dict(new_width=3, new_stride=2), k.ERR_SHAPE),
    (dict(w_width=-1), k.ERR_SHAPE), (dict(w_stride=511), k.ERR_SHAPE),
    (dict(w=None), k.ERR_NULL), (dict(new=None), k.ERR_NULL), (dict(kept=None), k.ERR_NULL),
    (dict(new_lens=None), k.ERR_NULL), (dict(new_w=None), k.ERR_NULL),
    (dict(w=A + 2), k.ERR_ALIGN), (dict(new=A + 2), k.ERR_ALIGN), (dict(kept=A + 2), k.ERR_ALIGN),
    (dict(new_lens=A + 2), k.ERR_ALIGN), (dict(new_w=A + 2), k.ERR_ALIGN),
])
def test_evict_refusals(kw, status):
    assert _evict(**kw) == status


def test_binding_refuses_tensors():
    torch = pytest.importorskip("torch")
    nb, bs, B = 3, 16, 2
    cache = torch.zeros(k.fp4_cache_bytes(nb, bs), dtype=torch.uint8)
    q = torch.zeros(B, 1, 4, 512, dtype=torch.bfloat16)
    table, lens = torch.zeros(B, 2, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    out = torch.empty_like(q)
    ws = torch.empty(k.fp4_attention_workspace_bytes(), dtype=torch.uint8)

    def call(q=q, cache=cache, table=table, lens=lens, out=out, **kw):
        k.fp4_attention(q, cache, nb, bs, table, lens, 0.1, out, workspace=ws, **kw)

    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(ValueError, match="batch, q_len"):
        call(q=q[0])
    with pytest.raises(TypeError, match="q"):
        call(q=q.float())
    with pytest.raises(ValueError, match="kv_cache"):
        call(cache=cache[:-1])
    with pytest.raises(TypeError, match="block_table"):
        call(table=table.long())
    with pytest.raises(ValueError, match="block_table"):
        call(table=table[:1])
    with pytest.raises(ValueError, match="block_table"):
        call(table=table.t().contiguous().t())
    with pytest.raises(ValueError, match="out"):
        call(out=out[:1])
    with pytest.raises(ValueError, match="lse"):
        call(lse=torch.zeros(3))
    with pytest.raises(ValueError, match="sinks"):
        call(sinks=torch.zeros(3))
    with pytest.raises(ValueError, match="handle"):
        k.fp4_attention(q, cache, nb, bs, table, lens, 0.1, out, stream=7)
    with pytest.raises(ValueError, match="weights"):
        k.fp4_attention_weights(q, cache, nb, bs, table, lens, 0.1, torch.zeros(B, 1, 4),
                                torch.zeros(B * 32))
    kept, w = torch.zeros(B, 8, dtype=torch.int32), torch.zeros(B, 32)
    with pytest.raises(ValueError, match="kept"):
        k.fp4_evict(cache, nb, bs, table, lens, w, 7, 2, table, kept, lens, torch.zeros(B, 7))
    with pytest.raises(ValueError, match="kv_cache"):
        k.fp4_dequant_gather(cache[:-1], nb, bs, torch.zeros(2, dtype=torch.int64),
                             torch.zeros(2, 512, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="kv_cache"):
        k.qnorm_rope_kv_fp4_insert(None, torch.zeros(2, 512, dtype=torch.bfloat16),
                                   torch.zeros(512, dtype=torch.bfloat16),
                                   torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64),
                                   torch.zeros(2, dtype=torch.int64), cache[:-1], nb, bs, 1e-6)


def test_no_cpu_fallback_without_a_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    assert _insert() == _gather() == _attention() == _weights() == _evict() == k.ERR_CUDA
