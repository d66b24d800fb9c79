"""kv_norm_rope_gb300: Python binding of libdsv4kv, the GB300 (sm_103a) library for the
fused DeepSeek-V4 attention-input step (q RMSNorm + RoPE in place; KV RMSNorm with a
weight + RoPE + UE8M0/E4M3 quantisation + paged-cache insert).

Argument marshalling only: every step runs in the CUDA kernels of ``csrc/``, reached
through the C ABI declared in ``include/dsv4kv.h``.  There is no CPU fallback: if the
shared library is missing and cannot be built, importing the entry points raises.
PyTorch supplies device memory and the current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
_CSRC = os.path.join(_HERE, "csrc")
_INCLUDE = os.path.join(_ROOT, "include")
LIB_PATH = os.path.join(_HERE, "libdsv4kv.so")
# the same sources with every global access tested against its buffer (DSV4_CHECK_BOUNDS)
CHECKED_LIB_PATH = os.path.join(_HERE, "libdsv4kv_checked.so")
_SOURCES = ["qnorm_rope_kv_insert.cu", "dequant_gather.cu",
            "gemma_rmsnorm_mxfp8.cu", "indexer_k.cu", "kv_rows.cu", "qnorm_rope_kv_insert_half.cu",
            "wait_check.cu", "fp4_gather.cu", "fp4_attention.cu", "fp4_weights.cu",
            "fp4_evict.cu", "latent_attention.cu", "tree_keep.cu", "rope_table.cu", "rope_rows.cu",
            "api.cpp", "fp4_api.cpp", "latent_api.cpp", "rope_api.cpp"]
_HEADERS = [os.path.join(_INCLUDE, "dsv4kv.h")] + [
    os.path.join(_CSRC, h)
    for h in ("launch.h", "ops.h", "fastdiv.h", "convert.cuh", "launch_status.h", "rowmath.cuh",
              "halfrow.cuh", "bulkcopy.cuh", "bounds.cuh", "bounds_range.h", "fp4.cuh",
              "fp4_tiles.cuh", "fp8_rows.cuh", "key_tiles.cuh", "run_join.cuh", "tcgen05.cuh", "tensor_copy.cuh", "hostcheck.h")]
NVCC_ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]

# status codes and constants (mirrors include/dsv4kv.h)
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_VALUE, ERR_CUDA = range(6)
DEVERR_SLOT_RANGE, DEVERR_POS_RANGE, DEVERR_TIMEOUT, DEVERR_BOUNDS = 1, 2, 4, 8
STORE_FP8, STORE_BF16, STORE_FP4, STORE_INDEXER = range(4)
VARIANT_AUTO, VARIANT_SMALL, VARIANT_STREAM, VARIANT_HALF = 0, 1, 2, 4
FP8_SLOT_BYTES, BF16_SLOT_BYTES, FP4_SLOT_BYTES, INDEXER_SLOT_BYTES = 584, 1024, 368, 132
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = range(4)  # scalings of the frequencies
ROPE_PAIRS, ROPE_HALF = range(2)                         # layouts of the rotated dims

EXPORTS = ("dsv4_qnorm_rope_kv_quant_insert", "dsv4_qnorm_rope_kv_bf16_insert",
           "dsv4_qnorm_rope_kv_insert_variant", "dsv4_qnorm_rope_kv_rope_quant_insert",
           "dsv4_kv_norm_rope_insert", "dsv4_insert_ex", "dsv4_dequant_gather",
           "dsv4_add_gemma_rmsnorm_mxfp8", "dsv4_mxfp8_scale_bytes", "dsv4_launch_plan",
           "dsv4_fp8_cache_bytes", "dsv4_bf16_cache_bytes", "dsv4_indexer_k_quant_insert",
           "dsv4_indexer_k_gather", "dsv4_indexer_cache_bytes", "dsv4_check_bounded_wait",
           "dsv4_debug_bounds_flags", "dsv4_status_string", "dsv4_fp4_cache_bytes",
           "dsv4_qnorm_rope_kv_fp4_insert", "dsv4_fp4_dequant_gather",
           "dsv4_fp4_attention_workspace_bytes", "dsv4_fp4_attention",
           "dsv4_fp4_attention_weights", "dsv4_fp4_evict",
           "dsv4_latent_attention_workspace_bytes", "dsv4_latent_attention", "dsv4_tree_keep",
           "dsv4_rope_frequencies", "dsv4_rope_table", "dsv4_rope_rows")


class Dsv4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(path: str) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    deps = [os.path.join(_CSRC, s) for s in _SOURCES] + _HEADERS
    return any(os.path.getmtime(d) > t for d in deps)


def _build_one(path: str, extra: list, verbose: bool) -> str:
    bdir = tempfile.mkdtemp(prefix="dsv4kv_build_", dir=_HERE)
    flags = NVCC_ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                         "-I", _INCLUDE, "-I", _CSRC] + extra
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        subprocess.run([_nvcc()] + flags + ["-c", os.path.join(_CSRC, src), "-o", obj], check=True)
        return obj

    with ThreadPoolExecutor(len(_SOURCES)) as ex:
        objs = list(ex.map(compile_one, _SOURCES))
    tmp = os.path.join(bdir, os.path.basename(path))
    subprocess.run([_nvcc()] + NVCC_ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs,
                   check=True)
    os.replace(tmp, path)
    for f in objs:
        os.remove(f)
    os.rmdir(bdir)
    return path


def build(force: bool = False, verbose: bool = False, checked: bool | None = None) -> str:
    """Compile csrc/ for sm_103a with nvcc into libdsv4kv.so and its checked twin
    libdsv4kv_checked.so (DSV4_CHECK_BOUNDS: every global access tested against its
    buffer), both in-tree.  checked=False builds the release library only, True the
    checked one only.  Translation units compile in parallel and link the static CUDA
    runtime, so the libraries need only the driver at run time.  Returns the path of
    the release library (of the checked one for checked=True)."""
    jobs = []
    if checked is not True and (force or _stale(LIB_PATH)):
        jobs.append((LIB_PATH, []))
    if checked is not False and (force or _stale(CHECKED_LIB_PATH)):
        jobs.append((CHECKED_LIB_PATH, ["-DDSV4_CHECK_BOUNDS"]))
    with ThreadPoolExecutor(max(1, len(jobs))) as ex:
        list(ex.map(lambda j: _build_one(j[0], j[1], verbose), jobs))
    return CHECKED_LIB_PATH if checked else LIB_PATH


_lib = None


def lib():
    """The loaded libdsv4kv (built first if missing or older than its sources).  With
    DSV4KV_CHECKED=1 in the environment this is the checked build instead."""
    global _lib
    if _lib is None:
        checked = os.environ.get("DSV4KV_CHECKED", "") == "1"
        _lib = _load(build(checked=checked))
    return _lib


@contextlib.contextmanager
def checked_build():
    """Route every call made in the block through libdsv4kv_checked.so, whose kernels
    test each global access against its buffer (see dsv4_debug_bounds_flags)."""
    global _lib
    saved = lib()
    _lib = _load(build(checked=True))
    try:
        yield _lib
    finally:
        _lib = saved


def debug_bounds_flags(reset: bool = True) -> int:
    """dsv4_debug_bounds_flags of the loaded library: 0 or DEVERR_BOUNDS (checked
    build), -1 (release build)."""
    return int(lib().dsv4_debug_bounds_flags(1 if reset else 0))


def _load(path: str):
    """Open a built library and declare its entry points' argument types."""
    L = ctypes.CDLL(path)
    vp, i64, i32, f32, c_int = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                ctypes.c_float, ctypes.c_int)
    common = [vp, vp, vp, vp, vp, i64, vp, vp, i64, i32, i64, i32, f32, vp, vp]
    L.dsv4_qnorm_rope_kv_quant_insert.argtypes = common
    L.dsv4_qnorm_rope_kv_quant_insert.restype = c_int
    L.dsv4_qnorm_rope_kv_bf16_insert.argtypes = common
    L.dsv4_qnorm_rope_kv_bf16_insert.restype = c_int
    L.dsv4_qnorm_rope_kv_insert_variant.argtypes = [c_int, c_int] + common
    L.dsv4_qnorm_rope_kv_insert_variant.restype = c_int
    L.dsv4_insert_ex.argtypes = [c_int, c_int, c_int] + common
    L.dsv4_insert_ex.restype = c_int
    L.dsv4_qnorm_rope_kv_rope_quant_insert.argtypes = [vp, vp, vp, vp, i64, vp, vp, i64, i32,
                                                       i64, i32, f32, vp, vp]
    L.dsv4_qnorm_rope_kv_rope_quant_insert.restype = c_int
    L.dsv4_kv_norm_rope_insert.argtypes = [c_int, vp, vp, vp, vp, i64, vp, vp, i64, i32, i64,
                                           f32, vp, vp]
    L.dsv4_kv_norm_rope_insert.restype = c_int
    L.dsv4_dequant_gather.argtypes = [vp, i64, i32, vp, i64, vp, vp, vp]
    L.dsv4_dequant_gather.restype = c_int
    L.dsv4_add_gemma_rmsnorm_mxfp8.argtypes = [vp, vp, vp, i64, i32, f32, vp, vp, vp, vp]
    L.dsv4_add_gemma_rmsnorm_mxfp8.restype = c_int
    L.dsv4_mxfp8_scale_bytes.argtypes = [i64, i32]
    L.dsv4_mxfp8_scale_bytes.restype = ctypes.c_size_t
    L.dsv4_launch_plan.argtypes = [i64, i32, i32, i32, i32, ctypes.POINTER(Plan)]
    L.dsv4_launch_plan.restype = c_int
    L.dsv4_fp8_cache_bytes.argtypes = [i64, i32]
    L.dsv4_fp8_cache_bytes.restype = ctypes.c_size_t
    L.dsv4_bf16_cache_bytes.argtypes = [i64, i32]
    L.dsv4_bf16_cache_bytes.restype = ctypes.c_size_t
    L.dsv4_indexer_k_quant_insert.argtypes = [vp, vp, vp, i64, i32, i64, vp, vp]
    L.dsv4_indexer_k_quant_insert.restype = c_int
    L.dsv4_indexer_k_gather.argtypes = [vp, i64, i32, vp, i64, vp, vp, vp, vp]
    L.dsv4_indexer_k_gather.restype = c_int
    L.dsv4_indexer_cache_bytes.argtypes = [i64, i32]
    L.dsv4_indexer_cache_bytes.restype = ctypes.c_size_t
    L.dsv4_fp4_cache_bytes.argtypes = [i64, i32]
    L.dsv4_fp4_cache_bytes.restype = ctypes.c_size_t
    L.dsv4_qnorm_rope_kv_fp4_insert.argtypes = common
    L.dsv4_qnorm_rope_kv_fp4_insert.restype = c_int
    L.dsv4_fp4_dequant_gather.argtypes = [vp, i64, i32, vp, i64, vp, vp, vp]
    L.dsv4_fp4_dequant_gather.restype = c_int
    L.dsv4_fp4_attention_workspace_bytes.argtypes = []
    L.dsv4_fp4_attention_workspace_bytes.restype = ctypes.c_size_t
    batch = [vp, i64, i32, vp, i64, i32, vp, i32]  # cache, its sizes, the table, lens, batch
    L.dsv4_fp4_attention.argtypes = ([vp] + batch + [i32, i32, f32, i32, vp, vp, vp, vp,
                                                     ctypes.c_size_t, vp, vp])
    L.dsv4_fp4_attention.restype = c_int
    L.dsv4_fp4_attention_weights.argtypes = ([vp] + batch + [i32, i32, f32, i32, vp, vp, i64, i32,
                                                             vp, vp])
    L.dsv4_fp4_attention_weights.restype = c_int
    L.dsv4_fp4_evict.argtypes = batch + [vp, i64, i32, i32, i32, vp, i64, i32, vp, vp, vp, vp, vp]
    L.dsv4_fp4_evict.restype = c_int
    L.dsv4_latent_attention_workspace_bytes.argtypes = []
    L.dsv4_latent_attention_workspace_bytes.restype = ctypes.c_size_t
    L.dsv4_latent_attention.argtypes = ([c_int, vp] + batch + [i32, i32, f32, i32, vp, vp, vp, vp, vp,
                                                               ctypes.c_size_t, vp, vp])
    L.dsv4_latent_attention.restype = c_int
    L.dsv4_tree_keep.argtypes = [c_int] + batch + [i32, vp, vp, vp, vp, vp]
    L.dsv4_tree_keep.restype = c_int
    f64, doubles = ctypes.c_double, ctypes.POINTER(ctypes.c_double)
    L.dsv4_rope_frequencies.argtypes = [c_int, i32, f64, f64, f64, f64, f64, doubles]
    L.dsv4_rope_frequencies.restype = c_int
    L.dsv4_rope_table.argtypes = [doubles, i32, f64, vp, i64, i64, vp, vp, vp]
    L.dsv4_rope_table.restype = c_int
    L.dsv4_rope_rows.argtypes = [c_int, vp, i64, i64, vp, i64, i64, i64, i32, i32, i32, i32, c_int,
                                 c_int, vp, vp, i64, vp, vp]
    L.dsv4_rope_rows.restype = c_int
    L.dsv4_check_bounded_wait.argtypes = [i64, vp, vp]
    L.dsv4_check_bounded_wait.restype = c_int
    L.dsv4_debug_bounds_flags.argtypes = [c_int]
    L.dsv4_debug_bounds_flags.restype = c_int
    L.dsv4_status_string.argtypes = [c_int]
    L.dsv4_status_string.restype = ctypes.c_char_p
    return L


class Plan(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("threads", ctypes.c_int32), ("ctas", ctypes.c_int64),
                ("rows_per_warp", ctypes.c_int32), ("rows", ctypes.c_int64)]


def status_string(status: int) -> str:
    return lib().dsv4_status_string(status).decode()


def launch_plan(num_tokens: int, num_heads: int, sm_count: int, ctas_per_sm: int,
                variant: int = VARIANT_AUTO) -> Plan:
    plan = Plan()
    st = lib().dsv4_launch_plan(num_tokens, num_heads, sm_count, ctas_per_sm, variant,
                                ctypes.byref(plan))
    if st != OK:
        raise Dsv4Error(st, "dsv4_launch_plan")
    return plan


def fp8_cache_bytes(num_blocks: int, block_size: int) -> int:
    return int(lib().dsv4_fp8_cache_bytes(num_blocks, block_size))


def bf16_cache_bytes(num_blocks: int, block_size: int) -> int:
    return int(lib().dsv4_bf16_cache_bytes(num_blocks, block_size))


def _ptr(t) -> int | None:
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _stream_handle(stream) -> int | None:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # no Stream object is made
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_kinds_table = None


def _kinds():
    global _kinds_table
    if _kinds_table is None:
        import torch
        two_byte = (torch.bfloat16, torch.int16) + ((torch.uint16,) if hasattr(torch, "uint16") else ())
        _kinds_table = {"bf16": two_byte, "i64": (torch.int64,), "f32": (torch.float32,),
                        "u8": (torch.uint8, torch.int8), "i32": (torch.int32,), "bytes": None}
    return _kinds_table


def _check(name: str, t, kind: str, numel: int | None = None, min_bytes: int | None = None):
    """Reject a tensor argument the C ABI cannot check: wrong element type (bf16 data
    may come as any 2-byte dtype), not contiguous, or the wrong number of elements /
    too few bytes.  Raw integer pointers pass unchecked; _on_cuda checks devices."""
    if t is None or isinstance(t, int):
        return
    allowed = (_kinds_table or _kinds())[kind]
    if allowed is not None and t.dtype not in allowed:
        raise TypeError(f"{name}: expected {kind} data, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
    if min_bytes is not None and t.numel() * t.element_size() < min_bytes:
        raise ValueError(f"{name}: needs at least {min_bytes} bytes, has "
                         f"{t.numel() * t.element_size()}")


def _on_cuda(**tensors):
    """Every tensor argument lives on one CUDA device: there is no CPU path."""
    first, several = None, False
    for name, t in tensors.items():
        if t is None or isinstance(t, int):
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
        index = t.get_device()
        several = several or first is not None and index != first
        first = index
    if several:
        devices = {str(t.device) for t in tensors.values() if t is not None and not isinstance(t, int)}
        raise ValueError(f"tensor arguments on several devices: {sorted(devices)}")


def _check_step(store_mode, q, kv, w, positions, cos_sin_cache, slot_mapping, kv_cache,
                num_blocks, block_size, device_error, T, H):
    _check("positions", positions, "i64", T)
    _check("slot_mapping", slot_mapping, "i64", T)
    _check("q", q, "bf16", T * H * 512)
    _check("kv", kv, "bf16", T * 512)
    _check("kv_norm_weight", w, "bf16", 512)
    _check("cos_sin_cache", cos_sin_cache, "f32")
    if not isinstance(cos_sin_cache, int) and cos_sin_cache.numel() % 64:
        raise ValueError("cos_sin_cache must hold rows of 64 fp32 (32 cos, 32 sin)")
    need = {STORE_FP8: fp8_cache_bytes, STORE_FP4: fp4_cache_bytes}.get(
        store_mode, bf16_cache_bytes)(num_blocks, block_size)
    _check("kv_cache", kv_cache, "bytes", min_bytes=need)
    _check("device_error", device_error, "i32")
    _on_cuda(q=q, kv=kv, kv_norm_weight=w, positions=positions, cos_sin_cache=cos_sin_cache,
             slot_mapping=slot_mapping, kv_cache=kv_cache, device_error=device_error)


def _shape_args(q, kv, positions, cos_sin_cache):
    T = int(positions.shape[0])
    if q is None:
        H = 0
    else:
        H = int(q.shape[-2]) if q.dim() == 3 else int(q.numel() // max(T, 1) // 512)
    return T, H, int(cos_sin_cache.shape[0])


def insert(store_mode: int, q, kv, kv_norm_weight, positions, cos_sin_cache, slot_mapping,
           kv_cache, num_blocks: int, block_size: int, eps: float, device_error=None,
           stream=None, variant: int = VARIANT_AUTO, num_heads: int | None = None,
           kv_norm: bool = True) -> None:
    """Enqueue the fused step on ``stream`` (default: torch's current stream).

    q: bf16 [T, H, 512] (rewritten in place; None for KV rows only); kv: bf16 [T, 512];
    kv_norm_weight: bf16 [512] (unused, may be None, when ``kv_norm`` is False: the KV
    rows then arrive normalised); positions, slot_mapping: int64 [T]; cos_sin_cache:
    fp32 [max_position, 64]; kv_cache: uint8 (FP8, num_blocks*block_size*584 bytes) or
    bf16 [num_blocks, block_size, 512]; device_error: optional int32 [1].  Raises
    Dsv4Error on a rejected call.  Goes through dsv4_insert_ex.
    """
    T, H, max_pos = _shape_args(q, kv, positions, cos_sin_cache)
    if num_heads is not None:
        H = num_heads
    _check_step(store_mode, q, kv, kv_norm_weight if kv_norm else None, positions, cos_sin_cache,
                slot_mapping, kv_cache, num_blocks, block_size, device_error, T, H)
    st = lib().dsv4_insert_ex(
        store_mode, variant, 1 if kv_norm else 0, _ptr(q), _ptr(kv), _ptr(kv_norm_weight),
        _ptr(positions), _ptr(cos_sin_cache), max_pos, _ptr(slot_mapping), _ptr(kv_cache),
        num_blocks, block_size, T, H, eps, _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_insert_ex")


def qnorm_rope_kv_rope_quant_insert(q, kv, positions, cos_sin_cache, slot_mapping, kv_cache,
                                    num_blocks, block_size, eps, device_error=None,
                                    stream=None) -> None:
    """dsv4_qnorm_rope_kv_rope_quant_insert: KV rows arrive normalised (rope + FP8 only)."""
    T, H, max_pos = _shape_args(q, kv, positions, cos_sin_cache)
    _check_step(STORE_FP8, q, kv, None, positions, cos_sin_cache, slot_mapping, kv_cache,
                num_blocks, block_size, device_error, T, H)
    st = lib().dsv4_qnorm_rope_kv_rope_quant_insert(
        _ptr(q), _ptr(kv), _ptr(positions), _ptr(cos_sin_cache), max_pos, _ptr(slot_mapping),
        _ptr(kv_cache), num_blocks, block_size, T, H, eps, _ptr(device_error),
        _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_qnorm_rope_kv_rope_quant_insert")


def kv_norm_rope_insert(store_mode: int, kv, kv_norm_weight, positions, cos_sin_cache,
                        slot_mapping, kv_cache, num_blocks, block_size, eps, device_error=None,
                        stream=None) -> None:
    """dsv4_kv_norm_rope_insert: KV rows only (norm with weight, rope, FP8 or bf16 store)."""
    T, _, max_pos = _shape_args(None, kv, positions, cos_sin_cache)
    _check_step(store_mode, None, kv, kv_norm_weight, positions, cos_sin_cache, slot_mapping,
                kv_cache, num_blocks, block_size, device_error, T, 0)
    st = lib().dsv4_kv_norm_rope_insert(
        store_mode, _ptr(kv), _ptr(kv_norm_weight), _ptr(positions), _ptr(cos_sin_cache),
        max_pos, _ptr(slot_mapping), _ptr(kv_cache), num_blocks, block_size, T, eps,
        _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_kv_norm_rope_insert")


def qnorm_rope_kv_quant_insert(q, kv, kv_norm_weight, positions, cos_sin_cache, slot_mapping,
                               kv_cache, num_blocks, block_size, eps, device_error=None,
                               stream=None) -> None:
    """dsv4_qnorm_rope_kv_quant_insert: FP8 (448 E4M3 + 7 UE8M0 + 64 bf16) cache rows."""
    T, H, max_pos = _shape_args(q, kv, positions, cos_sin_cache)
    _check_step(STORE_FP8, q, kv, kv_norm_weight, positions, cos_sin_cache, slot_mapping, kv_cache,
                num_blocks, block_size, device_error, T, H)
    st = lib().dsv4_qnorm_rope_kv_quant_insert(
        _ptr(q), _ptr(kv), _ptr(kv_norm_weight), _ptr(positions), _ptr(cos_sin_cache), max_pos,
        _ptr(slot_mapping), _ptr(kv_cache), num_blocks, block_size, T, H, eps,
        _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_qnorm_rope_kv_quant_insert")


def qnorm_rope_kv_bf16_insert(q, kv, kv_norm_weight, positions, cos_sin_cache, slot_mapping,
                              kv_cache, num_blocks, block_size, eps, device_error=None,
                              stream=None) -> None:
    """dsv4_qnorm_rope_kv_bf16_insert: 512 bf16 cache rows."""
    T, H, max_pos = _shape_args(q, kv, positions, cos_sin_cache)
    _check_step(STORE_BF16, q, kv, kv_norm_weight, positions, cos_sin_cache, slot_mapping,
                kv_cache, num_blocks, block_size, device_error, T, H)
    st = lib().dsv4_qnorm_rope_kv_bf16_insert(
        _ptr(q), _ptr(kv), _ptr(kv_norm_weight), _ptr(positions), _ptr(cos_sin_cache), max_pos,
        _ptr(slot_mapping), _ptr(kv_cache), num_blocks, block_size, T, H, eps,
        _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_qnorm_rope_kv_bf16_insert")


def dequant_gather(kv_cache, num_blocks: int, block_size: int, slots, out, device_error=None,
                   stream=None) -> None:
    """dsv4_dequant_gather: out (bf16 [n, 512]) = FP8 cache rows at ``slots`` read back."""
    n = int(slots.shape[0])
    _check("slots", slots, "i64", n)
    _check("kv_cache", kv_cache, "bytes", min_bytes=fp8_cache_bytes(num_blocks, block_size))
    _check("out", out, "bf16", n * 512)
    _check("device_error", device_error, "i32")
    _on_cuda(kv_cache=kv_cache, slots=slots, out=out, device_error=device_error)
    st = lib().dsv4_dequant_gather(_ptr(kv_cache), num_blocks, block_size, _ptr(slots),
                                   int(slots.shape[0]), _ptr(out), _ptr(device_error),
                                   _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_dequant_gather")


def check_bounded_wait(max_cycles: int = 0, device_error=None, stream=None) -> None:
    """dsv4_check_bounded_wait: one warp waits, through the bulk-copy kernels' bounded
    wait, on an mbarrier nothing completes; after max_cycles SM cycles (0: the kernels'
    own limit, about a second) it ORs DEVERR_TIMEOUT into device_error (int32 [1])."""
    if max_cycles < 0:
        raise ValueError("max_cycles must be >= 0")
    _check("device_error", device_error, "i32")
    _on_cuda(device_error=device_error)
    st = lib().dsv4_check_bounded_wait(int(max_cycles), _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_check_bounded_wait")


def indexer_cache_bytes(num_blocks: int, block_size: int) -> int:
    return int(lib().dsv4_indexer_cache_bytes(num_blocks, block_size))


def indexer_k_quant_insert(k, slot_mapping, indexer_cache, num_blocks: int, block_size: int,
                           device_error=None, stream=None) -> None:
    """dsv4_indexer_k_quant_insert: k (bf16 [T, 128]) quantised into the indexer cache
    (uint8, indexer_cache_bytes(num_blocks, block_size)) at slot_mapping (int64 [T])."""
    T = int(slot_mapping.shape[0])
    _check("slot_mapping", slot_mapping, "i64", T)
    _check("k", k, "bf16", T * 128)
    _check("indexer_cache", indexer_cache, "bytes",
           min_bytes=indexer_cache_bytes(num_blocks, block_size))
    _check("device_error", device_error, "i32")
    _on_cuda(k=k, slot_mapping=slot_mapping, indexer_cache=indexer_cache, device_error=device_error)
    st = lib().dsv4_indexer_k_quant_insert(_ptr(k), _ptr(slot_mapping), _ptr(indexer_cache),
                                           num_blocks, block_size, int(slot_mapping.shape[0]),
                                           _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_indexer_k_quant_insert")


def indexer_k_gather(indexer_cache, num_blocks: int, block_size: int, slots, k_out, scale_out,
                     device_error=None, stream=None) -> None:
    """dsv4_indexer_k_gather: k_out (uint8 [n, 128]) and scale_out (fp32 [n]) read from
    the indexer cache at ``slots`` (int64 [n])."""
    n = int(slots.shape[0])
    _check("slots", slots, "i64", n)
    _check("indexer_cache", indexer_cache, "bytes",
           min_bytes=indexer_cache_bytes(num_blocks, block_size))
    _check("k_out", k_out, "u8", n * 128)
    _check("scale_out", scale_out, "f32", n)
    _check("device_error", device_error, "i32")
    _on_cuda(indexer_cache=indexer_cache, slots=slots, k_out=k_out, scale_out=scale_out,
             device_error=device_error)
    st = lib().dsv4_indexer_k_gather(_ptr(indexer_cache), num_blocks, block_size, _ptr(slots),
                                     int(slots.shape[0]), _ptr(k_out), _ptr(scale_out),
                                     _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_indexer_k_gather")


def mxfp8_scale_bytes(num_rows: int, hidden: int) -> int:
    return int(lib().dsv4_mxfp8_scale_bytes(num_rows, hidden))


def add_gemma_rmsnorm_mxfp8(x, residual, gamma, eps: float, residual_out, codes, scales,
                            stream=None) -> None:
    """dsv4_add_gemma_rmsnorm_mxfp8: residual add + Gemma RMSNorm + MXFP8 rows.

    x, residual, residual_out: bf16 [m, n]; gamma: bf16 [n]; codes: uint8 [m, n];
    scales: uint8, mxfp8_scale_bytes(m, n) bytes."""
    m, n = int(x.shape[0]), int(x.shape[1])
    for name, t in (("x", x), ("residual", residual), ("residual_out", residual_out)):
        _check(name, t, "bf16", m * n)
    _check("gamma", gamma, "bf16", n)
    _check("codes", codes, "u8", m * n)
    _check("scales", scales, "u8", min_bytes=mxfp8_scale_bytes(m, n))
    _on_cuda(x=x, residual=residual, gamma=gamma, residual_out=residual_out, codes=codes,
             scales=scales)
    st = lib().dsv4_add_gemma_rmsnorm_mxfp8(_ptr(x), _ptr(residual), _ptr(gamma), m, n, eps,
                                            _ptr(residual_out), _ptr(codes), _ptr(scales),
                                            _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_add_gemma_rmsnorm_mxfp8")


# ---- the 4-bit cache


def fp4_cache_bytes(num_blocks: int, block_size: int) -> int:
    return num_blocks * block_size * FP4_SLOT_BYTES if num_blocks > 0 and block_size > 0 else 0


def qnorm_rope_kv_fp4_insert(q, kv, kv_norm_weight, positions, cos_sin_cache, slot_mapping,
                             kv_cache, num_blocks, block_size, eps, device_error=None,
                             stream=None) -> None:
    """dsv4_qnorm_rope_kv_fp4_insert: 4-bit (448 E2M1 + 14 UE8M0 + 64 bf16) cache rows;
    q may be None (KV rows only)."""
    T, H, max_pos = _shape_args(q, kv, positions, cos_sin_cache)
    _check_step(STORE_FP4, q, kv, kv_norm_weight, positions, cos_sin_cache, slot_mapping, kv_cache,
                num_blocks, block_size, device_error, T, H)
    st = lib().dsv4_qnorm_rope_kv_fp4_insert(
        _ptr(q), _ptr(kv), _ptr(kv_norm_weight), _ptr(positions), _ptr(cos_sin_cache), max_pos,
        _ptr(slot_mapping), _ptr(kv_cache), num_blocks, block_size, T, H, eps,
        _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_qnorm_rope_kv_fp4_insert")


def fp4_dequant_gather(kv_cache, num_blocks: int, block_size: int, slots, out, device_error=None,
                       stream=None) -> None:
    """dsv4_fp4_dequant_gather: out (bf16 [n, 512]) = 4-bit cache rows at ``slots`` read back."""
    n = int(slots.shape[0])
    _check("slots", slots, "i64", n)
    _check("kv_cache", kv_cache, "bytes", min_bytes=fp4_cache_bytes(num_blocks, block_size))
    _check("out", out, "bf16", n * 512)
    _check("device_error", device_error, "i32")
    _on_cuda(kv_cache=kv_cache, slots=slots, out=out, device_error=device_error)
    st = lib().dsv4_fp4_dequant_gather(_ptr(kv_cache), num_blocks, block_size, _ptr(slots), n,
                                       _ptr(out), _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_fp4_dequant_gather")


def _check_rows(name: str, t, kind: str, batch: int) -> tuple:
    """(stride, width) in elements of a 2-d tensor with one row per request, whose rows are
    contiguous and may be further apart than they are long."""
    if t.dtype not in _kinds()[kind]:
        raise TypeError(f"{name}: expected {kind} data, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != batch:
        raise ValueError(f"{name}: expected one row for each of {batch} requests, got "
                         f"{tuple(shape)}")
    (stride, inner), width = t.stride(), shape[1]
    if width > 1 and inner != 1 or batch > 1 and stride < width:
        raise ValueError(f"{name}: its rows must be contiguous and apart")
    return (stride if batch > 1 else width), width


def _check_attention(q, kv_cache, num_blocks, block_size, block_table, seq_lens):
    shape = q.shape
    if len(shape) != 4 or shape[3] != 512:
        raise ValueError(f"q: expected [batch, q_len, heads, 512], got {tuple(shape)}")
    B, Q, H, _ = shape
    _check("q", q, "bf16")
    _check("kv_cache", kv_cache, "bytes", min_bytes=fp4_cache_bytes(num_blocks, block_size))
    _check("seq_lens", seq_lens, "i32", B)
    return B, Q, H, _check_rows("block_table", block_table, "i32", B)


def _int32(n: int) -> int:
    """n in 32 bits, which ctypes would cut to its low ones: past the largest the largest
    (a window of all keys, a number past any limit), below 0 the -1 that is refused."""
    return max(-1, min(n, 2 ** 31 - 1))


_workspace_bytes = 0


def fp4_attention_workspace_bytes() -> int:
    global _workspace_bytes
    if _workspace_bytes == 0:
        _workspace_bytes = int(lib().dsv4_fp4_attention_workspace_bytes())
    return _workspace_bytes


def fp4_attention(q, kv_cache, num_blocks: int, block_size: int, block_table, seq_lens,
                  scale: float, out, lse=None, sinks=None, window: int = 0, workspace=None,
                  device_error=None, stream=None) -> None:
    """dsv4_fp4_attention: out (bf16 [B, Q, H, 512]) = attention of q (bf16, same shape)
    over the 4-bit rows of each request, key and value in one.

    block_table: int32 [B, W] (rows may be strided); seq_lens: int32 [B], the Q new tokens
    included; lse: optional fp32 [B, Q, H]; sinks: optional fp32 [H]; window: keys a token
    sees, 0 for all.  workspace: uint8 of fp4_attention_workspace_bytes(), or the address of
    that many; None takes one from torch's allocator for the call, on ``stream``, which is
    then torch's current one, or a torch stream."""
    B, Q, H, (stride, width) = _check_attention(q, kv_cache, num_blocks, block_size, block_table,
                                                seq_lens)
    _check("out", out, "bf16", q.numel())
    _check("lse", lse, "f32", B * Q * H)
    _check("sinks", sinks, "f32", H)
    _check("device_error", device_error, "i32")
    workspace_bytes = fp4_attention_workspace_bytes()
    if workspace is None:
        workspace = _workspace(workspace_bytes, q.device, stream)
    elif not isinstance(workspace, int):
        _check("workspace", workspace, "bytes")
        workspace_bytes = workspace.numel() * workspace.element_size()
    _on_cuda(q=q, kv_cache=kv_cache, block_table=block_table, seq_lens=seq_lens, out=out, lse=lse,
             sinks=sinks, workspace=workspace, device_error=device_error)
    st = lib().dsv4_fp4_attention(
        q.data_ptr(), _ptr(kv_cache), num_blocks, block_size, block_table.data_ptr(), stride, width,
        _ptr(seq_lens), B, Q, H, scale, _int32(window), _ptr(sinks), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace_bytes, _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_fp4_attention")


def _workspace(nbytes: int, device, stream):
    import torch
    if isinstance(stream, int):
        raise ValueError("workspace: pass one for a stream given by its handle")
    if device.type != "cuda":
        raise ValueError("q must be a CUDA tensor (there is no CPU path)")
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):  # the allocator gives it out again on this stream only
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def fp4_attention_weights(q, kv_cache, num_blocks: int, block_size: int, block_table, seq_lens,
                          scale: float, lse, weights, window: int = 0, device_error=None,
                          stream=None) -> None:
    """dsv4_fp4_attention_weights: weights (fp32 [B, n], rows may be strided) += the attention
    that each key of each request got from q, with the lse that fp4_attention returned."""
    B, Q, H, (stride, width) = _check_attention(q, kv_cache, num_blocks, block_size, block_table,
                                                seq_lens)
    _check("lse", lse, "f32", B * Q * H)
    w_stride, w_width = _check_rows("weights", weights, "f32", B)
    _check("device_error", device_error, "i32")
    _on_cuda(q=q, kv_cache=kv_cache, block_table=block_table, seq_lens=seq_lens, lse=lse,
             weights=weights, device_error=device_error)
    st = lib().dsv4_fp4_attention_weights(
        q.data_ptr(), _ptr(kv_cache), num_blocks, block_size, block_table.data_ptr(), stride, width,
        _ptr(seq_lens), B, Q, H, scale, _int32(window), _ptr(lse), weights.data_ptr(), w_stride, w_width,
        _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_fp4_attention_weights")


def fp4_evict(kv_cache, num_blocks: int, block_size: int, block_table, seq_lens, weights,
              budget: int, recent: int, new_block_table, kept, new_seq_lens, new_weights,
              device_error=None, stream=None) -> None:
    """dsv4_fp4_evict: each request keeps its last ``recent`` rows and the others of the
    highest weights (fp32 [B, n]), ``budget`` in all, moved in order to new_block_table
    (int32 [B, W]; blocks of the same cache that no request of the call reads).

    kept: int32 [B, budget], the rows' old indices, -1 after them; new_seq_lens: int32 [B]
    (may be seq_lens); new_weights: fp32 [B, budget]."""
    B = int(seq_lens.shape[0])
    _check("kv_cache", kv_cache, "bytes", min_bytes=fp4_cache_bytes(num_blocks, block_size))
    _check("seq_lens", seq_lens, "i32", B)
    stride, width = _check_rows("block_table", block_table, "i32", B)
    w_stride, w_width = _check_rows("weights", weights, "f32", B)
    n_stride, n_width = _check_rows("new_block_table", new_block_table, "i32", B)
    _check("kept", kept, "i32", B * budget)
    _check("new_seq_lens", new_seq_lens, "i32", B)
    _check("new_weights", new_weights, "f32", B * budget)
    _check("device_error", device_error, "i32")
    _on_cuda(kv_cache=kv_cache, block_table=block_table, seq_lens=seq_lens, weights=weights,
             new_block_table=new_block_table, kept=kept, new_seq_lens=new_seq_lens,
             new_weights=new_weights, device_error=device_error)
    st = lib().dsv4_fp4_evict(
        _ptr(kv_cache), num_blocks, block_size, block_table.data_ptr(), stride, width,
        _ptr(seq_lens), B, weights.data_ptr(), w_stride, w_width, budget, _int32(recent),
        new_block_table.data_ptr(), n_stride, n_width, _ptr(kept), _ptr(new_seq_lens),
        _ptr(new_weights), _ptr(device_error), _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, "dsv4_fp4_evict")


# ---- attention over the FP8 and bf16 caches, trees of drafted tokens

_latent_workspace_bytes = 0


def latent_attention_workspace_bytes() -> int:
    global _latent_workspace_bytes
    if _latent_workspace_bytes == 0:
        _latent_workspace_bytes = int(lib().dsv4_latent_attention_workspace_bytes())
    return _latent_workspace_bytes


def _placed(name: str, t, where: int) -> None:
    """Refuse a tensor that is not on the device with the index ``where`` (-1: the host)."""
    if t.get_device() != where:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
        raise ValueError(f"{name}: on {t.device}, other tensor arguments on "
                         f"{'the host' if where < 0 else f'cuda:{where}'}")


def _address(name: str, t, kind: str, numel: int | None, where: int) -> int | None:
    """The address of an argument: a tensor's, once it has passed _check and lies where the others do
    (the host is refused at the launch), or the address or None that it is."""
    if t is None or isinstance(t, int):
        return t
    allowed = (_kinds_table or _kinds())[kind]
    if allowed is not None and t.dtype not in allowed or not t.is_contiguous() or \
            numel is not None and t.numel() != numel:
        _check(name, t, kind, numel)
    if t.get_device() != where:
        _placed(name, t, where)
    return t.data_ptr()


_SLOT_BYTES = {STORE_FP8: FP8_SLOT_BYTES, STORE_BF16: BF16_SLOT_BYTES, STORE_FP4: FP4_SLOT_BYTES,
               STORE_INDEXER: INDEXER_SLOT_BYTES}


def _cache_address(t, store_mode: int, num_blocks: int, block_size: int, where: int) -> int | None:
    if t is not None and not isinstance(t, int) and num_blocks > 0 and block_size > 0:
        need = num_blocks * block_size * _SLOT_BYTES.get(store_mode, 0)
        if t.numel() * t.element_size() < need:
            _check("kv_cache", t, "bytes", min_bytes=need)
    return _address("kv_cache", t, "bytes", None, where)


def _launch(what: str, where: int, stream, entry, *args) -> None:
    """entry(*args, stream handle) on the device with this index, which need not be torch's current one."""
    import torch
    if where < 0:
        raise ValueError(f"{what}: tensor arguments must be CUDA tensors (there is no CPU path)")
    if stream is not None and not isinstance(stream, int) and stream.device.index != where:
        raise ValueError(f"stream: on {stream.device}, the tensors on cuda:{where}")
    current = torch.cuda.current_device()
    if where == current:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) if stream is None else None
        st = entry(*args, raw(current) if raw is not None else _stream_handle(stream))
    else:
        with torch.cuda.device(where):
            st = entry(*args, _stream_handle(stream))
    if st != OK:
        raise Dsv4Error(st, what)


def latent_attention(store_mode: int, q, kv_cache, num_blocks: int, block_size: int, block_table, seq_lens,
                     scale: float, out, lse=None, sinks=None, window: int = 0, tree=None, workspace=None,
                     device_error=None, stream=None) -> None:
    """dsv4_latent_attention: out (bf16 [B, Q, H, 512]) = attention of q (bf16, same shape) over
    the rows of each request in an FP8 (STORE_FP8) or bf16 (STORE_BF16) cache, key and value in one.

    block_table: int32 [B, W] (rows may be strided); seq_lens: int32 [B], the Q new tokens
    included; lse: optional fp32 [B, Q, H]; sinks: optional fp32 [H]; window: keys a token
    sees, 0 for all.  tree: int64 [B, Q], Q at most 64, for drafted tokens that form a tree instead of
    a chain: bit i of tree[b, j] says that token j sees drafted token i, its ancestors and itself; 0 for a
    token that is padding.  workspace: uint8 of latent_attention_workspace_bytes(), or the address
    of that many; None takes one from torch's allocator for the call, on ``stream``, which is
    then torch's current one, or a torch stream."""
    shape, where = q.shape, q.get_device()
    if len(shape) != 4 or shape[3] != 512:
        raise ValueError(f"q: expected [batch, q_len, heads, 512], got {tuple(shape)}")
    B, Q, H, _ = shape
    rows = B * Q * H
    q_at = _address("q", q, "bf16", None, where)
    cache_at = _cache_address(kv_cache, store_mode, num_blocks, block_size, where)
    lens_at = _address("seq_lens", seq_lens, "i32", B, where)
    stride, width = _check_rows("block_table", block_table, "i32", B)
    out_at = _address("out", out, "bf16", rows * 512, where)
    lse_at = _address("lse", lse, "f32", rows, where)
    sinks_at = _address("sinks", sinks, "f32", H, where)
    tree_at = _address("tree", tree, "i64", B * Q, where)
    error_at = _address("device_error", device_error, "i32", None, where)
    workspace_bytes = _latent_workspace_bytes or latent_attention_workspace_bytes()
    if workspace is None:
        workspace = _workspace(workspace_bytes, q.device, stream)
        workspace_at = workspace.data_ptr()
    else:
        if not isinstance(workspace, int):
            workspace_bytes = workspace.numel() * workspace.element_size()
        workspace_at = _address("workspace", workspace, "bytes", None, where)
    _placed("block_table", block_table, where)
    if out_at is not None and abs(q_at - out_at) < 1024 * rows:
        raise ValueError("out overlaps q")
    _launch("dsv4_latent_attention", where, stream, lib().dsv4_latent_attention,
            store_mode if store_mode in _SLOT_BYTES else -1, q_at, cache_at, num_blocks,
            block_size if 0 < block_size < 2 ** 31 else -1, block_table.data_ptr(), stride, width, lens_at, B, Q, H,
            scale, _int32(window), tree_at, sinks_at, out_at, lse_at, workspace_at, workspace_bytes, error_at)


def tree_keep(store_mode: int, kv_cache, num_blocks: int, block_size: int, block_table, seq_lens, path,
              path_lens, new_seq_lens, device_error=None, stream=None) -> None:
    """dsv4_tree_keep: of each request's last Q rows (the drafted tokens') those of the accepted
    path move together, in place: path (int32 [B, Q]) holds path_lens[b] of their indices, rising;
    new_seq_lens (int32 [B], may be seq_lens) = what is left.  store_mode: STORE_FP8, STORE_BF16,
    STORE_FP4 or STORE_INDEXER."""
    if path.dim() != 2:
        raise ValueError(f"path: expected [batch, q_len], got {tuple(path.shape)}")
    B, Q = path.shape
    where = path.get_device()
    cache_at = _cache_address(kv_cache, store_mode, num_blocks, block_size, where)
    lens_at = _address("seq_lens", seq_lens, "i32", B, where)
    stride, width = _check_rows("block_table", block_table, "i32", B)
    path_at = _address("path", path, "i32", None, where)
    path_lens_at = _address("path_lens", path_lens, "i32", B, where)
    new_at = _address("new_seq_lens", new_seq_lens, "i32", B, where)
    error_at = _address("device_error", device_error, "i32", None, where)
    _placed("block_table", block_table, where)
    _launch("dsv4_tree_keep", where, stream, lib().dsv4_tree_keep, store_mode if store_mode in _SLOT_BYTES else -1,
            cache_at, num_blocks, block_size if 0 < block_size < 2 ** 31 else -1, block_table.data_ptr(), stride, width,
            lens_at, B, Q, path_at, path_lens_at, new_at, error_at)


# ---- rotary positions


def rope_frequencies(rope_dim: int, theta: float = 10000.0, scaling: int = ROPE_PLAIN, factor: float = 1.0,
                     original_positions: float = 0.0, turns_fast: float = 32.0,
                     turns_slow: float = 1.0) -> tuple:
    """dsv4_rope_frequencies: the rope_dim / 2 angles per position (floats, on the host), plain or
    stretched for long contexts (ROPE_LINEAR, ROPE_NTK, ROPE_YARN)."""
    out = (ctypes.c_double * (max(2, min(rope_dim, 256)) // 2))()
    st = lib().dsv4_rope_frequencies(_int32(scaling), _int32(rope_dim), theta, factor, original_positions, turns_fast,
                                     turns_slow, out)
    if st != OK:
        raise Dsv4Error(st, "dsv4_rope_frequencies")
    return tuple(out)


def rope_table(frequencies, out, positions=None, first: int = 0, magnitude: float = 1.0, device_error=None,
               stream=None) -> None:
    """dsv4_rope_table: out (fp32 [n, 2 * len(frequencies)]) = magnitude times the cosines and sines
    of the angles of positions (int64 [n]), or of first, first + 1, ...: the cos_sin_cache that the
    inserts and rope_rows take."""
    pairs = len(frequencies)
    if out.dim() != 2 or out.shape[1] != 2 * pairs:
        raise ValueError(f"out: expected [n, {2 * pairs}], got {tuple(out.shape)}")
    where = out.get_device()
    out_at = _address("out", out, "f32", None, where)
    positions_at = _address("positions", positions, "i64", out.shape[0], where)
    error_at = _address("device_error", device_error, "i32", None, where)
    angles = (ctypes.c_double * pairs)(*frequencies)
    _launch("dsv4_rope_table", where, stream, lib().dsv4_rope_table, angles, 2 * pairs, magnitude, positions_at,
            first if 0 <= first < 2 ** 62 else -1, out.shape[0], out_at, error_at)


def _row_strides(name: str, t):
    strides = t.stride()
    if strides[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: its innermost stride must be 1")
    return strides[:2] if len(strides) == 3 else (strides[0], t.shape[1])


_row_types = None


def _find_row_types():
    global _row_types
    import torch
    _row_types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    return _row_types


def rope_rows(x, positions, cos_sin_cache, out=None, offset: int | None = None, inverse: bool = False,
              layout: int = ROPE_PAIRS, device_error=None, stream=None) -> None:
    """dsv4_rope_rows: dims [offset, offset + d) of x ([T, H, D] or [T, D]; bf16, fp16 or fp32; the
    outer dims may be strided) turned by the angles of each token's position into out (None: x
    itself), d being the width of cos_sin_cache (fp32 [max_position, d]) and offset D - d (the
    trailing dims) unless given.  inverse: the transpose, which is the gradient's way and, with a
    table of magnitude 1, turns back; what a table of magnitude m turned (rows, and an attention's output
    over such rows) is turned back with one of magnitude 1 / m.  layout: ROPE_PAIRS (neighbouring
    dims) or ROPE_HALF (i and i + d / 2)."""
    types = _row_types or _find_row_types()
    if out is None:
        out = x
    if x.dtype not in types:
        raise TypeError(f"x: expected bf16, fp16 or fp32 data, got {x.dtype}")
    if out.dtype != x.dtype:
        raise TypeError(f"out: expected {x.dtype} data, got {out.dtype}")
    shape, where = x.shape, x.get_device()
    if len(shape) not in (2, 3) or out.shape != shape:
        raise ValueError(f"x, out: expected [tokens, heads, width] of one shape, got {tuple(shape)} and "
                         f"{tuple(out.shape)}")
    if cos_sin_cache.dim() != 2:
        raise ValueError("cos_sin_cache: expected [max_position, d]")
    max_position, dim = cos_sin_cache.shape
    T, H, D = shape[0], (shape[1] if len(shape) == 3 else 1), shape[-1]
    positions_at = _address("positions", positions, "i64", T, where)
    table_at = _address("cos_sin_cache", cos_sin_cache, "f32", None, where)
    error_at = _address("device_error", device_error, "i32", None, where)
    _placed("out", out, where)
    offset = D - dim if offset is None else offset
    x_strides, out_strides = _row_strides("x", x), _row_strides("out", out)
    _launch("dsv4_rope_rows", where, stream, lib().dsv4_rope_rows, types[x.dtype], x.data_ptr(), *x_strides,
            out.data_ptr(), *out_strides, T, H, D, _int32(offset), dim, layout if layout in (ROPE_PAIRS, ROPE_HALF) else -1, 1 if inverse else 0, positions_at,
            table_at, max_position, error_at)
