"""ctypes binding of libq4.so with the C ABI's own names (include/q4.h).

Argument marshalling only: tensors become their data pointers, streams their
cudaStream_t handles, and a negative status becomes a Q4Error.  Every step of
the computation runs in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re

from . import build as _build

_lib = None

c_p = ctypes.c_void_p
c_int = ctypes.c_int
c_size = ctypes.c_size_t
c_i64 = ctypes.c_int64

Q4_OK = 0
Q4_ERR_ARG = -1
Q4_ERR_ALIGN = -2
Q4_ERR_CUDA = -3
Q4_ERR_TIMEOUT = -4
Q4_ERR_OOM = -5
Q4_ERR_DEVICE = -6

Q4_KERNEL_AUTO = 0
Q4_KERNEL_STREAM = 1
Q4_KERNEL_SIMPLE = 2
Q4_KERNEL_MMA = 3
Q4_KERNEL_TC = 4
Q4_KERNEL_ONESHOT = 5
Q4_GEMV_CHAIN = 0x100      # OR into q4_gemv_ex's kernel: a chained one-shot call

Q4_DEC_FUSED = 0
Q4_DEC_PER_LAYER = 1
Q4_DEC_TENSOR_CORE = 2
Q4_DEC_BARRIER = 4
Q4_DEC_CUDA_CORE = 8
Q4_DEC_BATCH_ENGINE = 16
Q4_KV_F16 = 0
Q4_KV_Q8 = 1
Q4_TYPE_F32 = 0
Q4_TYPE_F16 = 1
Q4_STREAM_POISON = 1
Q4_STREAM_TENSOR_CORE = 2
Q4_STREAM_CHUNKED = 4
Q4_STREAM_BARRIER = 8
Q4_STREAM_CUDA_CORE = 16
Q4_STREAM_SINGLE_BUFFER = 32
Q4_STREAM_TIMELINE = 64

WS_NAMES = ("control", "program", "qkv", "o", "gate", "up", "down", "act", "x", "attn", "x2", "t1", "t2", "flags", "xt", "vt", "actt")
WS_COUNT = len(WS_NAMES)


class Q4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = status_string(status) if _lib is not None else str(status)
        extra = ""
        if status == Q4_ERR_CUDA and _lib is not None:
            extra = f" (cudaError {_lib.q4_last_cuda_error()})"
        super().__init__(f"{what}: {msg}{extra}")


class LayerShape(ctypes.Structure):
    """q4_layer_shape."""
    _fields_ = [("hidden", c_int), ("q_dim", c_int), ("kv_dim", c_int), ("ffn", c_int),
                ("head_dim", c_int), ("eps", ctypes.c_float)]

    @classmethod
    def of(cls, hidden, q_dim, kv_dim, ffn, head_dim=128, eps=1e-5, **_):
        return cls(hidden, q_dim, kv_dim, ffn, head_dim, eps)


class KVCache(ctypes.Structure):
    """q4_kv_cache."""
    _fields_ = [("capacity", c_int), ("k_layers", ctypes.POINTER(c_p)), ("v_layers", ctypes.POINTER(c_p)),
                ("pos", c_p), ("attn_workspace", c_p), ("attn_workspace_bytes", c_size)]


class PagedKV(ctypes.Structure):
    """q4_paged_kv.  Made once per layer cache; keeps its tensors alive, which
    have to be of the cache's type and as large as it (or larger)."""
    _fields_ = [("k_pages", c_p), ("v_pages", c_p), ("k_scales", c_p), ("v_scales", c_p), ("n_pages", c_int),
                ("page_size", c_int), ("n_kv_heads", c_int), ("head_dim", c_int), ("type", c_int)]
    _at = None       # the device of its tensors

    @classmethod
    def of(cls, k_pages, v_pages, n_pages, page_size, n_kv_heads, head_dim, cache_type=Q4_KV_F16, k_scales=None,
           v_scales=None):
        n = n_pages * n_kv_heads * page_size * head_dim
        kinds = _CODES if cache_type == Q4_KV_Q8 else _BITS16
        scales = (_BITS16, n // 32) if cache_type == Q4_KV_Q8 else ()
        s = cls(_dev_ptr(k_pages, kinds, n), _dev_ptr(v_pages, kinds, n), _dev_ptr(k_scales, *scales),
                _dev_ptr(v_scales, *scales), n_pages, page_size, n_kv_heads, head_dim, cache_type)
        s._keep = (k_pages, v_pages, k_scales, v_scales)
        s._at = _device_of(*s._keep)
        return s


class PagedBatch(ctypes.Structure):
    """q4_paged_batch.  The kernels read the arrays, so one object serves every
    content of them; keeps its tensors alive, int32 of at least n_seqs + 1,
    n_seqs and n_seqs * table_width elements."""
    _fields_ = [("token_starts", c_p), ("kv_lens", c_p), ("page_table", c_p), ("n_seqs", c_int), ("n_tokens", c_int),
                ("table_width", c_int), ("max_new", c_int)]
    _at = None

    @classmethod
    def of(cls, token_starts, kv_lens, page_table, n_seqs, n_tokens, table_width, max_new):
        n = n_seqs if n_seqs > 0 else -1
        s = cls(_dev_ptr(token_starts, _INDEX, n + 1), _dev_ptr(kv_lens, _INDEX, n),
                _dev_ptr(page_table, _INDEX, n * table_width), n_seqs, n_tokens, table_width, max_new)
        if hasattr(page_table, "dim") and page_table.dim() == 2 and n > 1 and page_table.shape[1] != table_width:
            raise Q4Error(Q4_ERR_ARG, f"a page table of width {page_table.shape[1]}, not {table_width}")
        s._keep = (token_starts, kv_lens, page_table)
        s._at = _device_of(*s._keep)
        return s


def _declare(lib):
    sig = {
        "q4_status_string": ([c_int], ctypes.c_char_p),
        "q4_last_cuda_error": ([], c_int),
        "q4_version": ([], c_int),
        "q4_matrix_bytes": ([c_int, c_int], c_size),
        "q4_gemv": ([c_p, c_p, c_p, c_int, c_int, c_int, c_p], c_int),
        "q4_gemv_ex": ([c_p, c_p, c_p, c_int, c_int, c_int, c_int, c_p], c_int),
        "q4_device_status": ([], c_int),
        "q4_dequant_debug": ([c_p, c_p, c_int, c_int, c_p], c_int),
        "q4_layer_offsets": ([ctypes.POINTER(LayerShape), ctypes.POINTER(c_size), ctypes.POINTER(c_size)], c_int),
        "q4_workspace_layout": ([ctypes.POINTER(LayerShape), c_int, c_int, ctypes.POINTER(c_size),
                                 ctypes.POINTER(c_size)], c_int),
        "q4_decoder_create": ([ctypes.POINTER(c_p), ctypes.POINTER(LayerShape), ctypes.POINTER(c_p), c_int, c_int,
                               c_p, c_size, c_int, c_p], c_int),
        "q4_layer_decode": ([c_p, c_p, c_p], c_int),
        "q4_layer_decode_eager": ([c_p, c_p, c_p], c_int),
        "q4_decoder_status": ([c_p, c_p, ctypes.POINTER(c_int)], c_int),
        "q4_decoder_tagged": ([c_p, ctypes.POINTER(c_int)], c_int),
        "q4_decoder_debug_stall": ([c_p, ctypes.c_uint32, c_p, ctypes.POINTER(c_int)], c_int),
        "q4_decoder_destroy": ([c_p], c_int),
        "q4_decoder_create_kv": ([ctypes.POINTER(c_p), ctypes.POINTER(LayerShape), ctypes.POINTER(c_p), c_int,
                                  ctypes.POINTER(KVCache), c_p, c_size, c_p], c_int),
        "q4_layer_decode_noalloc": ([ctypes.POINTER(LayerShape), ctypes.POINTER(c_p), c_int, c_p, c_p], c_int),
        "q4_noalloc_scratch_bytes": ([], c_size),
        "q4_noalloc_status": ([c_p, ctypes.POINTER(c_int)], c_int),
        "q4_stream_create": ([ctypes.POINTER(c_p), ctypes.POINTER(LayerShape), ctypes.POINTER(c_p), c_int, c_int,
                              c_p, c_p, c_size, c_p, c_size, c_int], c_int),
        "q4_stream_create_ex": ([ctypes.POINTER(c_p), ctypes.POINTER(LayerShape), ctypes.POINTER(c_p),
                                 ctypes.POINTER(c_p), c_int, c_int, c_p, c_p, c_size, c_p, c_size, c_int], c_int),
        "q4_stream_layers": ([c_p, c_p, c_p, c_i64], c_int),
        "q4_attn_decode": ([c_p, c_p, c_p, c_p, c_int, c_int, c_int, c_int, c_p, c_p, c_size, c_p], c_int),
        "q4_attn_workspace_bytes": ([c_int, c_int, c_int, c_int], c_size),
        "q4_kv_append": ([c_p, c_p, c_p, c_p, c_p, c_int, c_int, c_p], c_int),
        "q4_paged_write": ([ctypes.POINTER(PagedKV), ctypes.POINTER(PagedBatch), c_p, c_p, c_int, c_i64, c_p], c_int),
        "q4_paged_read": ([ctypes.POINTER(PagedKV), ctypes.POINTER(PagedBatch), c_p, c_p, c_int, c_i64, c_p], c_int),
        "q4_attn_paged": ([ctypes.POINTER(PagedKV), ctypes.POINTER(PagedBatch), c_p, c_int, c_i64, c_int, c_int, c_int,
                           c_p, c_i64, c_p, c_size, c_p], c_int),
        "q4_attn_paged_workspace_bytes": ([c_int, c_int, c_int], c_size),
        "q4_stream_status": ([c_p, c_p, ctypes.POINTER(c_int)], c_int),
        "q4_stream_tagged": ([c_p, ctypes.POINTER(c_int)], c_int),
        "q4_stream_timeline": ([c_p, c_p, c_int, c_p], c_int),
        "q4_timeline_read": ([c_p, c_size, c_int], c_int),
        "q4_stream_destroy": ([c_p], c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


def lib():
    """The loaded libq4.so; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        path = _build.lib_path("libq4.so")
        if not os.path.exists(path):
            raise ImportError(f"libq4.so is not built ({path}); run weight_streaming_q4_gb300.build.build()")
        _lib = _declare(ctypes.CDLL(path))
    return _lib


def use_library(path: str):
    """Bind every call to another build of the library (the timeline build)."""
    global _lib
    _lib = _declare(ctypes.CDLL(path))
    return _lib


def header_functions() -> list:
    """Names of the functions include/q4.h declares."""
    text = open(os.path.join(_build.INCLUDE, "q4.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(q4_[a-z0-9_]+)\s*\(", text)))


# ------------------------------------------------------------------ marshalling

def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# The current CUDA device and its current stream's handle.  torch.cuda.current_stream()
# builds an object per call (2.9 us on a Grace core, a launch takes 2); after a
# first call of it, which initialises CUDA, the handle is asked for directly
# where this torch has the functions.
_device = None
_raw_stream = None
_stream_of = None       # the current stream's handle of a device, where torch gives it


def _init_current():
    global _device, _raw_stream, _stream_of
    import torch
    torch.cuda.current_stream()
    get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    _device = dev or torch.cuda.current_device
    _stream_of = get
    _raw_stream = (lambda: get(dev())) if get and dev else (lambda: torch.cuda.current_stream().cuda_stream)


def _current_device() -> int:
    """The current CUDA device; -2, where no tensor is, without one."""
    if _device is None:
        import torch
        if not torch.cuda.is_available():
            return -2
        _init_current()
    return _device()


# Tensor types that hold binary16 values (or their bits), and Q8 codes.
_BITS16 = ("torch.float16", "torch.int16", "torch.uint16")
_CODES = ("torch.int8", "torch.uint8")
_INDEX = ("torch.int32",)
_F32 = ("torch.float32",)


def _dev_ptr(t, kinds=None, n=0):
    """_ptr of a tensor that the kernels can reach: contiguous, on the current
    CUDA device, of one of the given types and at least n elements (an integer
    is taken as an address)."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != _current_device():
        raise Q4Error(Q4_ERR_ARG, f"a tensor on {t.device}, not the current CUDA device")
    if not t.is_contiguous() or (kinds and str(t.dtype) not in kinds):
        raise Q4Error(Q4_ERR_ARG, f"a {t.dtype} tensor of strides {tuple(t.stride())}")
    if t.numel() < n:
        raise Q4Error(Q4_ERR_ARG, f"a tensor of {t.numel()} elements where {n} are meant")
    return t.data_ptr()


def _device_of(*tensors):
    """The device of the tensors among the arguments, all of it the current one when they were taken (None: addresses)."""
    for t in tensors:
        if t is not None and not isinstance(t, int):
            return t.get_device()
    return None


def _device_for(what, kv, batch) -> int:
    """The current device, where the kernels will run: the descriptors have to have been made there."""
    dev = _device() if _device else _current_device()
    a, b = kv._at, batch._at
    if a is not None and a != dev or b is not None and b != dev:
        raise Q4Error(Q4_ERR_ARG, f"{what}: tensors on another device than the current one, {dev}")
    return dev


def _bytes_ptr(t, n, dev):
    """_ptr of a workspace of n bytes, contiguous and on the device."""
    if t is None or isinstance(t, int):
        return t
    if t.nbytes < n or t.get_device() != dev or not t.is_contiguous():
        raise Q4Error(Q4_ERR_ARG, f"workspace: a tensor of {t.nbytes} bytes and strides {tuple(t.stride())} on {t.device}, where {n} bytes are meant")
    return t.data_ptr()


_plain = {}      # torch's type of each Q4_TYPE_*


def _find_plain():
    import torch
    _plain.update({Q4_TYPE_F32: torch.float32, Q4_TYPE_F16: torch.float16})
    return _plain


def _rows_ptr(t, what, rows, row, ld, kind, dev):
    """_ptr of a buffer of ``rows`` rows of ``row`` values, ``ld`` apart: a
    tensor has to be on the device, of that type, and hold them (a view that
    starts inside a wider row does: its storage counts).  Its own rows have to
    be ld apart; a contiguous tensor of another number of rows is memory."""
    if t is None or isinstance(t, int):
        return t
    # (a matrix that holds the rows itself: the rest costs as much as a launch)
    if (t.dtype is (_plain or _find_plain()).get(kind) and t.stride() == (ld, 1) and t.size(0) >= rows
            and t.size(1) >= row and t.get_device() == dev):
        return t.data_ptr()
    size = 4 if kind == Q4_TYPE_F32 else 2
    if t.get_device() != dev:
        raise Q4Error(Q4_ERR_ARG, f"{what}: a tensor on {t.device}, not the current CUDA device")
    if str(t.dtype) not in (_F32 if kind == Q4_TYPE_F32 else _BITS16):
        raise Q4Error(Q4_ERR_ARG, f"{what}: a {t.dtype} tensor for {'fp32' if size == 4 else 'binary16'} values")
    # its rows (the first dimension, or all of it) lie ld values apart, each in one piece
    n = t.dim()
    apart = rows <= 1 or n < 2 or t.stride(0) == ld
    if t.is_contiguous():
        apart = apart or t.size(0) != rows
    else:
        apart = apart and (t.stride(1) == 1 if n == 2 else n > 2 and t[0].is_contiguous())
    if not apart:
        raise Q4Error(Q4_ERR_ARG, f"{what}: a tensor of shape {tuple(t.shape)} and strides {tuple(t.stride())} for rows {ld} apart")
    if rows > 0 and t.storage_offset() + (rows - 1) * ld + row > t.untyped_storage().nbytes() // size:
        raise Q4Error(Q4_ERR_ARG, f"{what}: {rows} rows of {row} values {ld} apart do not fit its storage")
    return t.data_ptr()


def _stream(s):
    if s is None:
        if _raw_stream is None:
            _init_current()
        return _raw_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _stream_on(s, dev):
    """_stream, with the current device known."""
    return _stream_of(dev) if s is None and _stream_of else _stream(s)


def _check(st: int, what: str):
    if st < 0:
        raise Q4Error(st, what)
    return st


def status_string(st: int) -> str:
    return lib().q4_status_string(st).decode()


def q4_last_cuda_error() -> int:
    return lib().q4_last_cuda_error()


def q4_version() -> int:
    return lib().q4_version()


def q4_matrix_bytes(n: int, k: int) -> int:
    return lib().q4_matrix_bytes(n, k)


def q4_gemv(w, x, y, n: int, k: int, batch: int = 1, stream=None, chain: bool = False):
    if chain:   # Q4_GEMV_CHAIN: may overlap the product before it on the stream
        _check(lib().q4_gemv_ex(_ptr(w), _ptr(x), _ptr(y), n, k, batch, Q4_KERNEL_AUTO | Q4_GEMV_CHAIN,
                                _stream(stream)), "q4_gemv_ex")
        return
    _check(lib().q4_gemv(_ptr(w), _ptr(x), _ptr(y), n, k, batch, _stream(stream)), "q4_gemv")


def q4_gemv_ex(w, x, y, n: int, k: int, batch: int, kernel: int, stream=None):
    _check(lib().q4_gemv_ex(_ptr(w), _ptr(x), _ptr(y), n, k, batch, kernel, _stream(stream)), "q4_gemv_ex")


def q4_device_status() -> int:
    return _check(lib().q4_device_status(), "q4_device_status")


def q4_dequant_debug(w, out, n: int, k: int, stream=None):
    _check(lib().q4_dequant_debug(_ptr(w), _ptr(out), n, k, _stream(stream)), "q4_dequant_debug")


def q4_layer_offsets(shape: LayerShape):
    offs = (c_size * 7)()
    total = c_size(0)
    _check(lib().q4_layer_offsets(ctypes.byref(shape), offs, ctypes.byref(total)), "q4_layer_offsets")
    return list(offs), total.value


def q4_workspace_layout(shape: LayerShape, n_layers: int, batch: int):
    offs = (c_size * WS_COUNT)()
    total = c_size(0)
    _check(lib().q4_workspace_layout(ctypes.byref(shape), n_layers, batch, offs, ctypes.byref(total)),
           "q4_workspace_layout")
    return dict(zip(WS_NAMES, list(offs))), total.value


def q4_decoder_create_kv(shape: LayerShape, layer_ptrs, capacity: int, k_layers, v_layers, pos, attn_workspace,
                         attn_workspace_bytes: int, workspace, workspace_bytes: int, stream=None):
    """Batch-1 decoder with decode attention over per-layer KV caches (device
    pointers or tensors; ``pos`` a device int32)."""
    h = c_p()
    arr = (c_p * len(layer_ptrs))(*[int(p) for p in layer_ptrs])
    ks = (c_p * len(k_layers))(*[_ptr(t) for t in k_layers])
    vs = (c_p * len(v_layers))(*[_ptr(t) for t in v_layers])
    kv = KVCache(capacity, ks, vs, _ptr(pos), _ptr(attn_workspace), attn_workspace_bytes)
    kv._keep = (ks, vs)
    _check(lib().q4_decoder_create_kv(ctypes.byref(h), ctypes.byref(shape), arr, len(layer_ptrs), ctypes.byref(kv),
                                      _ptr(workspace), workspace_bytes, _stream(stream)), "q4_decoder_create_kv")
    return h


def q4_decoder_create(shape: LayerShape, layer_ptrs, batch: int, workspace, workspace_bytes: int,
                      mode: int = Q4_DEC_FUSED, stream=None):
    h = c_p()
    arr = (c_p * len(layer_ptrs))(*[int(p) for p in layer_ptrs])
    _check(lib().q4_decoder_create(ctypes.byref(h), ctypes.byref(shape), arr, len(layer_ptrs), batch,
                                   _ptr(workspace), workspace_bytes, mode, _stream(stream)), "q4_decoder_create")
    return h


def q4_layer_decode(dec, hidden, stream=None):
    _check(lib().q4_layer_decode(dec, _ptr(hidden), _stream(stream)), "q4_layer_decode")


def q4_layer_decode_eager(dec, hidden, stream=None):
    _check(lib().q4_layer_decode_eager(dec, _ptr(hidden), _stream(stream)), "q4_layer_decode_eager")


def q4_decoder_status(dec, stream=None) -> int:
    v = c_int(0)
    _check(lib().q4_decoder_status(dec, _stream(stream), ctypes.byref(v)), "q4_decoder_status")
    return v.value


def q4_decoder_tagged(dec) -> bool:
    v = c_int(0)
    _check(lib().q4_decoder_tagged(dec, ctypes.byref(v)), "q4_decoder_tagged")
    return bool(v.value)


def q4_decoder_debug_stall(dec, wait_limit, stream=None) -> int:
    v = c_int(0)
    _check(lib().q4_decoder_debug_stall(dec, wait_limit, _stream(stream), ctypes.byref(v)), "q4_decoder_debug_stall")
    return v.value


def q4_decoder_destroy(dec):
    _check(lib().q4_decoder_destroy(dec), "q4_decoder_destroy")


def q4_layer_decode_noalloc(shape: LayerShape, layer_ptrs, hidden, stream=None):
    """The decoder stack with its scratch in the library's static device array (no allocation)."""
    arr = (c_p * len(layer_ptrs))(*[int(p) for p in layer_ptrs])
    _check(lib().q4_layer_decode_noalloc(ctypes.byref(shape), arr, len(layer_ptrs), _ptr(hidden), _stream(stream)),
           "q4_layer_decode_noalloc")


def q4_noalloc_scratch_bytes() -> int:
    return lib().q4_noalloc_scratch_bytes()


def q4_noalloc_status(stream=None) -> int:
    v = c_int(0)
    _check(lib().q4_noalloc_status(_stream(stream), ctypes.byref(v)), "q4_noalloc_status")
    return v.value


def q4_stream_create(shape: LayerShape, host_ptrs, batch: int, buf0, buf1, buf_bytes: int, workspace,
                     workspace_bytes: int, flags: int = 0):
    h = c_p()
    arr = (c_p * len(host_ptrs))(*[int(p) for p in host_ptrs])
    _check(lib().q4_stream_create(ctypes.byref(h), ctypes.byref(shape), arr, len(host_ptrs), batch, _ptr(buf0),
                                  _ptr(buf1), buf_bytes, _ptr(workspace), workspace_bytes, flags),
           "q4_stream_create")
    return h


def q4_stream_create_ex(shape: LayerShape, host_ptrs, resident_ptrs, batch: int, buf0, buf1, buf_bytes: int,
                        workspace, workspace_bytes: int, flags: int = 0):
    """host_ptrs[i] / resident_ptrs[i]: pinned host block or device block of layer i (0 = none)."""
    h = c_p()
    n = len(host_ptrs)
    harr = (c_p * n)(*[int(p) if p else None for p in host_ptrs])
    rarr = None if resident_ptrs is None else (c_p * n)(*[int(p) if p else None for p in resident_ptrs])
    _check(lib().q4_stream_create_ex(ctypes.byref(h), ctypes.byref(shape), harr, rarr, n, batch, _ptr(buf0),
                                     _ptr(buf1), buf_bytes, _ptr(workspace), workspace_bytes, flags),
           "q4_stream_create_ex")
    return h


def q4_attn_decode(q, k_cache, v_cache, ctx_len, capacity: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                   out, workspace, workspace_bytes: int, stream=None):
    _check(lib().q4_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(ctx_len), capacity, n_q_heads,
                                n_kv_heads, head_dim, _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)),
           "q4_attn_decode")


def q4_attn_workspace_bytes(n_q_heads: int, n_kv_heads: int, head_dim: int, capacity: int) -> int:
    return lib().q4_attn_workspace_bytes(n_q_heads, n_kv_heads, head_dim, capacity)


def q4_kv_append(k, v, k_cache, v_cache, pos, capacity: int, kv_dim: int, stream=None):
    _check(lib().q4_kv_append(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(pos), capacity, kv_dim,
                              _stream(stream)), "q4_kv_append")


def q4_paged_write(kv: PagedKV, batch: PagedBatch, k, v, kind: int, ld: int, stream=None):
    """The new tokens' keys and values (rows of Q4_TYPE_F32 or Q4_TYPE_F16 values, ld apart) into their pages."""
    dev, rows, row = _device_for("q4_paged_write", kv, batch), batch.n_tokens, kv.n_kv_heads * kv.head_dim
    _check(lib().q4_paged_write(kv, batch, _rows_ptr(k, "q4_paged_write: k", rows, row, ld, kind, dev),
                                _rows_ptr(v, "q4_paged_write: v", rows, row, ld, kind, dev), kind, ld,
                                _stream_on(stream, dev)), "q4_paged_write")


def q4_paged_read(kv: PagedKV, batch: PagedBatch, k, v, kind: int, ld: int, stream=None):
    """The batch's positions out of their pages into rows of Q4_TYPE_F32 or Q4_TYPE_F16 values, ld apart."""
    dev, rows, row = _device_for("q4_paged_read", kv, batch), batch.n_tokens, kv.n_kv_heads * kv.head_dim
    _check(lib().q4_paged_read(kv, batch, _rows_ptr(k, "q4_paged_read: k", rows, row, ld, kind, dev),
                               _rows_ptr(v, "q4_paged_read: v", rows, row, ld, kind, dev), kind, ld,
                               _stream_on(stream, dev)), "q4_paged_read")


def q4_attn_paged(kv: PagedKV, batch: PagedBatch, q, q_type: int, q_ld: int, n_q_heads: int, window: int, sinks: int,
                  out, out_ld: int, workspace, workspace_bytes: int, stream=None):
    """Attention of the new tokens over their sequences' pages, into binary16 rows out_ld apart."""
    dev, rows, row = _device_for("q4_attn_paged", kv, batch), batch.n_tokens, n_q_heads * kv.head_dim
    _check(lib().q4_attn_paged(kv, batch, _rows_ptr(q, "q4_attn_paged: q", rows, row, q_ld, q_type, dev), q_type, q_ld,
                               n_q_heads, window, sinks,
                               _rows_ptr(out, "q4_attn_paged: out", rows, row, out_ld, Q4_TYPE_F16, dev), out_ld,
                               _bytes_ptr(workspace, workspace_bytes, dev), workspace_bytes, _stream_on(stream, dev)), "q4_attn_paged")


def q4_attn_paged_workspace_bytes(n_q_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return lib().q4_attn_paged_workspace_bytes(n_q_heads, n_kv_heads, head_dim)


def q4_stream_layers(st, hidden, stream=None, timeout_us: int = 0):
    return _check(lib().q4_stream_layers(st, _ptr(hidden), _stream(stream), timeout_us), "q4_stream_layers")


def q4_stream_timeline(st, n_layers: int, stream=None):
    """[n_layers][4] globaltimer ns: copy begin, copy end, compute begin, compute end."""
    import numpy as np
    out = np.zeros(4 * n_layers, dtype=np.uint64)
    _check(lib().q4_stream_timeline(st, out.ctypes.data_as(ctypes.c_void_p), out.size, _stream(stream)),
           "q4_stream_timeline")
    return out.reshape(n_layers, 4)


TIMELINE_CTAS, TIMELINE_PHASES, TIMELINE_EVENTS = 256, 64, 6


def q4_timeline_read(clear: bool = True):
    """[CTA][phase][event] globaltimer ns of the engine's last launches (timeline build only)."""
    import numpy as np
    out = np.zeros(TIMELINE_CTAS * TIMELINE_PHASES * TIMELINE_EVENTS, dtype=np.uint64)
    _check(lib().q4_timeline_read(out.ctypes.data_as(ctypes.c_void_p), out.size, 1 if clear else 0),
           "q4_timeline_read")
    return out.reshape(TIMELINE_CTAS, TIMELINE_PHASES, TIMELINE_EVENTS)


def q4_stream_tagged(st) -> bool:
    v = c_int(0)
    _check(lib().q4_stream_tagged(st, ctypes.byref(v)), "q4_stream_tagged")
    return bool(v.value)


def q4_stream_status(st, stream=None) -> int:
    v = c_int(0)
    _check(lib().q4_stream_status(st, _stream(stream), ctypes.byref(v)), "q4_stream_status")
    return v.value


def q4_stream_destroy(st):
    _check(lib().q4_stream_destroy(st), "q4_stream_destroy")
