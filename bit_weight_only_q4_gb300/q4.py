"""Thin ctypes binding of the C ABI in ``include/q4.h`` (same entry-point names).

Only argument marshalling happens here: tensors are passed as raw device
pointers with their sizes and the current CUDA stream; every step of the
computation runs in the library's sm_103a kernels.  Output and workspace tensors
are allocated with PyTorch when the caller does not pass them (the library
itself never allocates).  If the shared library has not been built, the first
call raises :class:`Q4Error` -- there is no fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import build as _build

LAYOUT_INT4G128 = 0
LAYOUT_NVFP4 = 1
CACHE_INT8 = 0
CACHE_INT4 = 1
KV_COUNTER_BYTES = 4096
FLAG_PDL = 0x1
FLAG_FORCE_CUDA_CORE = 0x2
FLAG_FORCE_TENSOR_CORE = 0x4

STATUS = {0: "Q4_OK", 1: "Q4_ERR_NULL", 2: "Q4_ERR_SHAPE", 3: "Q4_ERR_ALIGN",
          4: "Q4_ERR_WORKSPACE", 5: "Q4_ERR_ARG", 6: "Q4_ERR_CUDA", 7: "Q4_ERR_DEVICE"}

_lib = None
_lock = threading.Lock()


class Q4Error(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {detail}")


def lib_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load the shared library (raises Q4Error if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if not os.path.exists(path):
            raise Q4Error(-1, f"{path} is missing: build it with "
                              f"`python -m bit_weight_only_q4_gb300.build` (no fallback exists)")
        L = ctypes.CDLL(path)
        p, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        i64, f = ctypes.c_int64, ctypes.c_float
        st = ctypes.c_int
        sig = {
            "q4_abi_version": ([], ctypes.c_int),
            "q4_status_string": ([st], ctypes.c_char_p),
            "q4_last_error_string": ([], ctypes.c_char_p),
            "q4_set_launch_flags": ([ctypes.c_uint], st),
            "q4_get_launch_flags": ([], ctypes.c_uint),
            "q4_workspace_bytes": ([i, i, i, i], sz),
            "q4_linear_int4g128": ([p, p, p, p, p, i, i, i, p, sz, p], st),
            "q4_linear_nvfp4": ([p, p, p, p, p, i, i, i, p, sz, p], st),
            "q4_linear_int4g128_noalloc": ([p, p, p, p, p, i, i, i, p], st),
            "audio_head_logits_restricted": ([p, p, i, i, i, i, p, i, i, p], st),
            "q4_device_error_flags": ([ctypes.POINTER(ctypes.c_uint), i], st),
            "q4_dequant_int4g128_f32": ([p, p, p, p, i, i, p], st),
            "q4_dequant_nvfp4_f32": ([p, p, p, p, i, i, p], st),
            "q4_quantize_int4g128": ([p, p, p, p, i, i, p], st),
            "q4_embedding_int8": ([p, p, p, p, i, i, i, p], st),
            "q4_linear_int8": ([p, p, p, p, i, i, i, p], st),
            "q4_quantize_nvfp4": ([p, p, p, p, i, i, p], st),
            "q4_kv_block_bytes": ([i, i], sz),
            # of the CUDA runtime that the library is linked with
            "cudaStreamIsCapturing": ([p, p], ctypes.c_int),
            "cudaStreamGetCaptureInfo": ([p] * 7, ctypes.c_int),
            "q4_kv_write": ([p, i64, p, i64, p, i, p, i, i, i, i, i, p], st),
            "q4_kv_read": ([p, i, i, i, i, i, p, i, p, i, i, p, p, p], st),
            "q4_test_kv_give_up": ([i, i], None),
            "q4_kv_attention_workspace_bytes": ([i, i, i, i, i, i, i], sz),
            "q4_kv_attention": ([p, i64, p, i, i, i, i, i, p, i, p, i, i, i, f, p, p, sz, p], st),
            "q4_kv_attention_shared": ([p, i64, p, i, i, i, i, i, p, i, p, i, p, i, i, i, f, p, p,
                                        sz, p], st),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        return L


def symbols() -> list[str]:
    """Entry points the binding expects the library to export."""
    return ["q4_abi_version", "q4_status_string", "q4_last_error_string",
            "q4_set_launch_flags", "q4_get_launch_flags", "q4_workspace_bytes",
            "q4_linear_int4g128", "q4_linear_nvfp4", "audio_head_logits_restricted",
            "q4_linear_int4g128_noalloc", "q4_device_error_flags", "q4_dequant_int4g128_f32",
            "q4_dequant_nvfp4_f32", "q4_quantize_int4g128", "q4_quantize_nvfp4",
            "q4_embedding_int8", "q4_linear_int8", "q4_kv_block_bytes", "q4_kv_write",
            "q4_kv_read", "q4_kv_attention_workspace_bytes", "q4_kv_attention",
            "q4_kv_attention_shared", "q4_test_kv_give_up"]


def _check(status: int) -> None:
    if status != 0:
        detail = load().q4_last_error_string().decode(errors="replace")
        raise Q4Error(status, detail)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _cuda(t, name, dtype=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def set_launch_flags(flags: int) -> None:
    _check(load().q4_set_launch_flags(flags))


def get_launch_flags() -> int:
    return int(load().q4_get_launch_flags())


def device_error_flags(clear: bool = True) -> int:
    """Device error word (bit 0: a bounded in-kernel wait timed out; bit 2: an
    embedding id, a cache slot or a page id out of range). Synchronises."""
    v = ctypes.c_uint(0)
    _check(load().q4_device_error_flags(ctypes.byref(v), 1 if clear else 0))
    return int(v.value)


def workspace_bytes(layout: int, M: int, N: int, K: int) -> int:
    return int(load().q4_workspace_bytes(layout, M, N, K))


def alloc_workspace(layout: int, M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """Zero-filled workspace for the given call shape (None when none is needed)."""
    n = workspace_bytes(layout, M, N, K)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _ws_args(ws):
    if ws is None:
        return None, 0
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _on(stream):
    """Allocations made inside belong to the stream that the call runs on, so that neither
    their fill nor their reuse by the allocator overlaps the call."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _capture_id(handle, stream):
    """Nonzero, and the same for one capture, while the call's stream is being captured into a graph."""
    if not handle:                       # (the legacy default stream cannot be)
        return 0
    lib, state = _lib or load(), ctypes.c_int()
    if stream is None:
        if not torch.cuda.is_current_stream_capturing():
            return 0
    elif lib.cudaStreamIsCapturing(handle, ctypes.byref(state)) or not state.value:
        return 0
    number = ctypes.c_ulonglong()
    status = lib.cudaStreamGetCaptureInfo(handle, ctypes.byref(state), ctypes.byref(number), None, None, None, None)
    return number.value if status == 0 and state.value == 1 else 0


# A graph keeps the addresses of the workspaces that its calls used, and nothing else of
# them: what a captured call has been given is never freed (by its address), and what a
# capture had to make for itself lies in the graph's own memory, filled by the graph.
_ws_held: dict = {}
_ws_graph: dict = {}


def _new_workspace(n, zeroed, device, stream):
    with _on(stream) if stream is not None else contextlib.nullcontext():
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        ws[:zeroed].zero_()
    return ws


def _graph_workspace(capture, key, n, zeroed, device, stream):
    """For a call that is captured before any has made a workspace that would do: one for all such
    calls of the capture, and for no others, for its fill has not run yet."""
    last = _ws_graph.get(key)
    if last is not None and last[0] == capture and last[1].numel() >= n:
        return last[1]
    ws = _new_workspace(n, zeroed, device, stream)
    if len(_ws_graph) >= 64:
        _ws_graph.clear()
    _ws_graph[key] = capture, ws
    return ws


# Workspaces the binding supplies when the caller passes none: one per (device,
# stream, layout and shape), zero-filled once.  Calls of one shape on one stream
# run in order (with programmatic dependent launch a kernel touches the
# workspace only after the previous kernel has finished) and leave its counters
# at zero, so they can share it; a different shape lays counters and partial
# sums out differently and gets its own.  Reuse also keeps allocations, and
# their fill kernels, out of captured CUDA graphs once a stream has made one
# call of each shape.
_ws_cache: dict = {}


def _default_workspace(layout: int, M: int, N: int, K: int, device, handle, stream) -> torch.Tensor | None:
    n = workspace_bytes(layout, M, N, K)
    if n == 0:
        return None
    key = (device.index, handle, layout, M, N, K)
    ws = _ws_cache.get(key)
    capture = _capture_id(handle, stream)
    if ws is not None and ws.numel() >= n:       # (a launch flag can change the size)
        if capture:
            _ws_held[ws.data_ptr()] = ws
        return ws
    if capture:
        return _graph_workspace(capture, key, n, n, device, stream)
    if len(_ws_cache) >= 64:            # many distinct shapes: start over (memory is
        _ws_cache.clear()               # returned in stream order by the allocator)
    ws = _new_workspace(n, n, device, stream)
    _ws_cache[key] = ws
    return ws


def q4_linear_int4g128(x, qweight, scale, minv, y=None, workspace=None, stream=None):
    """y[M, N] (bf16) = x[M, K] (bf16) W^T, W in the int4-g128-minmax layout."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(qweight, "qweight", torch.uint8)
    _cuda(scale, "scale")
    _cuda(minv, "min")
    M, K = x.shape
    N = qweight.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    handle = _stream(stream)
    if workspace is None:
        workspace = _default_workspace(LAYOUT_INT4G128, M, N, K, x.device, handle, stream)
    wp, wn = _ws_args(workspace)
    _check(load().q4_linear_int4g128(_ptr(x), _ptr(qweight), _ptr(scale), _ptr(minv), _ptr(y),
                                     M, N, K, wp, wn, handle))
    return y


def q4_linear_int4g128_noalloc(x, qweight, scale, minv, y, stream=None):
    """As q4_linear_int4g128, for callers that cannot allocate device memory: the
    library's own static scratch replaces the workspace and ``y`` must be given."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(qweight, "qweight", torch.uint8)
    _cuda(scale, "scale")
    _cuda(minv, "min")
    _cuda(y, "y", torch.bfloat16)
    M, K = x.shape
    N = qweight.shape[0]
    _check(load().q4_linear_int4g128_noalloc(_ptr(x), _ptr(qweight), _ptr(scale), _ptr(minv),
                                             _ptr(y), M, N, K, _stream(stream)))
    return y


def q4_linear_nvfp4(x, codes, scale_e4m3, global_scale, y=None, workspace=None, stream=None):
    """y[M, N] (bf16) = x[M, K] (bf16) W^T, W in the NVFP4 weight-only layout;
    ``global_scale`` is a one-element fp32 CUDA tensor."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(codes, "codes", torch.uint8)
    _cuda(scale_e4m3, "scale_e4m3")
    _cuda(global_scale, "global_scale", torch.float32)
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    handle = _stream(stream)
    if workspace is None:
        workspace = _default_workspace(LAYOUT_NVFP4, M, N, K, x.device, handle, stream)
    wp, wn = _ws_args(workspace)
    _check(load().q4_linear_nvfp4(_ptr(x), _ptr(codes), _ptr(scale_e4m3), _ptr(global_scale),
                                  _ptr(y), M, N, K, wp, wn, handle))
    return y


def audio_head_logits_restricted(h, head, row_begin, n_rows, extra_row=-1, logits=None,
                                 stream=None):
    """logits[M, n_rows + (extra_row >= 0)] (bf16) of the restricted head."""
    _cuda(h, "h", torch.bfloat16)
    _cuda(head, "head", torch.bfloat16)
    M, H = h.shape
    cols = n_rows + (1 if extra_row >= 0 else 0)
    if logits is None:
        logits = torch.empty((M, max(cols, 1)), dtype=torch.bfloat16, device=h.device)
    _check(load().audio_head_logits_restricted(_ptr(h), _ptr(head), head.shape[0], row_begin,
                                               n_rows, extra_row, _ptr(logits), M, H,
                                               _stream(stream)))
    return logits


def q4_dequant_int4g128_f32(qweight, scale, minv, stream=None):
    N, K = qweight.shape[0], 2 * qweight.shape[1]
    w = torch.empty((N, K), dtype=torch.float32, device=qweight.device)
    _check(load().q4_dequant_int4g128_f32(_ptr(qweight), _ptr(scale), _ptr(minv), _ptr(w), N, K,
                                          _stream(stream)))
    return w


def q4_dequant_nvfp4_f32(codes, scale_e4m3, global_scale, stream=None):
    N, K = codes.shape[0], 2 * codes.shape[1]
    w = torch.empty((N, K), dtype=torch.float32, device=codes.device)
    _check(load().q4_dequant_nvfp4_f32(_ptr(codes), _ptr(scale_e4m3), _ptr(global_scale),
                                       _ptr(w), N, K, _stream(stream)))
    return w


# Short aliases
linear_int4g128 = q4_linear_int4g128
linear_nvfp4 = q4_linear_nvfp4
dequant_int4g128_f32 = q4_dequant_int4g128_f32
dequant_nvfp4_f32 = q4_dequant_nvfp4_f32


def q4_quantize_int4g128(w, stream=None):
    """(qweight uint8 [N, K/2], scale fp16 [N, K/128], min fp16 [N, K/128]) of the
    round-to-nearest min/max int4-g128 quantisation of bf16 weights w [N, K]."""
    _cuda(w, "w", torch.bfloat16)
    N, K = w.shape
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((N, K // 128), dtype=torch.float16, device=w.device)
    m = torch.empty((N, K // 128), dtype=torch.float16, device=w.device)
    _check(load().q4_quantize_int4g128(_ptr(w), _ptr(q), _ptr(s), _ptr(m), N, K,
                                       _stream(stream)))
    return q, s, m


def q4_quantize_nvfp4(w, stream=None):
    """(codes uint8 [N, K/2], e4m3 scales uint8 [N, K/16], global scale fp32 [1]) of
    the round-to-nearest NVFP4 quantisation of bf16 weights w [N, K]."""
    _cuda(w, "w", torch.bfloat16)
    N, K = w.shape
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((N, K // 16), dtype=torch.uint8, device=w.device)
    g = torch.empty((1,), dtype=torch.float32, device=w.device)
    _check(load().q4_quantize_nvfp4(_ptr(w), _ptr(q), _ptr(s), _ptr(g), N, K, _stream(stream)))
    return q, s, g


def q4_embedding_int8(ids, qweight, scale, out=None, stream=None):
    """bf16 [M, H] rows of the int8 token embedding for int32 ids [M]."""
    _cuda(ids, "ids", torch.int32)
    _cuda(qweight, "qweight", torch.int8)
    _cuda(scale, "scale", torch.float16)
    V, H = qweight.shape
    M = ids.numel()
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=qweight.device)
    _check(load().q4_embedding_int8(_ptr(ids), _ptr(qweight), _ptr(scale), _ptr(out), M, V, H,
                                    _stream(stream)))
    return out


def q4_linear_int8(x, qweight, scale, y=None, stream=None):
    """y[M, N] (bf16) = x[M, K] (bf16) W^T, W int8 [N, K] with an fp16 scale per row."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(qweight, "qweight", torch.int8)
    _cuda(scale, "scale", torch.float16)
    M, K = x.shape
    N = qweight.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check(load().q4_linear_int8(_ptr(x), _ptr(qweight), _ptr(scale), _ptr(y), M, N, K,
                                 _stream(stream)))
    return y


# ------------------------------------------------------------ paged K/V cache
# Bytes that 16 tokens of one head take, by (format, head_dim): 32 code rows, 32 scales.
_KV_BLOCK = {(CACHE_INT8, 64): 32 * (64 + 2), (CACHE_INT8, 128): 32 * (128 + 2),
             (CACHE_INT4, 64): 32 * (32 + 4), (CACHE_INT4, 128): 32 * (64 + 4)}
# The handle of a device's current stream without building a Stream object around it:
# these calls take a few microseconds on the GPU, and building one takes three.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def kv_block_bytes(fmt: int, head_dim: int) -> int:
    """Bytes that 16 tokens of one head take in a cache of the given format (0: no such cache)."""
    return _KV_BLOCK.get((fmt, head_dim), 0)


def alloc_kv_cache(fmt: int, pages: int, page_size: int, kv_heads: int, head_dim: int,
                   device=None) -> torch.Tensor:
    """An uninitialised K/V cache: uint8 [pages, kv_heads, page_size / 16, block bytes].
    Tokens are written with q4_kv_write; what no write has reached is never used."""
    n = kv_block_bytes(fmt, head_dim)
    if n == 0 or not 16 <= page_size <= 1024 or page_size & (page_size - 1):
        raise ValueError(f"no cache of format {fmt}, head_dim {head_dim}, page_size {page_size}")
    return torch.empty((pages, kv_heads, page_size // 16, n), dtype=torch.uint8,
                       device=device or "cuda")


def _kv_stream(stream, t):
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.get_device())
    return _stream(stream)


def _kv_empty(shape, like, stream):
    if stream is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=like.device)
    with _on(stream):
        return torch.empty(shape, dtype=torch.bfloat16, device=like.device)


def _kv_cache(cache, fmt, head_dim):
    """(format, pages, page_size, kv_heads, head_dim) of a cache tensor."""
    n = _KV_BLOCK.get((fmt, head_dim), 0)
    if not (cache.is_cuda and cache.is_contiguous() and cache.dtype is torch.uint8):
        raise ValueError("cache must be a contiguous uint8 CUDA tensor")
    shape = cache.shape
    if n == 0 or len(shape) != 4 or shape[3] != n:
        raise ValueError(f"cache must be [pages, kv_heads, page_size / 16, {n}] for format {fmt} "
                         f"and head_dim {head_dim}, got {tuple(shape)}")
    return fmt, shape[0], 16 * shape[2], shape[1], head_dim


def _kv_ints(t, name, dims):
    """An int32 CUDA tensor of the given number of dimensions: its shape."""
    if not (t.is_cuda and t.is_contiguous() and t.dtype is torch.int32 and t.dim() == dims):
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {dims} dimension(s)")
    return t.shape


def _kv_rows(t, name, shape):
    """A bf16 CUDA tensor [..., heads, D] whose tokens are evenly spaced and whose heads lie
    side by side (a slice of a fused q|k|v projection does): the token stride."""
    if not (t.is_cuda and t.dtype is torch.bfloat16):
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor")
    strides = t.stride()
    heads, D = shape[-2:]
    row, even = strides[-3], True
    if len(shape) == 4:
        if shape[1] == 1:
            row = strides[0]
        even = shape[0] == 1 or strides[0] == shape[1] * row
        if shape[0] == 1 and shape[1] == 1:
            row = heads * D
    elif shape[0] == 1:
        row = heads * D
    if not even or strides[-1] != 1 or (heads > 1 and strides[-2] != D):
        raise ValueError(f"{name} must have contiguous heads and evenly spaced tokens, got "
                         f"strides {strides}")
    return row


# What the checks of a call found, by the shapes and strides it was made with (types, devices
# and contiguity are looked at in every call): a small call's Python would take as long
# as its kernel.
_kv_plans: dict = {}


def _kv_plan(key, plan):
    if len(_kv_plans) >= 256:
        _kv_plans.clear()
    _kv_plans[key] = plan
    return plan


def _kv_typed(rows, cache, table, lengths):
    """True if a call's tensors are of the kinds that all of its checks ask for."""
    return (cache.dtype is torch.uint8 and cache.is_cuda and cache.is_contiguous() and
            table.dtype is torch.int32 and table.is_cuda and table.is_contiguous() and
            lengths.dtype is torch.int32 and lengths.is_cuda and lengths.is_contiguous() and
            (rows is None or (rows.dtype is torch.bfloat16 and rows.is_cuda)))


def q4_kv_write(k, v, cache, slots, fmt, stream=None):
    """Quantise K and V rows (bf16 [tokens, kv_heads, D]) into the cache's slots
    (int32 [tokens]; slot = page * page_size + token in the page, negative: left out)."""
    shape = k.shape
    if len(shape) != 3 or shape != v.shape:
        raise ValueError(f"k and v must be [tokens, kv_heads, D], got {tuple(shape)} and {tuple(v.shape)}")
    ks, vs = _kv_rows(k, "k", shape), _kv_rows(v, "v", shape)
    if _kv_ints(slots, "slots", 1)[0] != shape[0]:
        raise ValueError("slots must hold one slot for each token")
    geo = _kv_cache(cache, fmt, shape[2])
    if geo[3] != shape[1]:
        raise ValueError(f"the cache holds {geo[3]} heads, k has {shape[1]}")
    if shape[0] == 0:
        return cache
    status = (_lib or load()).q4_kv_write(k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(), shape[0],
                                          cache.data_ptr(), *geo, _kv_stream(stream, k))
    if status:
        _check(status)
    return cache


def q4_kv_read(cache, page_table, lengths, max_len, head_dim, fmt, k=None, v=None, stream=None):
    """(k, v) bf16 [batch, max_len, kv_heads, head_dim] of the first lengths[b] cached tokens
    of each sequence, zeros behind them."""
    key = (fmt, head_dim, max_len, cache.shape, page_table.shape, lengths.shape)
    plan = _kv_plans.get(key)
    if plan is None or not _kv_typed(None, cache, page_table, lengths):
        geo = _kv_cache(cache, fmt, head_dim)
        batch, width = _kv_ints(page_table, "page_table", 2)
        if _kv_ints(lengths, "lengths", 1)[0] != batch:
            raise ValueError("page_table must be [batch, width] and lengths [batch]")
        plan = _kv_plan(key, (geo, batch, width, (batch, max_len, geo[3], head_dim)))
    geo, batch, width, shape = plan
    if k is None:
        k = _kv_empty(shape, cache, stream)
    elif tuple(_cuda(k, "k", torch.bfloat16).shape) != shape:
        raise ValueError(f"k must be {shape}, got {tuple(k.shape)}")
    if v is None:
        v = _kv_empty(shape, cache, stream)
    elif tuple(_cuda(v, "v", torch.bfloat16).shape) != shape:
        raise ValueError(f"v must be {shape}, got {tuple(v.shape)}")
    if batch * max_len == 0:
        return k, v
    status = (_lib or load()).q4_kv_read(cache.data_ptr(), *geo, page_table.data_ptr(), width,
                                         lengths.data_ptr(), batch, max_len, k.data_ptr(), v.data_ptr(),
                                         _kv_stream(stream, cache))
    if status:
        _check(status)
    return k, v


def kv_attention_workspace_bytes(fmt, kv_heads, head_dim, batch, tokens, q_heads, prefix_len=0) -> int:
    return int(load().q4_kv_attention_workspace_bytes(fmt, kv_heads, head_dim, batch, tokens,
                                                      q_heads, prefix_len))


# Workspaces of attention calls: one per (device, stream), for calls of every shape.
_kv_ws: dict = {}


def _kv_workspace(n, device, handle, stream):
    key = (device.index, handle)
    ws = _kv_ws.get(key)
    capture = _capture_id(handle, stream)
    if ws is not None and ws.numel() >= n:
        if capture:
            _ws_held[ws.data_ptr()] = ws
        return ws
    if capture:
        return _graph_workspace(capture, key, n, KV_COUNTER_BYTES, device, stream)
    # (a list of growing calls makes a few, not one for each)
    ws = _new_workspace(n if ws is None else max(n, 2 * ws.numel()), KV_COUNTER_BYTES, device, stream)
    if len(_kv_ws) >= 64:
        _kv_ws.clear()
    _kv_ws[key] = ws
    return ws


def _kv_attention(q, cache, prefix_pages, prefix_len, page_table, lengths, fmt, scale, out, workspace,
                  stream):
    shape = q.shape
    key = (fmt, prefix_len, shape, q.stride(), cache.shape, page_table.shape, lengths.shape)
    plan = _kv_plans.get(key)
    if plan is None or not _kv_typed(q, cache, page_table, lengths):
        if len(shape) != 4:
            raise ValueError(f"q must be [batch, tokens, q_heads, D], got {tuple(shape)}")
        row = _kv_rows(q, "q", shape)
        B, T, Hq, D = shape
        geo = _kv_cache(cache, fmt, D)
        batch, width = _kv_ints(page_table, "page_table", 2)
        if batch != B or _kv_ints(lengths, "lengths", 1)[0] != B:
            raise ValueError(f"page_table must be [batch, width] and lengths [batch], q has {B} sequences")
        size = kv_attention_workspace_bytes(fmt, geo[3], D, B, T, Hq, prefix_len)
        plan = _kv_plan(key, (row, geo, width, B, T, Hq, D, D**-0.5 if D else 1.0, size))
    row, geo, width, B, T, Hq, D, s, size = plan
    if out is None:
        out = _kv_empty(shape, q, stream)
    elif _cuda(out, "out", torch.bfloat16).shape != shape:
        raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    if B * T * Hq == 0:
        return out
    handle = _kv_stream(stream, q)
    if workspace is None and size:
        workspace = _kv_workspace(size, q.device, handle, stream)
    wp, wn = _ws_args(workspace)
    if scale is not None:
        s = float(scale)
    lib = _lib or load()
    if prefix_pages is not None:
        status = lib.q4_kv_attention_shared(q.data_ptr(), row, cache.data_ptr(), *geo, prefix_pages.data_ptr(),
                                            prefix_len, page_table.data_ptr(), width, lengths.data_ptr(), B, T,
                                            Hq, s, out.data_ptr(), wp, wn, handle)
    else:
        status = lib.q4_kv_attention(q.data_ptr(), row, cache.data_ptr(), *geo, page_table.data_ptr(), width,
                                     lengths.data_ptr(), B, T, Hq, s, out.data_ptr(), wp, wn, handle)
    if status:
        _check(status)
    return out


def q4_kv_attention(q, cache, page_table, lengths, fmt, scale=None, out=None, workspace=None,
                    stream=None):
    """out [batch, tokens, q_heads, D] (bf16) = softmax(scale q K^T) V over the cached tokens of
    each sequence; the query tokens q (bf16, same shape) are the sequence's last ones.
    scale: D ** -0.5 if None; lengths int32 [batch], page_table int32 [batch, width]."""
    return _kv_attention(q, cache, None, 0, page_table, lengths, fmt, scale, out, workspace, stream)


def q4_kv_attention_shared(q, cache, prefix_pages, prefix_len, page_table, lengths, fmt, scale=None,
                           out=None, workspace=None, stream=None):
    """As q4_kv_attention where every sequence begins with the prefix_len tokens of the pages
    prefix_pages (int32): they are read and multiplied once for the whole batch.  page_table and
    lengths describe each sequence's own tokens behind them."""
    n = _kv_ints(prefix_pages, "prefix_pages", 1)[0]
    if cache.dim() != 4:
        raise ValueError(f"cache must be [pages, kv_heads, page_size / 16, block bytes], got {tuple(cache.shape)}")
    page = 16 * cache.shape[2]
    if prefix_len < 1 or n * page < prefix_len:
        raise ValueError(f"prefix_pages holds {n} pages of {page}, the prefix has {prefix_len} tokens")
    return _kv_attention(q, cache, prefix_pages, prefix_len, page_table, lengths, fmt, scale, out,
                         workspace, stream)
