"""ctypes binding of libfa2.so (declared in include/fa2.h).

Argument marshalling only: every step of the attention computation runs in the
library's CUDA kernels.  Tensors are torch CUDA tensors (PyTorch provides device
memory and streams); they are passed to the C ABI as raw device pointers.  A
missing or unloadable library raises ``RuntimeError`` -- there is no fallback.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa2.so")

FA2_OK = 0
FA2_ERR_INVALID_ARG = 1
FA2_ERR_UNSUPPORTED = 2
FA2_ERR_ARCH = 3
FA2_ERR_CUDA = 4
FA2_ERR_TIMEOUT = 5
FA2_ERR_WORKSPACE = 6
FA2_FP16 = 0
FA2_BF16 = 1
FA2_BWD_DETERMINISTIC = 1  # flag of fa2_bwd_ex

# Every symbol include/fa2.h declares.
EXPORTS = ("fa2_fwd", "fa2_fwd_window", "fa2_fwd_fp8", "fa2_fwd_tiles_per_cta",
           "fa2_fwd_decode_splits", "fa2_fwd_decode_workspace_size", "fa2_fwd_decode",
           "fa2_bwd_workspace_size", "fa2_bwd", "fa2_bwd_window", "fa2_bwd_ex",
           "fa2_bwd_ex_workspace_size", "fa2_bwd_noalloc", "fa2_get_device_status",
           "fa2_fwd_varlen", "fa2_bwd_varlen_workspace_size", "fa2_bwd_varlen",
           "fa2_fwd_paged_workspace_size", "fa2_fwd_paged", "fa2_paged_tables",
           "fa2_paged_append", "fa2_status_string", "fa2_debug_set", "fa2_debug_set_bwd_grid",
           "fa2_debug_set_fwd_tiles", "fa2_launch_count")

_lib = None


class FA2Packed(ctypes.Structure):
    """fa2_packed: a [T, heads, d] tensor by its address and strides in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_row", ctypes.c_longlong),
                ("stride_head", ctypes.c_longlong)]


class FA2Cache(ctypes.Structure):
    """fa2_cache: a [blocks, heads, block_size, d] cache by its address and strides."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_block", ctypes.c_longlong),
                ("stride_head", ctypes.c_longlong), ("stride_row", ctypes.c_longlong)]


class FA2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def load() -> ctypes.CDLL:
    """Open libfa2.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m exact_io_aware_74_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa2_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    lib.fa2_fwd.restype = i
    lib.fa2_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    lib.fa2_fwd_window.restype = i
    lib.fa2_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, f, f, f, vp]
    lib.fa2_fwd_fp8.restype = i
    lib.fa2_fwd_tiles_per_cta.argtypes = [i, i, i, i, i, i, i]
    lib.fa2_fwd_tiles_per_cta.restype = i
    lib.fa2_fwd_decode_splits.argtypes = [i, i, i, i, i, i]
    lib.fa2_fwd_decode_splits.restype = i
    lib.fa2_fwd_decode_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.fa2_fwd_decode_workspace_size.restype = sz
    lib.fa2_fwd_decode.argtypes = [vp] * 5 + [i, i, i, i, i, f, i, i, i, vp, sz, vp]
    lib.fa2_fwd_decode.restype = i
    lib.fa2_bwd_window.argtypes = [vp] * 10 + [sz, i, i, i, i, f, i, i, vp]
    lib.fa2_bwd_window.restype = i
    lib.fa2_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.fa2_bwd_workspace_size.restype = sz
    lib.fa2_bwd.argtypes = [vp] * 10 + [sz, i, i, i, i, f, i, i, vp]
    lib.fa2_bwd.restype = i
    lib.fa2_bwd_ex.argtypes = [vp] * 10 + [sz, i, i, i, i, f, i, i, i, i, vp]
    lib.fa2_bwd_ex.restype = i
    lib.fa2_bwd_ex_workspace_size.argtypes = [i, i, i, i, i]
    lib.fa2_bwd_ex_workspace_size.restype = sz
    lib.fa2_bwd_noalloc.argtypes = [vp] * 9 + [i, i, i, i, f, i, i, vp]
    lib.fa2_bwd_noalloc.restype = i
    pk, pc = ctypes.POINTER(FA2Packed), ctypes.POINTER(FA2Cache)
    lib.fa2_fwd_varlen.argtypes = [pk] * 4 + [vp, vp, i, i, i, i, i, f, i, i, i, vp]
    lib.fa2_fwd_varlen.restype = i
    lib.fa2_bwd_varlen_workspace_size.argtypes = [i] * 5
    lib.fa2_bwd_varlen_workspace_size.restype = sz
    lib.fa2_bwd_varlen.argtypes = [pk] * 5 + [vp] + [pk] * 3 + [vp, vp, sz, i, i, i, i, i, f, i, i,
                                                               i, vp]
    lib.fa2_bwd_varlen.restype = i
    lib.fa2_fwd_paged_workspace_size.argtypes = [i] * 6
    lib.fa2_fwd_paged_workspace_size.restype = sz
    lib.fa2_fwd_paged.argtypes = [pk, pc, pc, pk] + [vp] * 5 + [sz] + [i] * 8 + [f, i, i, i, vp]
    lib.fa2_fwd_paged.restype = i
    lib.fa2_paged_tables.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, vp, vp, i, i, i, i, vp]
    lib.fa2_paged_tables.restype = i
    lib.fa2_paged_append.argtypes = [pk, pk, pc, pc, vp, i, i, i, i, i, vp]
    lib.fa2_paged_append.restype = i
    lib.fa2_get_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    lib.fa2_get_device_status.restype = i
    lib.fa2_status_string.argtypes = [i]
    lib.fa2_status_string.restype = ctypes.c_char_p
    lib.fa2_debug_set.argtypes = [i, ctypes.c_uint]
    lib.fa2_debug_set.restype = None
    lib.fa2_debug_set_bwd_grid.argtypes = [i]
    lib.fa2_debug_set_bwd_grid.restype = None
    lib.fa2_debug_set_fwd_tiles.argtypes = [i]
    lib.fa2_debug_set_fwd_tiles.restype = None
    lib.fa2_launch_count.argtypes = []
    lib.fa2_launch_count.restype = ctypes.c_ulonglong
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().fa2_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FA2_BF16
    if t.dtype == torch.float16:
        return FA2_FP16
    raise TypeError(f"unsupported dtype {t.dtype}; use float16 or bfloat16")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check_layout(*ts):
    for t in ts:
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def fa2_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None) -> int:
    """Raw call: q, k, v, o [B,H,N,d] 16-bit; lse [B,H,N] float32.  Returns the status."""
    _check_layout(q, k, v, o, lse)
    B, H, N, d = q.shape
    return load().fa2_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                          float(scale), int(bool(causal)), _dtype_code(q), _stream(stream))


def fa2_fwd_window(q, k, v, o, lse, scale: float, window: int, stream=None) -> int:
    """Raw call of the sliding-window forward (causal, ``window`` most recent keys)."""
    _check_layout(q, k, v, o, lse)
    B, H, N, d = q.shape
    return load().fa2_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                                 float(scale), int(window), _dtype_code(q), _stream(stream))


def fa2_fwd_fp8(q, k, v, o, lse, scale: float, causal: bool, q_scale: float, k_scale: float,
                v_scale: float, stream=None) -> int:
    """Raw call: q, k, v [B,H,N,d] float8_e4m3fn; o [B,H,N,d] bfloat16; lse float32."""
    _check_layout(q, k, v, o, lse)
    for t in (q, k, v):
        if t.dtype != torch.float8_e4m3fn:
            raise TypeError("q, k, v must be float8_e4m3fn")
    if o.dtype != torch.bfloat16:
        raise TypeError("o must be bfloat16")
    B, H, N, d = q.shape
    return load().fa2_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                              float(scale), int(bool(causal)), float(q_scale), float(k_scale),
                              float(v_scale), _stream(stream))


def fa2_fwd_tiles_per_cta(B: int, H: int, N: int, d: int, causal: bool, window: int = 0,
                          sm_count: int = 0) -> int:
    """Query tiles per CTA the forward uses for these sizes (1 or 2; 0 if rejected)."""
    return load().fa2_fwd_tiles_per_cta(int(B), int(H), int(N), int(d), int(bool(causal)),
                                        int(window), int(sm_count))


def fa2_fwd_decode_splits(B: int, H: int, Nq: int, Nk: int, d: int, sm_count: int = 0) -> int:
    """Split count the library picks for these sizes (0: invalid sizes or no device)."""
    return int(load().fa2_fwd_decode_splits(B, H, Nq, Nk, d, sm_count))


def fa2_fwd_decode_workspace_size(B: int, H: int, Nq: int, Nk: int, d: int,
                                  n_splits: int) -> int:
    return int(load().fa2_fwd_decode_workspace_size(B, H, Nq, Nk, d, n_splits))


def fa2_fwd_decode(q, k, v, o, lse, scale: float, causal: bool, n_splits: int, workspace,
                   stream=None) -> int:
    """Raw call: q, o [B,H,Nq,d]; k, v [B,H,Nk,d]; lse [B,H,Nq] float32;
    ``workspace`` a uint8 CUDA tensor or None.  Returns the status."""
    _check_layout(q, k, v, o, lse)
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return load().fa2_fwd_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                                 float(scale), int(bool(causal)), _dtype_code(q), int(n_splits),
                                 _ptr(workspace), ws_bytes, _stream(stream))


def fa2_bwd_window(q, k, v, o, do, lse, dq, dk, dv, workspace, scale: float, window: int,
                   stream=None) -> int:
    """Raw call of the sliding-window backward."""
    _check_layout(q, k, v, o, do, lse, dq, dk, dv)
    B, H, N, d = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return load().fa2_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes, B, H,
                                 N, d, float(scale), int(window), _dtype_code(q),
                                 _stream(stream))


def fa2_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa2_bwd_workspace_size(B, H, N, d))


def fa2_bwd(q, k, v, o, do, lse, dq, dk, dv, workspace, scale: float, causal: bool,
            stream=None) -> int:
    """Raw call; ``workspace`` is a uint8 CUDA tensor.  Returns the status."""
    _check_layout(q, k, v, o, do, lse, dq, dk, dv)
    B, H, N, d = q.shape
    ws_ptr = _ptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return load().fa2_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                          _ptr(dk), _ptr(dv), ws_ptr, ws_bytes, B, H, N, d, float(scale),
                          int(bool(causal)), _dtype_code(q), _stream(stream))


def fa2_bwd_ex_workspace_size(B: int, H: int, N: int, d: int, flags: int) -> int:
    return int(load().fa2_bwd_ex_workspace_size(B, H, N, d, int(flags)))


def fa2_bwd_ex(q, k, v, o, do, lse, dq, dk, dv, workspace, scale: float, causal: bool,
               window: int = 0, flags: int = 0, stream=None) -> int:
    """Raw call of the backward with options (window, FA2_BWD_DETERMINISTIC)."""
    _check_layout(q, k, v, o, do, lse, dq, dk, dv)
    B, H, N, d = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return load().fa2_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                             _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes, B, H, N, d,
                             float(scale), int(bool(causal)), int(window), int(flags),
                             _dtype_code(q), _stream(stream))


def fa2_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, scale: float, causal: bool,
                    stream=None) -> int:
    """Raw call of the allocation-free backward (library-owned scratch).  Returns the status."""
    _check_layout(q, k, v, o, do, lse, dq, dk, dv)
    B, H, N, d = q.shape
    return load().fa2_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                  _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                  int(bool(causal)), _dtype_code(q), _stream(stream))


# ------------------------------------------------------------------------------------
# packed sequences, grouped heads and paged caches
# ------------------------------------------------------------------------------------

# These calls take few microseconds on the device for a decode step, so the checks are
# written for the host time they cost.

def _device_of(t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    return dev


def _rows(name: str, t, shape, dtype, dev: int) -> FA2Packed:
    """A [T, heads, d] tensor of the given shape, dtype and device, columns contiguous."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {list(shape)} {dtype} tensor on cuda:{dev}, not "
                         f"{list(t.shape)} {t.dtype} on {t.device}")
    row, head, col = t.stride()
    if col != 1 and shape[2] != 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    return FA2Packed(t.data_ptr(), row, head)


def _pages(name: str, t, shape, dtype, dev: int) -> FA2Cache:
    """A [blocks, heads, block_size, d] cache, columns contiguous."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {list(shape)} {dtype} tensor on cuda:{dev}, not "
                         f"{list(t.shape)} {t.dtype} on {t.device}")
    block, head, row, col = t.stride()
    if col != 1 and shape[3] != 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    return FA2Cache(t.data_ptr(), block, head, row)


def _ints(name: str, t, n: int, dev: int) -> int:
    """Address of a contiguous int32 tensor of n numbers."""
    if t.dtype != torch.int32 or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} numbers on cuda:{dev}, "
                         f"not {list(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _lse(t, H: int, T: int, dev: int) -> int:
    if t.dtype != torch.float32 or t.shape != (H, T) or t.get_device() != dev or \
            not t.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 [{H}, {T}] tensor on cuda:{dev}")
    return t.data_ptr()


def _dims(name: str, t, n: int):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, not {list(t.shape)}")
    return t.shape


def _call(fn, dev: int, stream, *args) -> int:
    """Calls ``fn`` with the stream (of ``dev``'s current one) last, on device ``dev``: the
    library works on the current device."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == dev:
        return fn(*args, raw)
    with torch.cuda.device(dev):
        return fn(*args, raw)


def _c_int(x) -> int:
    """A window or block size as a C int: ctypes would take it modulo 2^32."""
    return max(-1, min(x, 0x7fffffff))


def _home(t, stream):
    """Context in which outputs and workspaces of a call on ``stream`` are allocated: on that
    stream, so that their memory is free there when the call writes it and is not handed out
    to another stream while the call still runs."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        # Handle 0 is the default stream, and 1 (cudaStreamLegacy) another name of it.  torch takes
        # 0 for no handle and makes a stream of its own, and does not know 1.
        stream = torch.cuda.ExternalStream(int(stream), device=t.device) if int(stream) > 1 else \
            torch.cuda.default_stream(t.device)
    return torch.cuda.stream(stream)


def _bytes(workspace, dev: int) -> tuple[int | None, int]:
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def fa2_fwd_varlen(q, k, v, o, lse, cu_seqlens, scale: float, causal: bool, window: int = 0,
                   stream=None) -> int:
    """Raw call: q, o [T,H,d] and k, v [T,Hkv,d] 16-bit, any row and head strides that are
    multiples of 8; lse [H,T] float32; cu_seqlens [B+1] int32.  Returns the status."""
    dev, dt, code = _device_of(q), q.dtype, _dtype_code(q)
    T, H, d = shape = _dims("q", q, 3)
    Hkv = _dims("k", k, 3)[1]
    n = cu_seqlens.numel()
    return _call(load().fa2_fwd_varlen, dev, stream, _rows("q", q, shape, dt, dev),
                 _rows("k", k, (T, Hkv, d), dt, dev), _rows("v", v, (T, Hkv, d), dt, dev),
                 _rows("o", o, shape, dt, dev), _lse(lse, H, T, dev),
                 _ints("cu_seqlens", cu_seqlens, n, dev), n - 1, T, H, Hkv, d, scale,
                 1 if causal else 0, _c_int(window), code)


def fa2_bwd_varlen_workspace_size(B: int, T: int, H: int, Hkv: int, d: int) -> int:
    return load().fa2_bwd_varlen_workspace_size(B, T, H, Hkv, d)


def fa2_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens, workspace, scale: float,
                   causal: bool, window: int = 0, stream=None) -> int:
    """Raw call of the packed backward; ``workspace`` is a uint8 CUDA tensor."""
    dev, dt, code = _device_of(q), q.dtype, _dtype_code(q)
    T, H, d = shape = _dims("q", q, 3)
    Hkv = _dims("k", k, 3)[1]
    kv = (T, Hkv, d)
    n = cu_seqlens.numel()
    return _call(load().fa2_bwd_varlen, dev, stream, _rows("q", q, shape, dt, dev),
                 _rows("k", k, kv, dt, dev), _rows("v", v, kv, dt, dev),
                 _rows("o", o, shape, dt, dev), _rows("do", do, shape, dt, dev),
                 _lse(lse, H, T, dev), _rows("dq", dq, shape, dt, dev),
                 _rows("dk", dk, kv, dt, dev), _rows("dv", dv, kv, dt, dev),
                 _ints("cu_seqlens", cu_seqlens, n, dev), *_bytes(workspace, dev), n - 1, T, H,
                 Hkv, d, scale, 1 if causal else 0, _c_int(window), code)


def fa2_fwd_paged_workspace_size(B: int, T: int, H: int, Hkv: int, d: int,
                                 sm_count: int = 0) -> int:
    return load().fa2_fwd_paged_workspace_size(B, T, H, Hkv, d, sm_count)


def fa2_fwd_paged(q, k_cache, v_cache, o, lse, block_table, cu_seqlens, seq_lens, workspace,
                  scale: float, causal: bool, window: int = 0, stream=None) -> int:
    """Raw call: q, o [T,H,d]; caches [blocks,Hkv,block_size,d]; lse [H,T] float32;
    block_table [B,max_blocks], cu_seqlens [B+1], seq_lens [B] int32."""
    dev, dt, code = _device_of(q), q.dtype, _dtype_code(q)
    T, H, d = shape = _dims("q", q, 3)
    blocks, Hkv, bs, dc = _dims("k_cache", k_cache, 4)
    pages = (blocks, Hkv, bs, d)
    B, most = _dims("block_table", block_table, 2)
    return _call(load().fa2_fwd_paged, dev, stream, _rows("q", q, shape, dt, dev),
                 _pages("k_cache", k_cache, pages, dt, dev),
                 _pages("v_cache", v_cache, pages, dt, dev), _rows("o", o, shape, dt, dev),
                 _lse(lse, H, T, dev), _ints("cu_seqlens", cu_seqlens, B + 1, dev),
                 _ints("seq_lens", seq_lens, B, dev),
                 _ints("block_table", block_table, B * most, dev), *_bytes(workspace, dev), B, T,
                 H, Hkv, d, blocks, bs, most, scale, 1 if causal else 0, _c_int(window), code)


def fa2_paged_tables(context_lens, new_lens, free_blocks, block_table, cu_seqlens, seq_lens,
                     positions, slots, used, block_size: int, stream=None) -> int:
    """Raw call: int32 tensors, context_lens and new_lens [B], free_blocks [num_free],
    block_table [B,max_blocks] (updated), cu_seqlens [B+1], seq_lens [B], positions and
    slots [T], used [1]."""
    dev = _device_of(block_table)
    B, most = _dims("block_table", block_table, 2)
    free, T = free_blocks.numel(), slots.numel()
    return _call(load().fa2_paged_tables, dev, stream,
                 _ints("context_lens", context_lens, B, dev), _ints("new_lens", new_lens, B, dev),
                 _ints("free_blocks", free_blocks, free, dev), free,
                 _ints("block_table", block_table, B * most, dev),
                 _ints("cu_seqlens", cu_seqlens, B + 1, dev), _ints("seq_lens", seq_lens, B, dev),
                 _ints("positions", positions, T, dev), _ints("slots", slots, T, dev),
                 _ints("used", used, 1, dev), B, T, _c_int(block_size), most)


def fa2_paged_append(k, v, k_cache, v_cache, slots, stream=None) -> int:
    """Raw call: k, v [T,Hkv,d], caches [blocks,Hkv,block_size,d], slots [T] int32."""
    dev, dt = _device_of(k), k.dtype
    _dtype_code(k)
    T, Hkv, d = shape = _dims("k", k, 3)
    blocks, _, bs, _ = _dims("k_cache", k_cache, 4)
    pages = (blocks, Hkv, bs, d)
    return _call(load().fa2_paged_append, dev, stream, _rows("k", k, shape, dt, dev),
                 _rows("v", v, shape, dt, dev), _pages("k_cache", k_cache, pages, dt, dev),
                 _pages("v_cache", v_cache, pages, dt, dev), _ints("slots", slots, T, dev), T, Hkv,
                 d, blocks, bs)


def fa2_get_device_status(stream=None) -> tuple[int, int]:
    """(status, wait site) of the current device; synchronises ``stream``."""
    site = ctypes.c_int(0)
    rc = load().fa2_get_device_status(_stream(stream), ctypes.byref(site))
    return rc, site.value


def fa2_debug_set(fault: int, wait_limit_ms: int = 0) -> None:
    load().fa2_debug_set(int(fault), int(wait_limit_ms))


def fa2_debug_set_bwd_grid(max_ctas: int) -> None:
    """Test hook: cap the backward's persistent grid (0 = one CTA per SM)."""
    load().fa2_debug_set_bwd_grid(int(max_ctas))


def fa2_debug_set_fwd_tiles(tiles: int) -> None:
    """Test hook: force 1 or 2 query tiles per forward CTA (0 = the library's choice)."""
    load().fa2_debug_set_fwd_tiles(int(tiles))


def fa2_launch_count() -> int:
    return int(load().fa2_launch_count())


# ------------------------------------------------------------------------------------
# allocating conveniences (PyTorch owns the memory)
#
# Those of the packed and paged calls allocate on the stream that they are given; to use
# or free their outputs on another one, order the two streams as for any tensor (wait_stream,
# record_stream).
# ------------------------------------------------------------------------------------

def forward(q, k, v, scale: float, causal: bool, stream=None):
    """Allocates O and LSE, calls fa2_fwd, raises FA2Error on a bad status."""
    B, H, N, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    rc = fa2_fwd(q, k, v, o, lse, scale, causal, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd")
    return o, lse


def forward_fp8(q, k, v, scale: float, causal: bool, q_scale: float, k_scale: float,
                v_scale: float, stream=None):
    """Allocating wrapper of fa2_fwd_fp8: bf16 O and float32 LSE."""
    B, H, N, d = q.shape
    o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    rc = fa2_fwd_fp8(q, k, v, o, lse, scale, causal, q_scale, k_scale, v_scale, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_fp8")
    return o, lse


def forward_window(q, k, v, scale: float, window: int, stream=None):
    """Allocating wrapper of fa2_fwd_window."""
    B, H, N, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    rc = fa2_fwd_window(q, k, v, o, lse, scale, window, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_window")
    return o, lse


def forward_decode(q, k, v, scale: float, causal: bool, n_splits: int = 0, stream=None):
    """Allocating wrapper of fa2_fwd_decode: q [B,H,Nq,d] against k, v [B,H,Nk,d].

    ``n_splits`` = 0 takes the library's choice for the current device.
    """
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if n_splits == 0:
        n_splits = fa2_fwd_decode_splits(B, H, Nq, Nk, d)
        if n_splits == 0:
            raise FA2Error(FA2_ERR_INVALID_ARG, "fa2_fwd_decode_splits")
    ws = fa2_fwd_decode_workspace_size(B, H, Nq, Nk, d, n_splits)
    workspace = torch.empty(ws, dtype=torch.uint8, device=q.device) if ws else None
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    rc = fa2_fwd_decode(q, k, v, o, lse, scale, causal, n_splits, workspace, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_decode")
    return o, lse


def backward_window(q, k, v, o, do, lse, scale: float, window: int, stream=None):
    """Allocating wrapper of fa2_bwd_window."""
    B, H, N, d = q.shape
    workspace = torch.empty(fa2_bwd_workspace_size(B, H, N, d), dtype=torch.uint8,
                            device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    rc = fa2_bwd_window(q, k, v, o, do, lse, dq, dk, dv, workspace, scale, window, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_bwd_window")
    return dq, dk, dv


def backward(q, k, v, o, do, lse, scale: float, causal: bool, workspace=None, stream=None,
             deterministic: bool = False, window: int = 0):
    """Allocates dQ, dK, dV (and the workspace if not given), calls fa2_bwd, or
    fa2_bwd_ex when ``deterministic`` or a ``window`` is asked for."""
    B, H, N, d = q.shape
    flags = FA2_BWD_DETERMINISTIC if deterministic else 0
    if workspace is None:
        workspace = torch.empty(fa2_bwd_ex_workspace_size(B, H, N, d, flags), dtype=torch.uint8,
                                device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if flags or window:
        rc = fa2_bwd_ex(q, k, v, o, do, lse, dq, dk, dv, workspace, scale, causal, window, flags,
                        stream)
        where = "fa2_bwd_ex"
    else:
        rc = fa2_bwd(q, k, v, o, do, lse, dq, dk, dv, workspace, scale, causal, stream)
        where = "fa2_bwd"
    if rc != FA2_OK:
        raise FA2Error(rc, where)
    return dq, dk, dv


def forward_varlen(q, k, v, cu_seqlens, scale: float, causal: bool, window: int = 0, stream=None):
    """Attention over packed sequences: O [T,H,d] and LSE [H,T] of q [T,H,d] and k, v
    [T,Hkv,d], sequence b being rows cu_seqlens[b] .. cu_seqlens[b+1] - 1.  Rows behind
    the last sequence are not written (fa2_fwd_varlen takes outputs of your own)."""
    T, H, d = _dims("q", q, 3)
    with _home(q, stream):
        o = q.new_empty((T, H, d))
        lse = q.new_empty((H, T), dtype=torch.float32)
    rc = fa2_fwd_varlen(q, k, v, o, lse, cu_seqlens, scale, causal, window, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_varlen")
    return o, lse


def backward_varlen(q, k, v, o, do, lse, cu_seqlens, scale: float, causal: bool, window: int = 0,
                    workspace=None, stream=None):
    """Gradients dQ [T,H,d], dK and dV [T,Hkv,d] of forward_varlen; the workspace is
    allocated if not given."""
    T, H, d = _dims("q", q, 3)
    Hkv = _dims("k", k, 3)[1]
    with _home(q, stream):
        if workspace is None:
            n = fa2_bwd_varlen_workspace_size(cu_seqlens.numel() - 1, T, H, Hkv, d)
            workspace = q.new_empty(n, dtype=torch.uint8)
        dq = q.new_empty((T, H, d))
        dk, dv = q.new_empty((T, Hkv, d)), q.new_empty((T, Hkv, d))
    rc = fa2_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens, workspace, scale, causal,
                        window, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_bwd_varlen")
    return dq, dk, dv


@functools.lru_cache(maxsize=None)
def _sm_count(dev: int) -> int:
    return torch.cuda.get_device_properties(dev).multi_processor_count


def forward_paged(q, k_cache, v_cache, block_table, cu_seqlens, seq_lens, scale: float,
                  causal: bool, window: int = 0, workspace=None, stream=None):
    """Attention of a step's new tokens q [T,H,d] over paged caches
    [blocks,Hkv,block_size,d]: O [T,H,d] and LSE [H,T].  The workspace is allocated if
    not given."""
    T, H, d = _dims("q", q, 3)
    B, Hkv = _dims("block_table", block_table, 2)[0], _dims("k_cache", k_cache, 4)[1]
    with _home(q, stream):
        if workspace is None:
            n = fa2_fwd_paged_workspace_size(B, T, H, Hkv, d, _sm_count(_device_of(q)))
            workspace = q.new_empty(n, dtype=torch.uint8)
        o = q.new_empty((T, H, d))
        lse = q.new_empty((H, T), dtype=torch.float32)
    rc = fa2_fwd_paged(q, k_cache, v_cache, o, lse, block_table, cu_seqlens, seq_lens, workspace,
                       scale, causal, window, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_fwd_paged")
    return o, lse


def paged_tables(context_lens, new_lens, free_blocks, block_table, T: int, block_size: int,
                 stream=None):
    """Tables of a step of at most T new tokens: (block_table, updated in place,
    cu_seqlens [B+1], seq_lens [B], positions [T], slots [T], used [1])."""
    B = _dims("block_table", block_table, 2)[0]
    empty = block_table.new_empty
    with _home(block_table, stream):
        cu, lens, positions, slots, used = empty(B + 1), empty(B), empty(T), empty(T), empty(1)
    rc = fa2_paged_tables(context_lens, new_lens, free_blocks, block_table, cu, lens, positions,
                          slots, used, block_size, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_paged_tables")
    return block_table, cu, lens, positions, slots, used


def paged_append(k, v, k_cache, v_cache, slots, stream=None):
    """Writes k, v [T,Hkv,d] into the caches by slot; returns the caches."""
    rc = fa2_paged_append(k, v, k_cache, v_cache, slots, stream)
    if rc != FA2_OK:
        raise FA2Error(rc, "fa2_paged_append")
    return k_cache, v_cache
