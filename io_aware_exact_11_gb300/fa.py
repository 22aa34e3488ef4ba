"""ctypes binding for libfa.so (the C ABI in include/fa.h).

Argument marshalling only: tensors are passed as raw device pointers plus
sizes and strides, on the caller's current CUDA stream.  PyTorch provides
device memory and streams; every step of the computation runs in the
library's CUDA kernels.  If libfa.so has not been built this module raises,
there is no fallback path.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_DEVICE_TIMEOUT = range(5)
FA_BF16, FA_FP32, FA_E4M3, FA_E2M1 = 0, 1, 2, 3
FA_MASK_NONE, FA_MASK_CAUSAL = 0, 1
FA_ROPE_HALF, FA_ROPE_INTERLEAVED = 0, 1

EXPORTED = (
    "fa_abi_version",
    "fa_forward",
    "fa_forward_masked",
    "fa_forward_fp8",
    "fa_forward_host_workspace_size",
    "fa_forward_host",
    "fa_decode_choose_splits",
    "fa_decode_workspace_size",
    "fa_decode_splitkv",
    "fa_decode_splitkv_gqa",
    "fa_decode_paged",
    "fa_decode_splitkv_noalloc",
    "fa_backward_workspace_size",
    "fa_backward",
    "fa_backward_masked",
    "fa_rope",
    "fa_rope_axes",
    "fa_cache_append",
    "fa_cache_gather",
    "fa_cache_compact",
    "fa_cache_copy_pages",
    "fa_pages_fork",
    "fa_pages_free",
    "fa_pages_reserve_workspace_size",
    "fa_pages_reserve",
    "fa_decode_tree_workspace_size",
    "fa_decode_tree",
    "fa_device_status",
    "fa_watchdog_selftest",
    "fa_status_string",
    "fa_get_last_error",
    "fa_launch_count",
)


class FAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[status {status}] {message}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Open libfa.so once (raises FileNotFoundError if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FileNotFoundError(
                f"{LIB_PATH} is missing: build it with `python -m io_aware_exact_11_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.fa_abi_version.restype = i32
        L.fa_forward.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, vp]
        L.fa_forward.restype = i32
        L.fa_forward_masked.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, i32, vp]
        L.fa_forward_masked.restype = i32
        L.fa_forward_fp8.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, f32, f32, f32, i32, vp]
        L.fa_forward_fp8.restype = i32
        L.fa_forward_host_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        L.fa_forward_host_workspace_size.restype = sz
        L.fa_forward_host.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, i32, vp, sz, vp]
        L.fa_forward_host.restype = i32
        L.fa_decode_choose_splits.argtypes = [i32, i32, i32, i32]
        L.fa_decode_choose_splits.restype = i32
        L.fa_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        L.fa_decode_workspace_size.restype = sz
        L.fa_decode_splitkv.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp]
        L.fa_decode_splitkv.restype = i32
        L.fa_decode_splitkv_gqa.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp]
        L.fa_decode_splitkv_gqa.restype = i32
        L.fa_decode_paged.argtypes = [vp] * 7 + [i32] * 8 + [f32, i32, vp, sz, vp]
        L.fa_decode_paged.restype = i32
        L.fa_backward_workspace_size.argtypes = [i32, i32, i32, i32]
        L.fa_backward_workspace_size.restype = sz
        L.fa_backward.argtypes = [vp] * 9 + [i32, i32, i32, i32, i32, f32, vp, sz, vp]
        L.fa_backward.restype = i32
        L.fa_backward_masked.argtypes = [vp] * 9 + [i32, i32, i32, i32, i32, f32, vp, sz, i32, vp]
        L.fa_backward_masked.restype = i32
        L.fa_rope.argtypes = [vp] * 4 + [i32] * 7 + [vp, vp, ctypes.c_int64, i32, vp, f32, i32, i32, vp]
        L.fa_rope.restype = i32
        L.fa_rope_axes.argtypes = [vp] * 4 + [i32] * 7 + [vp, vp, i32, ctypes.c_int64, ctypes.c_int64, vp, vp, f32, i32, i32, vp]
        L.fa_rope_axes.restype = i32
        L.fa_cache_append.argtypes = [vp] * 9 + [i32] * 8 + [vp, vp]
        L.fa_cache_append.restype = i32
        L.fa_cache_gather.argtypes = [vp] * 8 + [i32] * 8 + [vp, vp]
        L.fa_cache_gather.restype = i32
        L.fa_cache_compact.argtypes = [vp] * 7 + [ctypes.c_int64, vp] + [i32] * 8 + [vp]
        L.fa_cache_compact.restype = i32
        L.fa_cache_copy_pages.argtypes = [vp] * 6 + [i32] * 6 + [vp]
        L.fa_cache_copy_pages.restype = i32
        L.fa_pages_fork.argtypes = [vp] * 5 + [i32] * 5 + [vp]
        L.fa_pages_fork.restype = i32
        L.fa_pages_free.argtypes = [vp] * 5 + [i32] * 5 + [vp]
        L.fa_pages_free.restype = i32
        L.fa_pages_reserve_workspace_size.argtypes = [i32, i32]
        L.fa_pages_reserve_workspace_size.restype = sz
        L.fa_pages_reserve.argtypes = [vp] * 7 + [i32] * 4 + [vp, sz, vp]
        L.fa_pages_reserve.restype = i32
        L.fa_decode_tree_workspace_size.argtypes = [i32] * 6
        L.fa_decode_tree_workspace_size.restype = sz
        L.fa_decode_tree.argtypes = [vp] * 9 + [ctypes.c_int64, vp, vp] + [i32] * 9 + [f32, vp, i32, vp, sz, vp]
        L.fa_decode_tree.restype = i32
        L.fa_device_status.argtypes = [vp]
        L.fa_device_status.restype = i32
        L.fa_watchdog_selftest.argtypes = [vp]
        L.fa_watchdog_selftest.restype = i32
        L.fa_status_string.argtypes = [i32]
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_get_last_error.restype = ctypes.c_char_p
        L.fa_launch_count.restype = ctypes.c_uint64
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != FA_OK:
        msg = lib().fa_get_last_error().decode(errors="replace")
        raise FAError(status, msg or lib().fa_status_string(status).decode())


def _torch():
    import torch
    return torch


def _stream_ptr(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float32:
        return FA_FP32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _check_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must live on a CUDA device")


def launch_count() -> int:
    """Kernels the library has enqueued since it was loaded."""
    return int(lib().fa_launch_count())


def device_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel's bounded wait gave up."""
    _check(lib().fa_device_status(_stream_ptr(stream)))


def watchdog_selftest(stream=None) -> None:
    """Enqueue a kernel whose bounded wait runs out (~1 s); the next
    device_status() raises FAError with FA_ERR_DEVICE_TIMEOUT."""
    _check(lib().fa_watchdog_selftest(_stream_ptr(stream)))


def forward(q, k, v, scale: float | None = None, out=None, lse=None, return_lse: bool = True, stream=None,
            causal: bool = False):
    """Exact attention forward.  q [B,H,Nq,d], k/v [B,H,Nkv,d] (bf16 or fp32).

    Returns (O, LSE) with O like q and LSE fp32 [B,H,Nq].  Non-contiguous
    inputs are passed by stride (d must be the contiguous dim).  ``causal``
    masks keys j > i + Nkv − Nq for query row i.
    """
    torch = _torch()
    _check_cuda(q, k, v)
    B, H, Nq, d = q.shape
    Nkv = k.shape[2]
    if k.shape != (B, H, Nkv, d) or v.shape != (B, H, Nkv, d):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, H, Nq, d), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
        for t in (q, k, v, out):
            if t.stride(3) != 1:
                raise ValueError("the head dim must be contiguous")
        arr = (ctypes.c_int64 * 12)(*[int(t.stride(i)) for t in (q, k, v, out) for i in range(3)])
        strides = ctypes.cast(arr, ctypes.c_void_p)
    if causal:
        _check(lib().fa_forward_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Nq, Nkv, d,
                                       _dtype_code(q), float(scale), strides, FA_MASK_CAUSAL, _stream_ptr(stream)))
    else:
        _check(lib().fa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Nq, Nkv, d,
                                _dtype_code(q), float(scale), strides, _stream_ptr(stream)))
    return out, lse


_host_ws = {}
_host_ws_lock = threading.Lock()


def forward_host(q, k, v, scale: float | None = None, out=None, lse=None, causal: bool = False,
                 heads_per_chunk: int = 0, device=None, stream=None):
    """Forward on host tensors: q [B,H,Nq,d], k/v [B,H,Nkv,d] contiguous CPU
    tensors (bf16 or fp32; page-locked ones let the copies overlap).  The
    library streams (b, h) chunks through a device workspace, overlapping the
    copies in and out with the forward.  Returns (O, LSE) as CPU tensors
    (page-locked when allocated here); they are valid once ``stream`` (default:
    the device's current stream) has been synchronised.  The workspace is cached
    per device and shared: eager calls from several threads or streams are
    ordered by the library, while a call captured in a CUDA graph is not, so
    replays must not overlap other calls on that device."""
    torch = _torch()
    for t in (q, k, v):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("forward_host takes contiguous CPU tensors")
    B, H, Nq, d = q.shape
    Nkv = k.shape[2]
    if k.shape != (B, H, Nkv, d) or v.shape != (B, H, Nkv, d):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, H, Nq, d), dtype=q.dtype, pin_memory=True)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, pin_memory=True)
    for t in (out, lse):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("out and lse must be contiguous CPU tensors")
    code = _dtype_code(q)
    with torch.cuda.device(dev):
        need = int(lib().fa_forward_host_workspace_size(B, H, Nq, Nkv, d, code, int(heads_per_chunk)))
        if need == 0:
            raise FAError(FA_ERR_INVALID_ARG, "fa_forward_host_workspace_size rejected the arguments")
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        # One cached workspace per device, shared by all threads and streams:
        # the library orders the calls that use it, and record_stream keeps the
        # caching allocator from handing it out again while a call on another
        # stream may still read it after it has been replaced by a larger one.
        with _host_ws_lock:
            ws = _host_ws.get(dev.index)
            if ws is None or ws.numel() < need:
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
                _host_ws[dev.index] = ws
            _check(lib().fa_forward_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Nq, Nkv, d, code,
                                         float(scale), FA_MASK_CAUSAL if causal else FA_MASK_NONE,
                                         int(heads_per_chunk), _ptr(ws), ws.numel(), _stream_ptr(s)))
            ws.record_stream(s)
    return out, lse


def forward_fp8(q8, k8, v8, q_descale: float = 1.0, k_descale: float = 1.0, v_descale: float = 1.0,
                scale: float | None = None, out=None, lse=None, causal: bool = False, stream=None):
    """FP8 forward.  q8/k8/v8: uint8 tensors of E4M3 codes [B,H,N,d] (or torch
    float8_e4m3fn); true values are descale × code value.  Returns (O bf16, LSE)."""
    torch = _torch()
    _check_cuda(q8, k8, v8)
    B, H, Nq, d = q8.shape
    Nkv = k8.shape[2]
    for t in (q8, k8, v8):
        if t.element_size() != 1 or not t.is_contiguous():
            raise ValueError("fp8 inputs must be contiguous one-byte tensors")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, H, Nq, d), dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q8.device)
    _check(lib().fa_forward_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(out), _ptr(lse), B, H, Nq, Nkv, d, float(scale),
                                float(q_descale), float(k_descale), float(v_descale),
                                FA_MASK_CAUSAL if causal else FA_MASK_NONE, _stream_ptr(stream)))
    return out, lse


def decode_workspace_size(B: int, H: int, d: int, n_splits: int) -> int:
    return int(lib().fa_decode_workspace_size(B, H, d, n_splits))


def choose_splits(B: int, Hq: int, Hkv: int, Nkv: int) -> int:
    """The library's split count for a decode shape (fa_decode_choose_splits)."""
    s = int(lib().fa_decode_choose_splits(B, Hq, Hkv, Nkv))
    if s <= 0:
        raise FAError(FA_ERR_INVALID_ARG, f"no split count for B={B} Hq={Hq} Hkv={Hkv} Nkv={Nkv}")
    return s


def _check_decode_kv(q, k, v) -> int:
    """k and v must be [B, H, N_kv, d] like q's B, H, d and share its dtype; returns N_kv."""
    B, H, _, d = q.shape
    if k.dim() != 4 or tuple(k.shape[:2]) != (B, H) or k.shape[3] != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("decode inputs must be contiguous")
    return int(k.shape[2])


def decode_splitkv(q, k, v, n_splits: int | None = None, scale: float | None = None, out=None, lse=None,
                   workspace=None, stream=None):
    """Split-KV decode: q [B,H,1,d] against k/v [B,H,Nkv,d]; returns (O, LSE).
    n_splits=None takes the library's choice for the shape."""
    torch = _torch()
    _check_cuda(q, k, v)
    B, H, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes one query row per head")
    Nkv = _check_decode_kv(q, k, v)
    if n_splits is None:
        n_splits = choose_splits(B, H, H, Nkv)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, H, 1, d), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    need = decode_workspace_size(B, H, d, n_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(lib().fa_decode_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Nkv, d,
                                   _dtype_code(q), float(scale), int(n_splits), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream_ptr(stream)))
    return out, lse


def decode_splitkv_gqa(q, k, v, n_splits: int | None = None, scale: float | None = None, out=None, lse=None,
                       workspace=None, stream=None):
    """Grouped-query split-KV decode: q [B,Hq,1,d], k/v [B,Hkv,Nkv,d], Hq = G·Hkv (G <= 128).
    n_splits=None takes the library's choice for the shape."""
    torch = _torch()
    _check_cuda(q, k, v)
    B, Hq, one, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    if one != 1:
        raise ValueError("decode takes one query row per head")
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("decode inputs must be contiguous")
    if n_splits is None:
        n_splits = choose_splits(B, Hq, Hkv, Nkv)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, 1, d), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = decode_workspace_size(B, Hq, d, n_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(lib().fa_decode_splitkv_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Nkv, d,
                                       _dtype_code(q), float(scale), int(n_splits), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream_ptr(stream)))
    return out, lse


def decode_paged(q, k_cache, v_cache, block_table, seq_lens, n_splits: int | None = None,
                 scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """Split-KV decode over a paged cache.

    q [B,Hq,1,d]; k_cache/v_cache [num_blocks, Hkv, block_size, d]; block_table
    [B, max_blocks] int32; seq_lens [B] int32 (device tensors).  n_splits=None
    takes the library's choice for the longest sequence the table can hold.
    """
    torch = _torch()
    _check_cuda(q, k_cache, v_cache, block_table, seq_lens)
    B, Hq, one, d = q.shape
    NB, Hkv, bs, d2 = k_cache.shape
    if one != 1 or d2 != d or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("shape mismatch")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    for t in (q, k_cache, v_cache, block_table, seq_lens):
        if not t.is_contiguous():
            raise ValueError("paged decode inputs must be contiguous")
    if n_splits is None:
        n_splits = choose_splits(B, Hq, Hkv, block_table.shape[1] * bs)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, 1, d), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = decode_workspace_size(B, Hq, d, n_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(lib().fa_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens), _ptr(out),
                                 _ptr(lse), B, Hq, Hkv, NB, bs, block_table.shape[1], d, _dtype_code(q), float(scale),
                                 int(n_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream)))
    return out, lse


DECODE_STATIC_SCRATCH_BYTES = 36 << 20


def decode_splitkv_noalloc(q, k, v, n_splits: int = 32, scale: float | None = None, out=None, lse=None,
                           return_lse: bool = True, stream=None):
    """Split-KV decode whose scratch is the library's fixed 36 MiB buffer.

    For callers that cannot provide device workspace (no allocator at decode
    time).  The library allocates nothing; `out` and `lse` are allocated here
    only when not given (with ``return_lse=False`` and no `lse`, the library
    writes no LSE and None is returned for it).  Calls overlapping on the GPU
    race on the buffer.
    """
    torch = _torch()
    _check_cuda(q, k, v)
    L = lib()
    fn = L.fa_decode_splitkv_noalloc
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    fn.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp]
    fn.restype = i32
    B, H, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes one query row per head")
    Nkv = _check_decode_kv(q, k, v)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, H, 1, d), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Nkv, d, _dtype_code(q), float(scale),
              int(n_splits), _stream_ptr(stream)))
    return out, lse


def backward_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(lib().fa_backward_workspace_size(B, H, N, d))


def backward(q, k, v, o, lse, do, scale: float | None = None, dq=None, dk=None, dv=None,
             workspace=None, stream=None, causal: bool = False):
    """Gradients (dQ, dK, dV) from the saved O and LSE; all [B,H,N,d] contiguous.

    ``causal`` must match the forward that produced O and LSE.
    """
    torch = _torch()
    _check_cuda(q, k, v, o, lse, do)
    B, H, N, d = q.shape
    for t in (q, k, v, o, do):
        if tuple(t.shape) != (B, H, N, d) or not t.is_contiguous():
            raise ValueError("backward tensors must be contiguous [B,H,N,d]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = backward_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d,
            _dtype_code(q), float(scale), _ptr(workspace), workspace.numel() * workspace.element_size())
    if causal:
        _check(lib().fa_backward_masked(*args, FA_MASK_CAUSAL, _stream_ptr(stream)))
    else:
        _check(lib().fa_backward(*args, _stream_ptr(stream)))
    return dq, dk, dv


# ---------------------------------------------------------------- rotary positions, paged cache, drafted tokens
#
# These calls run on the tensors' own device.  Without ``stream`` they use that
# device's current stream; with one, what they allocate belongs to that stream.
# At single tokens the host side is most of a call's time, so it does little: one
# look at the device, no contexts in the common case, plain integers to ctypes.


def _device_of(*ts) -> int:
    """Index of the one CUDA device that the given tensors live on (None entries are skipped)."""
    dev = None
    for t in ts:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if i < 0:
                    raise ValueError("all tensors must live on a CUDA device")
                if dev is not None:
                    raise ValueError("all tensors must live on the same CUDA device")
                dev = i
    return dev


def _elsewhere(dev: int, stream):
    """None where ``dev`` is the current device and its current stream is wanted; else a context in which that is so."""
    torch = _torch()
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        return torch.cuda.stream(stream)
    if dev != torch.cuda.current_device():
        return torch.cuda.device(dev)
    return None


def _current_stream(dev: int) -> int:
    """Handle of the device's current stream."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _addr(t):
    return t.data_ptr() if t is not None else None


_pack6, _pack12 = struct.Struct("=6q").pack, struct.Struct("=12q").pack


def _strides(*ts):
    """Element strides of all but the last dimension (which must be contiguous) as the bytes of int64 values, or None if
    all are contiguous."""
    for t in ts:
        if not t.is_contiguous():
            break
    else:
        return None
    st = []
    for t in ts:
        x = t.stride()
        if x[-1] != 1 and t.shape[-1] > 1:
            raise ValueError("the head dim must be contiguous")
        st += x[:-1]
    return (_pack6 if len(st) == 6 else _pack12)(*st)


def _check_out(name, t, shape, dtype, dev):
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 4096, low_turns: float = 1.0, high_turns: float = 32.0):
    """Inverse frequencies for ``rope`` (float64 array of rot_dim/2) and the magnitude that goes with them.

    w_i = base^(−2i/rot_dim), stretched for contexts ``factor`` times as long:
      * ``"linear"``: every w_i divided by factor (positions interpolated);
      * ``"base"``: base multiplied by factor^(rot_dim/(rot_dim − 2)), which leaves the fastest pair alone and
        divides the slowest by factor;
      * ``"ramp"``: pairs that make at least ``high_turns`` turns over ``original_len`` positions are left alone,
        those with at most ``low_turns`` divided by factor, a straight line between; magnitude 0.1·ln(factor) + 1.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor >= 1):
        raise ValueError("base must be > 0 and factor >= 1")
    if scaling not in ("none", "linear", "base", "ramp"):
        raise ValueError(f"unknown scaling {scaling!r} (none, linear, base, ramp)")
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("scaling 'base' needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    w = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "ramp":
        if not (original_len > 0 and 0 <= low_turns < high_turns):
            raise ValueError("ramp needs original_len > 0 and 0 <= low_turns < high_turns")
        keep = np.clip((original_len * w / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0.0, 1.0)
        return w * keep + w / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return w, 1.0


def _rope(q, k, inv_freq, positions, position0, magnitude, interleaved, out_q, out_k, stream, inverse, axes=None):
    torch = _torch()
    dev = _device_of(q, k, positions, out_q, out_k)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return _rope(q, k, inv_freq, positions, position0, magnitude, interleaved, out_q, out_k, None, inverse, axes)
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q must be [B, Hq, N, d] and k [B, Hk, N, d]")
    B, Hq, N, d = q.shape
    code = _dtype_code(q)
    Hk = 0
    if k is not None:
        if k.dtype != q.dtype:
            raise TypeError("q and k must share a dtype")
        Bk, Hk, Nk, dk = k.shape
        if Bk != B or Nk != N or dk != d:
            raise ValueError("q must be [B, Hq, N, d] and k [B, Hk, N, d]")
    elif out_k is not None:
        raise ValueError("out_k without k")
    if isinstance(inv_freq, torch.Tensor) and inv_freq.dtype == torch.float64 and not inv_freq.is_cuda:
        w = inv_freq.contiguous()
        w_ptr = w.data_ptr()
    else:
        w = np.ascontiguousarray(inv_freq, dtype=np.float64)
        w_ptr = w.tobytes()  # a copy costs less than the array's address
    if w.ndim != 1:
        raise ValueError("inv_freq must be one row of rot_dim/2 values")
    pos_ptr, pos_sb = None, 0
    if axes is not None:
        if positions is None or positions.dtype != torch.int32:
            raise TypeError("positions must be int32")
        shape, step = positions.shape, positions.stride()
        if len(shape) not in (2, 3) or shape[1:] != (B, N)[3 - len(shape):] or (N > 1 and step[-1] != 1):
            raise ValueError("positions must be [axes, N] or [axes, B, N] with the last dim contiguous")
        if isinstance(axes, torch.Tensor) and axes.dtype == torch.int32 and not axes.is_cuda:
            a = axes.contiguous()
            a_ptr = a.data_ptr()
        else:
            a = np.asarray(axes)
            if a.dtype != np.int32:
                if a.dtype.kind not in "iu" or a.size and not 0 <= a.min() <= a.max() < 1 << 31:
                    raise ValueError("axes must be whole numbers, one for each of inv_freq's pairs")
                a = a.astype(np.int32)
            a_ptr = a.tobytes()
        if a.shape != w.shape:
            raise ValueError("axes must name one axis for each of inv_freq's pairs")
        pos_ptr = positions.data_ptr()
        pos_sa = step[0] if shape[0] > 1 else 0
        pos_sb = step[1] if len(shape) == 3 and B > 1 else 0
    elif positions is not None:
        if positions.dtype != torch.int32:
            raise TypeError("positions must be int32")
        shape = positions.shape
        if shape != (B, N) and shape != (N,) or (N > 1 and positions.stride(-1) != 1):
            raise ValueError("positions must be [N] or [B, N] with the last dim contiguous")
        pos_ptr = positions.data_ptr()
        pos_sb = positions.stride(0) if len(shape) == 2 and B > 1 else 0
    if out_q is None:
        out_q = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _check_out("out_q", out_q, q.shape, q.dtype, dev)
    if k is None:
        st = _strides(q, q, out_q, out_q)
    else:
        if out_k is None:
            out_k = torch.empty_like(k, memory_format=torch.contiguous_format)
        else:
            _check_out("out_k", out_k, k.shape, q.dtype, dev)
        st = _strides(q, k, out_q, out_k)
    if axes is not None:
        status = lib().fa_rope_axes(q.data_ptr(), _addr(k), out_q.data_ptr(), _addr(out_k), B, Hq, Hk, N, d,
                                    2 * w.shape[0], code, st, pos_ptr, shape[0], pos_sa, pos_sb, a_ptr, w_ptr,
                                    float(magnitude), FA_ROPE_INTERLEAVED if interleaved else FA_ROPE_HALF, inverse,
                                    _current_stream(dev))
        if status:
            _check(status)
        return out_q, out_k
    if not -(1 << 31) <= position0 < 1 << 31:
        raise ValueError("position0 must be an int32")
    status = lib().fa_rope(q.data_ptr(), _addr(k), out_q.data_ptr(), _addr(out_k), B, Hq, Hk, N, d, 2 * w.shape[0],
                           code, st, pos_ptr, pos_sb, int(position0), w_ptr, float(magnitude),
                           FA_ROPE_INTERLEAVED if interleaved else FA_ROPE_HALF, inverse, _current_stream(dev))
    if status:
        _check(status)
    return out_q, out_k


def rope(q, k, inv_freq, positions=None, position0: int = 0, magnitude: float = 1.0, interleaved: bool = False,
         out_q=None, out_k=None, stream=None):
    """Rotary positions of q [B,Hq,N,d] and k [B,Hk,N,d] (k may be None), bf16 or fp32; returns (q', k').

    Pair i of the first 2·len(inv_freq) elements turns by position·inv_freq[i] and is multiplied by ``magnitude``;
    pairs are (i, i + rot/2), or (2i, 2i + 1) with ``interleaved``.  ``positions`` is int32 [N] or [B, N] on the
    device (None: 0 … N − 1), ``position0`` is added to it.  Strided inputs and outputs are taken as they are (the
    head dim contiguous); ``out_q=q, out_k=k`` works in place.
    """
    return _rope(q, k, inv_freq, positions, position0, magnitude, interleaved, out_q, out_k, stream, 0)


def rope_backward(dq, dk, inv_freq, positions=None, position0: int = 0, magnitude: float = 1.0,
                  interleaved: bool = False, out_q=None, out_k=None, stream=None):
    """Gradients of ``rope``'s inputs from those of its outputs; same arguments as the forward call."""
    return _rope(dq, dk, inv_freq, positions, position0, magnitude, interleaved, out_q, out_k, stream, 1)


def rope_axes(q, k, inv_freq, axes, positions, magnitude: float = 1.0, interleaved: bool = False, out_q=None,
              out_k=None, stream=None):
    """Rotary positions with several axes (time, height and width of a patch, say); returns (q', k').

    As ``rope``, with a position on each of up to four axes per token: ``positions`` is int32 [axes, N] or [axes, B, N] on
    the device, and pair i turns by positions[axes[i]]·inv_freq[i].  ``axes`` (on the host, one number per pair) may give
    each axis a block of pairs or take turns.
    """
    return _rope(q, k, inv_freq, positions, 0, magnitude, interleaved, out_q, out_k, stream, 0, axes)


def rope_axes_backward(dq, dk, inv_freq, axes, positions, magnitude: float = 1.0, interleaved: bool = False, out_q=None,
                       out_k=None, stream=None):
    """Gradients of ``rope_axes``'s inputs from those of its outputs; same arguments as the forward call."""
    return _rope(dq, dk, inv_freq, positions, 0, magnitude, interleaved, out_q, out_k, stream, 1, axes)


E2M1_GROUP = 32  # elements of a row that share a scale byte


def _cache_args(k_cache, v_cache, k_scale, v_scale, block_table):
    """Checks a paged cache; returns (num_blocks, Hkv, block_size, d, dtype code).  One-byte elements are E4M3 codes, or,
    where the scales have a fourth dimension, pairs of E2M1 codes."""
    torch = _torch()
    shape, dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [num_blocks, Hkv, block_size, d]")
    if v_cache.dtype != dtype:
        raise TypeError("k_cache and v_cache must share a dtype")
    contiguous = k_cache.is_contiguous() and v_cache.is_contiguous() and (block_table is None or block_table.is_contiguous())
    if dtype == torch.bfloat16:
        code = FA_BF16
    elif dtype == torch.uint8 and k_scale is not None and k_scale.dim() == 4:
        code = FA_E2M1
        shape = (*shape[:3], 2 * shape[3])
        for s in (k_scale, v_scale):
            if s is None or s.dtype != torch.uint8 or s.shape != (*shape[:3], shape[3] // E2M1_GROUP):
                raise ValueError("an E2M1 cache needs uint8 k_scale and v_scale [num_blocks, Hkv, block_size, d/32]")
            contiguous = contiguous and s.is_contiguous()
    elif dtype == torch.float8_e4m3fn or dtype == torch.uint8:
        code = FA_E4M3
        for s in (k_scale, v_scale):
            if s is None or s.dtype != torch.uint8 or s.shape != shape[:3]:
                raise ValueError("an E4M3 cache needs uint8 k_scale and v_scale [num_blocks, Hkv, block_size]")
            contiguous = contiguous and s.is_contiguous()
    else:
        raise TypeError(f"unsupported cache dtype {dtype} (bfloat16, float8_e4m3fn or uint8 codes)")
    if block_table is not None and (block_table.dtype != torch.int32 or block_table.dim() != 2):
        raise TypeError("block_table must be int32 [B, max_blocks]")
    if not contiguous:
        raise ValueError("caches, scales and block_table must be contiguous")
    return *shape, code


def _check_lens(name, t, B):
    torch = _torch()
    if t.dtype != torch.int32 or t.shape != (B,) or not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous int32 [{B}]")


def cache_append(k, v, k_cache, v_cache, block_table, start, new_lens=None, k_scale=None, v_scale=None, stream=None):
    """Write new keys and values k, v (bf16 [B,Hkv,N,d], strided or not) into a paged cache, in place.

    Token n of sequence b goes to logical position start[b] + n (start: int32 [B]); with ``new_lens`` (int32 [B]) only
    the first new_lens[b] are written.  k_cache/v_cache [num_blocks, Hkv, block_size, d]: bfloat16 takes the rows as
    they are; float8_e4m3fn (or uint8 codes) quantises each row with the power of two whose E8M0 byte goes to
    k_scale/v_scale (uint8 [num_blocks, Hkv, block_size]); uint8 [num_blocks, Hkv, block_size, d/2] with scales
    [num_blocks, Hkv, block_size, d/32] holds E2M1 codes, two to a byte, with a power of two for every 32 elements.
    """
    torch = _torch()
    dev = _device_of(k, v, k_cache, v_cache, block_table, start, new_lens, k_scale, v_scale)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return cache_append(k, v, k_cache, v_cache, block_table, start, new_lens, k_scale, v_scale)
    nb, hkv, bs, d, code = _cache_args(k_cache, v_cache, k_scale, v_scale, block_table)
    B, max_blocks = block_table.shape
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or shape[0] != B or shape[1] != hkv or shape[3] != d:
        raise ValueError(f"k and v must be [{B}, {hkv}, N, {d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("k and v must be bfloat16")
    _check_lens("start", start, B)
    if new_lens is not None:
        _check_lens("new_lens", new_lens, B)
    status = lib().fa_cache_append(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale),
                                   _addr(v_scale), block_table.data_ptr(), start.data_ptr(), _addr(new_lens), B, hkv,
                                   shape[2], nb, bs, max_blocks, d, code, _strides(k, v),
                                   _current_stream(dev))
    if status:
        _check(status)


def cache_gather(k_cache, v_cache, block_table, seq_lens, n: int, k_scale=None, v_scale=None, out_k=None, out_v=None,
                 stream=None):
    """The first n keys and values of every sequence as bf16 [B,Hkv,n,d]; rows past seq_lens[b] are zero."""
    torch = _torch()
    dev = _device_of(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, out_k, out_v)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return cache_gather(k_cache, v_cache, block_table, seq_lens, n, k_scale, v_scale, out_k, out_v)
    nb, hkv, bs, d, code = _cache_args(k_cache, v_cache, k_scale, v_scale, block_table)
    B = block_table.shape[0]
    _check_lens("seq_lens", seq_lens, B)
    n = int(n)
    if not 1 <= n < 1 << 31:
        raise ValueError("n must be at least 1, and an int32")
    shape = (B, hkv, n, d)
    if out_k is None:
        out_k = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
    else:
        _check_out("out_k", out_k, shape, torch.bfloat16, dev)
    if out_v is None:
        out_v = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
    else:
        _check_out("out_v", out_v, shape, torch.bfloat16, dev)
    status = lib().fa_cache_gather(k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale),
                                   block_table.data_ptr(), seq_lens.data_ptr(), out_k.data_ptr(), out_v.data_ptr(), B,
                                   hkv, n, nb, bs, block_table.shape[1], d, code, _strides(out_k, out_v),
                                   _current_stream(dev))
    if status:
        _check(status)
    return out_k, out_v


def cache_compact(k_cache, v_cache, block_table, first, keep, keep_lens=None, k_scale=None, v_scale=None, stream=None):
    """Moves the kept rows of every sequence together, in place (accepted drafts, or what an eviction leaves).

    Row keep[b, i] of sequence b (a position; int32 [B,N] or [N]) goes to position first[b] + i (int32 [B]) for
    i < keep_lens[b] (int32 [B]; None: N).  keep[b, i] >= first[b] + i, in any order.  Caches and scales as for
    ``cache_append``; the pages written must not be shared with another sequence.
    """
    torch = _torch()
    dev = _device_of(k_cache, v_cache, block_table, first, keep, keep_lens, k_scale, v_scale)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return cache_compact(k_cache, v_cache, block_table, first, keep, keep_lens, k_scale, v_scale)
    nb, hkv, bs, d, code = _cache_args(k_cache, v_cache, k_scale, v_scale, block_table)
    B, max_blocks = block_table.shape
    _check_lens("first", first, B)
    if keep_lens is not None:
        _check_lens("keep_lens", keep_lens, B)
    shape = keep.shape
    if keep.dtype != torch.int32:
        raise TypeError("keep must be int32")
    if len(shape) not in (1, 2) or (len(shape) == 2 and shape[0] != B) or (shape[-1] > 1 and keep.stride(-1) != 1):
        raise ValueError(f"keep must be [N] or [{B}, N] with the last dim contiguous")
    status = lib().fa_cache_compact(k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale),
                                    block_table.data_ptr(), first.data_ptr(), keep.data_ptr(),
                                    keep.stride(0) if len(shape) == 2 and B > 1 else 0, _addr(keep_lens), B, hkv,
                                    shape[-1], nb, bs, max_blocks, d, code, _current_stream(dev))
    if status:
        _check(status)


def cache_copy_pages(k_cache, v_cache, src, dst, k_scale=None, v_scale=None, stream=None):
    """Copies whole pages within a pool, page src[i] to page dst[i] (int32 [n]; −1 in both: nothing to copy).

    No page may be written twice in one call, or written and read.
    """
    dev = _device_of(k_cache, v_cache, src, dst, k_scale, v_scale)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return cache_copy_pages(k_cache, v_cache, src, dst, k_scale, v_scale)
    nb, hkv, bs, d, code = _cache_args(k_cache, v_cache, k_scale, v_scale, None)
    n = src.shape[0] if src.dim() == 1 else -1
    _check_lens("src", src, n)
    _check_lens("dst", dst, n)
    status = lib().fa_cache_copy_pages(k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale),
                                       src.data_ptr(), dst.data_ptr(), n, hkv, nb, bs, d, code, _current_stream(dev))
    if status:
        _check(status)


def _check_pages(block_table, seq_lens, holders):
    """Checks the tables of a page pool; returns (B, max_blocks, num_blocks)."""
    torch = _torch()
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
        raise TypeError("block_table must be contiguous int32 [B, max_blocks]")
    B, max_blocks = block_table.shape
    _check_lens("seq_lens", seq_lens, B)
    nb = holders.shape[0] if holders.dim() == 1 else -1
    _check_lens("holders", holders, nb)
    return B, max_blocks, nb


def pages_fork(block_table, seq_lens, holders, src, dst, block_size: int, stream=None):
    """Sequences dst[i], empty so far, take the pages and the length of sequences src[i] (int32 [n]), in place.

    ``block_table`` int32 [B, max_blocks] (−1 where there is no page), ``seq_lens`` int32 [B] and ``holders`` int32
    [num_blocks], the number of sequences that hold each page (0: free).  Nothing is copied: who writes into a page that
    others hold gets one of its own from ``pages_reserve``.
    """
    dev = _device_of(block_table, seq_lens, holders, src, dst)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return pages_fork(block_table, seq_lens, holders, src, dst, block_size)
    B, max_blocks, nb = _check_pages(block_table, seq_lens, holders)
    n = src.shape[0] if src.dim() == 1 else -1
    _check_lens("src", src, n)
    _check_lens("dst", dst, n)
    status = lib().fa_pages_fork(block_table.data_ptr(), seq_lens.data_ptr(), holders.data_ptr(), src.data_ptr(),
                                 dst.data_ptr(), n, B, nb, block_size, max_blocks, _current_stream(dev))
    if status:
        _check(status)


def pages_free(block_table, seq_lens, holders, seqs, block_size: int, keep_lens=None, stream=None):
    """Sequences seqs[i] (int32 [n]) give up their pages, all but those of the first keep_lens[i] tokens (int32 [n]).

    In place: their entries become −1, their lengths at most keep_lens[i] (0 without), and pages that nobody holds any
    more are free.  ``keep_lens`` may be ``seq_lens`` itself where seqs[i] = i: pages reserved in vain are given back.
    """
    dev = _device_of(block_table, seq_lens, holders, seqs, keep_lens)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return pages_free(block_table, seq_lens, holders, seqs, block_size, keep_lens)
    B, max_blocks, nb = _check_pages(block_table, seq_lens, holders)
    n = seqs.shape[0] if seqs.dim() == 1 else -1
    _check_lens("seqs", seqs, n)
    if keep_lens is not None:
        _check_lens("keep_lens", keep_lens, n)
    status = lib().fa_pages_free(block_table.data_ptr(), seq_lens.data_ptr(), holders.data_ptr(), seqs.data_ptr(),
                                 _addr(keep_lens), n, B, nb, block_size, max_blocks, _current_stream(dev))
    if status:
        _check(status)


def pages_reserve_workspace_size(B: int, num_blocks: int) -> int:
    return int(lib().fa_pages_reserve_workspace_size(B, num_blocks))


def pages_reserve(block_table, seq_lens, holders, new_lens, block_size: int, workspace=None, stream=None):
    """Pages for the next new_lens[b] tokens of every sequence (int32 [B]); returns (granted, copy_src, copy_dst), int32 [B].

    Missing table entries get free pages, and an entry that the tokens go into and whose page others hold too gets one of
    its own in its place.  Where tokens of the sequence lie in it, copy_src[b] → copy_dst[b] (−1: nothing) are to be
    copied with ``cache_copy_pages`` before anything is written.  Sequences are served in order, from the free pages by rising number; from the first one that
    finds too few on, none with tokens to come is (granted[b] = 0, its table as it was).
    """
    torch = _torch()
    dev = _device_of(block_table, seq_lens, holders, new_lens, workspace)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return pages_reserve(block_table, seq_lens, holders, new_lens, block_size, workspace)
    B, max_blocks, nb = _check_pages(block_table, seq_lens, holders)
    _check_lens("new_lens", new_lens, B)
    granted, src, dst = torch.empty_like(new_lens), torch.empty_like(new_lens), torch.empty_like(new_lens)
    if workspace is None:
        workspace = torch.empty(max(pages_reserve_workspace_size(B, nb), 16), dtype=torch.uint8, device=block_table.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    status = lib().fa_pages_reserve(block_table.data_ptr(), seq_lens.data_ptr(), holders.data_ptr(), new_lens.data_ptr(),
                                    granted.data_ptr(), src.data_ptr(), dst.data_ptr(), B, nb, block_size, max_blocks,
                                    workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    _current_stream(dev))
    if status:
        _check(status)
    return granted, src, dst


def decode_tree_workspace_size(B: int, Hq: int, Hkv: int, T: int, d: int, max_parts: int = 0) -> int:
    """Workspace bytes with which ``decode_tree`` uses the whole current device (or at most ``max_parts`` CTAs)."""
    return int(lib().fa_decode_tree_workspace_size(B, Hq, Hkv, T, d, max_parts))


def decode_tree(q, k_cache, v_cache, block_table, seq_lens, tree_mask=None, draft_lens=None, k_scale=None,
                v_scale=None, max_parts: int = 0, scale: float | None = None, out=None, lse=None, workspace=None,
                stream=None):
    """Attention of T drafted tokens per sequence over a paged cache (T = 1: plain decode); returns (O, LSE).

    q [B,Hq,T,d] bf16 (strided or not).  The drafted tokens' keys are in the cache: seq_lens[b] counts them, and the
    last draft_lens[b] (int32 [B]; None: T) keys of sequence b are theirs.  Token t sees the context before them and
    drafted key u where tree_mask[b, t, u] (bool or uint8 [B,T,T] or [T,T]; None: u <= t).  Rows that see nothing,
    padding rows t >= draft_lens[b] among them, give O = 0 and LSE = −inf.  The cache is bfloat16, or E4M3 or E2M1 codes
    with k_scale/v_scale as ``cache_append`` writes them.  O like q (contiguous), LSE fp32 [B,Hq,T].  The work is cut
    into equal parts over the machine (at most ``max_parts``, 0: no limit), fewer where a given workspace is small.
    """
    torch = _torch()
    dev = _device_of(q, k_cache, v_cache, block_table, seq_lens, tree_mask, draft_lens, k_scale, v_scale, out, lse,
                     workspace)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return decode_tree(q, k_cache, v_cache, block_table, seq_lens, tree_mask, draft_lens, k_scale, v_scale,
                               max_parts, scale, out, lse, workspace)
    nb, hkv, bs, d, code = _cache_args(k_cache, v_cache, k_scale, v_scale, block_table)
    B, max_blocks = block_table.shape
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != d:
        raise ValueError(f"q must be [{B}, Hq, T, {d}], got {tuple(shape)}")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bfloat16")
    _, Hq, T, _ = shape
    _check_lens("seq_lens", seq_lens, B)
    if draft_lens is not None:
        _check_lens("draft_lens", draft_lens, B)
    mask_ptr, mask_sb = None, 0
    if tree_mask is not None:
        if tree_mask.dtype != torch.bool and tree_mask.dtype != torch.uint8:
            raise TypeError("tree_mask must be bool or uint8")
        shape, step = tree_mask.shape, tree_mask.stride()
        if shape != (B, T, T) and shape != (T, T) or (T > 1 and step[-2:] != (T, 1)):
            raise ValueError("tree_mask must be [T, T] or [B, T, T] with contiguous rows")
        mask_ptr = tree_mask.data_ptr()
        mask_sb = step[0] if len(shape) == 3 and B > 1 else 0
    if not -(1 << 31) <= max_parts < 1 << 31:
        raise ValueError("max_parts must be an int32")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _check_out("out", out, q.shape, torch.bfloat16, dev)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    else:
        _check_out("lse", lse, (B, Hq, T), torch.float32, dev)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    if workspace is None:
        size = max(decode_tree_workspace_size(B, Hq, hkv, T, d, max_parts), 16)
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    status = lib().fa_decode_tree(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale),
                                  block_table.data_ptr(), seq_lens.data_ptr(), _addr(draft_lens), mask_ptr, mask_sb,
                                  out.data_ptr(), lse.data_ptr(), B, Hq, hkv, T, nb, bs, max_blocks, d, code,
                                  float(scale), _strides(q, out), int(max_parts), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _current_stream(dev))
    if status:
        _check(status)
    return out, lse
