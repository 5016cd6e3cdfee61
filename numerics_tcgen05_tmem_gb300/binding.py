"""Thin ctypes binding of ``libfa.so`` (see ``include/fa.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  PyTorch supplies device memory and the stream.
There is no fallback: if the library is missing or a call fails, an exception
is raised.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_TIMEOUT = 4
FA_ERR_DEVICE_BOUNDS = 5
FA_WARN_NONFINITE = 6

# which output a non-finite count belongs to (fa_device_report.nonfinite[i])
FA_OUT_O, FA_OUT_LSE, FA_OUT_DQ, FA_OUT_DK, FA_OUT_DV = range(5)
OUTPUT_NAMES = ("o", "lse", "dq", "dk", "dv")
FA_DEVFLAG_TIMEOUT, FA_DEVFLAG_BOUNDS, FA_DEVFLAG_NONFINITE = 1, 2, 4

# every symbol include/fa.h declares
EXPORTS = ("fa_fwd", "fa_fwd_window", "fa_fwd_fp8", "fa_quantize_fp8", "fa_bwd", "fa_bwd_window",
           "fa_bwd_window_workspace_size", "fa_bwd_staged",
           "fa_bwd_noalloc", "fa_bwd_noalloc_status", "fa_bwd_workspace_size", "fa_device_status",
           "fa_device_report_read", "fa_last_error", "fa_version", "fa_kv_append", "fa_kv_read",
           "fa_fwd_paged", "fa_fwd_paged_workspace_size", "fa_norm_rotate", "fa_norm_rotate_bwd",
           "fa_norm_rotate_bwd_workspace_size", "fa_qkv_append", "fa_kv_accumulate",
           "fa_kv_accumulate_workspace_size", "fa_kv_evict")

# size of the fixed device scratch behind fa_bwd_noalloc (FA_NOALLOC_SCRATCH_BYTES in fa.h)
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024

FA_BWD_PREPROCESS, FA_BWD_MAIN, FA_BWD_DQ_CONVERT, FA_BWD_ALL = 1, 2, 4, 7


class FAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"fa error {code}: {msg}")
        self.code = code


class RowStats(ctypes.Structure):
    _fields_ = [("row_max_raw", ctypes.c_void_p), ("row_ties", ctypes.c_void_p),
                ("row_branch", ctypes.c_void_p), ("row_ones", ctypes.c_void_p),
                ("row_min_raw", ctypes.c_void_p)]


# element types of a paged cache (fa_paged_kv.dtype)
FA_KV_BF16, FA_KV_E4M3 = 0, 1


class PagedKV(ctypes.Structure):
    """fa_paged_kv: a paged key/value cache with its block table and lengths."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("kv_len", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Rotation(ctypes.Structure):
    """fa_rotation: how queries and keys are normed and rotated."""
    _fields_ = [("inv_freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("weight_bf16", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("eps", ctypes.c_float)]


class Heads(ctypes.Structure):
    """fa_heads: a view [B, H, N, d] with its strides."""
    _fields_ = [("p", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_n", ctypes.c_int64)]


class DeviceReport(ctypes.Structure):
    """fa_device_report: flags, the first failed index check and non-finite counts per output."""
    _fields_ = [("flags", ctypes.c_uint32), ("bounds_site", ctypes.c_uint32), ("bounds_value", ctypes.c_int64),
                ("nonfinite", ctypes.c_uint64 * 5), ("reserved", ctypes.c_uint64)]

    def as_dict(self):
        return {"flags": int(self.flags), "bounds_site": int(self.bounds_site),
                "bounds_value": int(self.bounds_value),
                "nonfinite": {n: int(self.nonfinite[i]) for i, n in enumerate(OUTPUT_NAMES)}}


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m numerics_tcgen05_tmem_gb300.build`")
    L = ctypes.CDLL(path)
    vp, ci, cf, cs = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, cf, ctypes.POINTER(RowStats), vp]
    L.fa_fwd.restype = ci
    L.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, cf, ctypes.POINTER(RowStats), vp]
    L.fa_fwd_window.restype = ci
    L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, cf, ctypes.POINTER(RowStats), vp]
    L.fa_fwd_fp8.restype = ci
    L.fa_quantize_fp8.argtypes = [vp, cs, vp, vp, vp]
    L.fa_quantize_fp8.restype = ci
    L.fa_bwd_workspace_size.argtypes = [ci, ci, ci, ci]
    L.fa_bwd_workspace_size.restype = cs
    L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp, cs, vp]
    L.fa_bwd.restype = ci
    L.fa_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, vp, cs, vp]
    L.fa_bwd_window.restype = ci
    L.fa_bwd_window_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci]
    L.fa_bwd_window_workspace_size.restype = cs
    L.fa_bwd_staged.argtypes = L.fa_bwd.argtypes + [ci]
    L.fa_bwd_staged.restype = ci
    L.fa_kv_append.argtypes = [ctypes.POINTER(PagedKV), vp, vp, ctypes.c_int64, vp, ci, vp]
    L.fa_kv_append.restype = ci
    L.fa_kv_read.argtypes = [ctypes.POINTER(PagedKV), vp, vp, vp, ci, vp]
    L.fa_kv_read.restype = ci
    L.fa_fwd_paged_workspace_size.argtypes = [ci] * 10
    L.fa_fwd_paged_workspace_size.restype = cs
    L.fa_fwd_paged.argtypes = [ctypes.POINTER(PagedKV), vp, ctypes.c_int64, vp, ci, ci, ci, vp, vp, ci, ci, cf, vp, cs, vp]
    L.fa_fwd_paged.restype = ci
    heads, rotation, c64 = ctypes.POINTER(Heads), ctypes.POINTER(Rotation), ctypes.c_int64
    L.fa_norm_rotate.argtypes = [rotation] + [heads] * 4 + [ci] * 5 + [vp, c64, vp]
    L.fa_norm_rotate.restype = ci
    L.fa_norm_rotate_bwd_workspace_size.argtypes = [ci] * 5
    L.fa_norm_rotate_bwd_workspace_size.restype = cs
    L.fa_norm_rotate_bwd.argtypes = [rotation] + [heads] * 6 + [vp, vp] + [ci] * 5 + [vp, c64, vp, cs, vp]
    L.fa_norm_rotate_bwd.restype = ci
    L.fa_qkv_append.argtypes = [ctypes.POINTER(PagedKV), rotation, vp, c64, vp, ci, vp, vp, c64, vp, vp, ci, vp]
    L.fa_qkv_append.restype = ci
    L.fa_kv_accumulate_workspace_size.argtypes = [ci] * 6
    L.fa_kv_accumulate_workspace_size.restype = cs
    L.fa_kv_accumulate.argtypes = [ctypes.POINTER(PagedKV), vp, c64, vp, c64, vp, vp, ci, ci, ci, ci, ci, cf, vp, cs, vp]
    L.fa_kv_accumulate.restype = ci
    L.fa_kv_evict.argtypes = [ctypes.POINTER(PagedKV), vp, c64, vp, c64, ci, ci, ci, ci, vp, vp, vp]
    L.fa_kv_evict.restype = ci
    L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp]
    L.fa_bwd_noalloc.restype = ci
    L.fa_device_status.argtypes = [vp]
    L.fa_device_status.restype = ci
    L.fa_device_report_read.argtypes = [vp, ctypes.POINTER(DeviceReport)]
    L.fa_device_report_read.restype = ci
    L.fa_bwd_noalloc_status.argtypes = [vp, ctypes.POINTER(DeviceReport)]
    L.fa_bwd_noalloc_status.restype = ci
    L.fa_last_error.argtypes = []
    L.fa_last_error.restype = ctypes.c_char_p
    L.fa_version.argtypes = []
    L.fa_version.restype = ctypes.c_char_p
    _lib = L
    return L


def last_error() -> str:
    return load().fa_last_error().decode()


def _check(rc: int):
    if rc != FA_OK:
        raise FAError(rc, last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if torch.cuda.is_initialized():   # the current stream's handle, without a Stream object for it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, like, stream):
    """A fresh tensor that belongs to the stream the call runs on, so that its memory is not handed out
    to another stream's work while a kernel of the call still uses it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _empty_like(t, stream):
    """_empty with a contiguous tensor's shape and type (PyTorch makes it in four fifths of the time)."""
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


class _Here:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


class _OnDevice:
    """Makes a device current for a call."""

    def __init__(self, dev):
        self.dev = dev

    def __enter__(self):
        self.back = torch._C._cuda_getDevice()
        torch.cuda.set_device(self.dev)

    def __exit__(self, *exc):
        torch.cuda.set_device(self.back)


_HERE = _Here()


def _on_device(t):
    """A context in which a tensor's device is current; nothing to do where it is already."""
    dev = t.get_device()
    return _HERE if torch._C._cuda_getDevice() == dev else _OnDevice(dev)


def _c_int(x):
    """A window, a number of sinks or a largest length as a C int.  Past 32 bits it means what the largest
    int does (no tensor is that long), where ctypes would keep the low bits."""
    return min(max(int(x), -2 ** 31), 2 ** 31 - 1)


def _check_qkv(*ts):
    shape, dev = ts[0].shape, ts[0].get_device()
    for t in ts:
        if not (t.is_cuda and t.dtype is torch.bfloat16 and t.is_contiguous() and t.dim() == 4):
            raise ValueError("expected contiguous CUDA bfloat16 tensors of shape [B, H, N, d]")
        if t.shape != shape or t.get_device() != dev:
            raise ValueError("q, k, v (and o, dO) must have the same shape and device")


# ----------------------------------------------------------------- raw C calls

def fa_fwd(q, k, v, o, lse, causal: bool, scale: float, stable: int, beta: float, stats=None, stream=None) -> int:
    B, H, N, d = q.shape
    st = _row_stats(stats)
    return load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, int(bool(causal)),
                         float(scale), int(stable), float(beta), ctypes.byref(st) if st is not None else None,
                         _stream(stream))


def fa_fwd_window(q, k, v, o, lse, window: int, sinks: int, scale: float, stable: int, beta: float, stats=None,
                  stream=None) -> int:
    B, H, N, d = q.shape
    st = _row_stats(stats)
    return load().fa_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, _c_int(window), _c_int(sinks),
                                float(scale), int(stable), float(beta), ctypes.byref(st) if st is not None else None,
                                _stream(stream))


def _row_stats(stats):
    if stats is None:
        return None
    return RowStats(*(None if stats.get(n) is None else stats[n].data_ptr()
                      for n in ("row_max_raw", "row_ties", "row_branch", "row_ones", "row_min_raw")))


def fa_fwd_fp8(q8, k8, v8, descale, o, lse, causal: bool, scale: float, stable: int, beta: float, stats=None,
               stream=None) -> int:
    B, H, N, d = q8.shape
    st = _row_stats(stats)
    return load().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(descale), _ptr(o), _ptr(lse), B, H, N, d,
                             int(bool(causal)), float(scale), int(stable), float(beta),
                             ctypes.byref(st) if st is not None else None, _stream(stream))


def fa_quantize_fp8(x, x8, descale, stream=None) -> int:
    return load().fa_quantize_fp8(_ptr(x), int(x.numel()), _ptr(x8), _ptr(descale), _stream(stream))


def fa_fwd_paged_workspace_size(T: int, B: int, max_q: int, Hq: int, Hkv: int, d: int, max_kv: int,
                                window: int = 0, sinks: int = 0, dtype: int = FA_KV_BF16) -> int:
    return int(load().fa_fwd_paged_workspace_size(T, B, _c_int(max_q), Hq, Hkv, d, _c_int(max_kv), _c_int(window),
                                                  _c_int(sinks), dtype))


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(q, k, v, o, lse, do, dq, dk, dv, delta, causal: bool, scale: float, workspace, stream=None,
           stages: int = FA_BWD_ALL) -> int:
    B, H, N, d = q.shape
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(delta),
            B, H, N, d, int(bool(causal)), float(scale), _ptr(workspace), nbytes, _stream(stream))
    if stages == FA_BWD_ALL:
        return load().fa_bwd(*args)
    return load().fa_bwd_staged(*args, int(stages))


def fa_bwd_window_workspace_size(B: int, H: int, N: int, d: int, window: int, sinks: int = 0) -> int:
    return int(load().fa_bwd_window_workspace_size(B, H, N, d, _c_int(window), _c_int(sinks)))


def fa_bwd_window(q, k, v, o, lse, do, dq, dk, dv, delta, window: int, sinks: int, scale: float, workspace,
                  stream=None) -> int:
    B, H, N, d = q.shape
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return load().fa_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                                _ptr(delta), B, H, N, d, _c_int(window), _c_int(sinks), float(scale), _ptr(workspace),
                                nbytes, _stream(stream))


def fa_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, delta, causal: bool, scale: float, stream=None) -> int:
    """fa_bwd without a workspace: the library's fixed device scratch is used (nothing is allocated)."""
    B, H, N, d = q.shape
    return load().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                                 _ptr(dv), _ptr(delta), B, H, N, d, int(bool(causal)), float(scale),
                                 _stream(stream))


def fa_device_status(stream=None) -> int:
    return load().fa_device_status(_stream(stream))


def fa_device_report_read(stream=None):
    """(status code, report dict) of the library's device status record; reading clears it."""
    rep = DeviceReport()
    rc = load().fa_device_report_read(_stream(stream), ctypes.byref(rep))
    return rc, rep.as_dict()


def fa_bwd_noalloc_status(stream=None):
    """(status code, report dict) of fa_bwd_noalloc's own status record; reading clears it."""
    rep = DeviceReport()
    rc = load().fa_bwd_noalloc_status(_stream(stream), ctypes.byref(rep))
    return rc, rep.as_dict()


# ----------------------------------------------------------------- tensor-level helpers

def _stats_dict(B, H, N, like, stream):
    return {name: _empty((B, H, N), dtype, like, stream)
            for name, dtype in (("row_max_raw", torch.float32), ("row_ties", torch.int32), ("row_branch", torch.int8),
                                ("row_ones", torch.int32), ("row_min_raw", torch.float32))}


def _check_window(causal, window, sinks):
    if window is None:
        if sinks:
            raise ValueError("sinks need a window")
    elif not causal:
        raise ValueError("a window needs causal=True")


def forward(q, k, v, causal: bool = True, scale=None, stable: int = 1, beta: float = 1.25, stats: bool = False,
            stream=None, window=None, sinks: int = 0):
    """Returns (o, lse) or (o, lse, stats_dict); outputs are freshly allocated.

    With a window (causal only), query i sees the keys j <= i with i - j < window and the
    first ``sinks`` keys.
    """
    _check_qkv(q, k, v)
    _check_window(causal, window, sinks)
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = _empty_like(q, stream)
    lse = _empty((B, H, N), torch.float32, q, stream)
    sd = _stats_dict(B, H, N, q, stream) if stats else None
    with _on_device(q):
        if window is None:
            _check(fa_fwd(q, k, v, o, lse, causal, scale, stable, beta, sd, stream))
        else:
            _check(fa_fwd_window(q, k, v, o, lse, window, sinks, scale, stable, beta, sd, stream))
    return (o, lse, sd) if stats else (o, lse)


def quantize_fp8(x, stream=None):
    """Dynamic per-tensor E4M3 scaling of a contiguous CUDA bfloat16 tensor.

    Returns (x8, descale): x8 holds the E4M3 codes as uint8 with x's shape, descale is a
    1-element FP32 CUDA tensor; x is represented by x8 * descale.
    """
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("expected a contiguous CUDA bfloat16 tensor")
    x8 = _empty(x.shape, torch.uint8, x, stream)
    descale = _empty(1, torch.float32, x, stream)
    _check(fa_quantize_fp8(x, x8, descale, stream))
    return x8, descale


def forward_fp8(q8, k8, v8, descale, causal: bool = True, scale=None, stable: int = 1, beta: float = 1.25,
                stats: bool = False, stream=None):
    """FP8 forward: q8, k8, v8 are uint8 E4M3 codes [B, H, N, d]; descale is an FP32 CUDA
    tensor of 3 per-tensor scales (Q, K, V).  Returns (o, lse) or (o, lse, stats_dict)."""
    for t in (q8, k8, v8):
        if not (t.is_cuda and t.dtype == torch.uint8 and t.is_contiguous() and t.dim() == 4 and t.shape == q8.shape):
            raise ValueError("expected contiguous CUDA uint8 tensors of one shape [B, H, N, d]")
    if not (descale.is_cuda and descale.dtype == torch.float32 and descale.numel() == 3 and descale.is_contiguous()):
        raise ValueError("descale must be a contiguous CUDA float32 tensor of 3 elements")
    B, H, N, d = q8.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = _empty((B, H, N, d), torch.bfloat16, q8, stream)
    lse = _empty((B, H, N), torch.float32, q8, stream)
    sd = _stats_dict(B, H, N, q8, stream) if stats else None
    _check(fa_fwd_fp8(q8, k8, v8, descale, o, lse, causal, scale, stable, beta, sd, stream))
    return (o, lse, sd) if stats else (o, lse)


def backward(q, k, v, o, lse, do, causal: bool = True, scale=None, workspace=None, want_delta: bool = False,
             stream=None, window=None, sinks: int = 0):
    """Returns (dq, dk, dv) or (dq, dk, dv, delta); window and sinks are the forward's, a workspace
    has fa_bwd_workspace_size (with a window: fa_bwd_window_workspace_size) bytes."""
    _check_qkv(q, k, v, o, do)
    _check_window(causal, window, sinks)
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if workspace is None:
        size = fa_bwd_workspace_size(B, H, N, d) if window is None else \
            fa_bwd_window_workspace_size(B, H, N, d, window, sinks)
        workspace = _empty(size, torch.uint8, q, stream)
    dq, dk, dv = _empty_like(q, stream), _empty_like(q, stream), _empty_like(q, stream)
    delta = _empty((B, H, N), torch.float32, q, stream) if want_delta else None
    with _on_device(q):
        if window is None:
            _check(fa_bwd(q, k, v, o, lse, do, dq, dk, dv, delta, causal, scale, workspace, stream))
        else:
            _check(fa_bwd_window(q, k, v, o, lse, do, dq, dk, dv, delta, window, sinks, scale, workspace, stream))
    return (dq, dk, dv, delta) if want_delta else (dq, dk, dv)


# ----------------------------------------------------------------- paged key/value caches

def _outer(n, stride, least, name):
    """The stride of the outermost dimension (n entries); one entry's may be anything."""
    if n <= 1:
        return least
    if stride < least:
        raise ValueError(f"{name}: entries must not overlap (stride {stride} is less than {least})")
    return stride


def _alike(a, b, inner):
    """Whether two tensors of one shape have contiguous pages (strides `inner` behind the first dimension)
    that lie the same distance apart; a dimension of one entry has no stride."""
    sa, sb = a.stride(), b.stride()
    if sa == sb and sa[1:] == inner:
        return True
    n = a.shape
    return all(n[i + 1] == 1 or sa[i + 1] == sb[i + 1] == w for i, w in enumerate(inner)) and \
        (n[0] == 1 or sa[0] == sb[0])


def _int32(t, n, name, dev):
    if t.dtype is not torch.int32 or t.get_device() != dev or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector on the cache's device")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} entries (got {t.numel()})")
    return t.data_ptr()


def _paged(k, v, table, kv_len, k_scale, v_scale):
    """The fa_paged_kv of a cache's tensors (shapes, types and strides checked)."""
    shape, dtype, dev = k.shape, k.dtype, k.get_device()
    if dev < 0 or len(shape) != 4 or v.shape != shape or v.dtype is not dtype or v.get_device() != dev:
        raise ValueError("expected CUDA cache tensors of one shape [pages, Hkv, page_size, d] and one type")
    P, H, S, d = shape
    if not _alike(k, v, (S * d, d, 1)):
        raise ValueError("cache pages must be contiguous, with the same page stride for K and V")
    rows = table.stride()
    if table.dtype is not torch.int32 or len(rows) != 2 or (rows[1] != 1 and table.shape[1] != 1) or \
            table.get_device() != dev:
        raise ValueError("block_table must be an int32 tensor [B, max_pages] on the cache's device, rows contiguous")
    B, width = table.shape
    kv_ptr = _int32(kv_len, B, "kv_len", dev)
    ks = vs = None
    scale_stride, code = 0, FA_KV_BF16
    if dtype is torch.bfloat16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
    elif dtype is torch.uint8 or dtype is torch.float8_e4m3fn:
        if k_scale is None or v_scale is None:
            raise ValueError("an E4M3 cache needs k_scale and v_scale")
        for s in (k_scale, v_scale):
            if s.dtype is not torch.float32 or s.shape != shape[:3] or s.get_device() != dev:
                raise ValueError("k_scale and v_scale must be float32 [pages, Hkv, page_size] on the cache's device")
        if not _alike(k_scale, v_scale, (S, 1)):
            raise ValueError("scale pages must be contiguous, with the same page stride for K and V")
        ks, vs, code = k_scale.data_ptr(), v_scale.data_ptr(), FA_KV_E4M3
        scale_stride = _outer(P, k_scale.stride(0), H * S, "k_scale")
    else:
        raise ValueError("cache tensors must be bfloat16, or uint8 (or float8_e4m3fn) E4M3 codes")
    return PagedKV(k.data_ptr(), v.data_ptr(), ks, vs, _outer(P, k.stride(0), H * S * d, "cache"), scale_stride,
                   table.data_ptr(), _outer(B, rows[0], width, "block_table"), kv_ptr, B, H, d, S, P, width, code)


def _check_rows(x, heads, d, dev, name):
    """Packed rows [rows, heads, d], a row's heads contiguous: the rows' number and stride."""
    shape, stride = x.shape, x.stride()
    if x.dtype is not torch.bfloat16 or x.get_device() != dev or len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor [rows, {heads}, {d}] on the cache's device")
    if shape[0] and (stride[2] != 1 or (heads > 1 and stride[1] != d)):
        raise ValueError(f"{name}: a row's heads must be contiguous")
    return shape[0], _outer(shape[0], stride[0], heads * d, name)


def kv_append(k_new, v_new, k_cache, v_cache, block_table, kv_len, q_indptr, k_scale=None, v_scale=None, stream=None):
    """Write new tokens into a paged cache (in place).

    k_new, v_new: bfloat16 [T, Hkv, d], rows strided alike; sequence b's are the rows
    q_indptr[b] .. q_indptr[b + 1] - 1 and become the positions kv_len[b] - n .. kv_len[b] - 1.
    k_cache, v_cache: [pages, Hkv, page_size, d], bfloat16, or E4M3 codes (uint8 or float8_e4m3fn)
    with float32 scales [pages, Hkv, page_size].  block_table: int32 [B, max_pages].
    """
    kv = _paged(k_cache, v_cache, block_table, kv_len, k_scale, v_scale)
    dev = k_cache.get_device()
    T, stride = rows = _check_rows(k_new, kv.Hkv, kv.d, dev, "k_new")
    if _check_rows(v_new, kv.Hkv, kv.d, dev, "v_new") != rows:
        raise ValueError("k_new and v_new must have the same rows and row stride")
    indptr = _int32(q_indptr, kv.B + 1, "q_indptr", dev)
    if T:
        with _on_device(k_cache):
            _check(load().fa_kv_append(ctypes.byref(kv), k_new.data_ptr(), v_new.data_ptr(), stride, indptr, T,
                                       _stream(stream)))


def kv_read(k_cache, v_cache, block_table, kv_len, kv_indptr, rows, k_scale=None, v_scale=None, out=None, stream=None):
    """Read a paged cache back: (k, v) bfloat16 [rows, Hkv, d].

    Sequence b's positions 0, 1, ... go to the rows kv_indptr[b], kv_indptr[b] + 1, ..., up to
    kv_indptr[b + 1] or kv_len[b].  Other rows stay as they were (out: the pair of tensors to write
    to) or are not defined (fresh tensors).
    """
    kv = _paged(k_cache, v_cache, block_table, kv_len, k_scale, v_scale)
    dev, shape = k_cache.get_device(), (rows, kv.Hkv, kv.d)
    indptr = _int32(kv_indptr, kv.B + 1, "kv_indptr", dev)
    if out is None:
        k = _empty(shape, torch.bfloat16, k_cache, stream)
        v = _empty_like(k, stream)
    else:
        k, v = out
        for t in out:
            if _check_rows(t, kv.Hkv, kv.d, dev, "out")[0] != rows or not t.is_contiguous():
                raise ValueError("out tensors must be contiguous with `rows` rows")
    if rows:
        with _on_device(k_cache):
            _check(load().fa_kv_read(ctypes.byref(kv), indptr, k.data_ptr(), v.data_ptr(), int(rows), _stream(stream)))
    return k, v


def forward_paged(q, k_cache, v_cache, block_table, kv_len, q_indptr, max_q, k_scale=None, v_scale=None, scale=None,
                  window=None, sinks: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of each sequence's newest tokens over its paged cache: (o, lse).

    q: bfloat16 [T, Hq, d] (rows may be strided); sequence b's new tokens are the rows q_indptr[b] ..
    q_indptr[b + 1] - 1 and the last positions of its cache, which already holds their keys and
    values (kv_append).  max_q: at least the largest number of new tokens of a sequence; 0 says that there
    are none, and nothing is written.  Hq is a multiple of the cache's heads.  With a window, the token at position p sees the keys
    p - window < j <= p and the first ``sinks`` keys; otherwise every key j <= p.
    out, lse: tensors to write to ([T, Hq, d] bfloat16, [T, Hq] float32); rows behind the last
    sequence stay as they were (undefined in fresh tensors).
    workspace: fa_fwd_paged_workspace_size bytes, for calls that do not overlap; else allocated.  For
    long chunks over an E4M3 cache it holds a BF16 copy of what they see (2 GiB at most, from the
    block table's width).
    """
    kv = _paged(k_cache, v_cache, block_table, kv_len, k_scale, v_scale)
    if window is None:
        if sinks:
            raise ValueError("sinks need a window")
        window = 0
    elif window < 1:
        raise ValueError("window must be >= 1 (None: no window)")
    window, sinks, max_q = _c_int(window), _c_int(sinks), _c_int(max_q)
    dev, d = k_cache.get_device(), kv.d
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, d]")
    Hq = q.shape[1]
    T, stride = _check_rows(q, Hq, d, dev, "q")
    indptr = _int32(q_indptr, kv.B + 1, "q_indptr", dev)
    if out is None:
        out = _empty_like(q, stream) if stride == Hq * d else _empty((T, Hq, d), torch.bfloat16, q, stream)
    elif out.dtype is not torch.bfloat16 or out.shape != q.shape or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out must be a contiguous bfloat16 tensor of q's shape")
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q, stream)
    elif lse.dtype is not torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous() or \
            lse.get_device() != dev:
        raise ValueError("lse must be a contiguous float32 tensor [T, Hq]")
    if T == 0:
        return out, lse
    lib = load()
    if workspace is None:
        n = lib.fa_fwd_paged_workspace_size(T, kv.B, max_q, Hq, kv.Hkv, d, kv.max_pages * kv.page_size, window, sinks,
                                            kv.dtype)
        workspace = _empty(n, torch.uint8, q, stream) if n else None
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    ws, nbytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    with _on_device(k_cache):
        _check(lib.fa_fwd_paged(ctypes.byref(kv), q.data_ptr(), stride, indptr, T, max_q, Hq, out.data_ptr(),
                                lse.data_ptr(), window, sinks, 1.0 / math.sqrt(d) if scale is None else float(scale),
                                ws, nbytes, _stream(stream)))
    return out, lse


# ----------------------------------------------------------------- norm and rotation of queries and keys

def _rotation(inv_freq, d, dev, q_weight, k_weight, eps, interleaved, norm):
    """The fa_rotation of these tensors (types, shapes and devices checked)."""
    rot, freq = 0, None
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != dev or inv_freq.dim() != 1 or \
                not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float64 vector on the queries' device")
        rot, freq = 2 * inv_freq.numel(), inv_freq.data_ptr()
    if q_weight is None and k_weight is None:
        return Rotation(freq, None, None, rot, bool(interleaved), 0, bool(norm), eps)
    if q_weight is None or k_weight is None or q_weight.dtype is not k_weight.dtype:
        raise ValueError("q_weight and k_weight are given together, in one type")
    for w in (q_weight, k_weight):
        if w.dtype not in (torch.float32, torch.bfloat16) or w.get_device() != dev or w.dim() != 1 or w.numel() != d or \
                not w.is_contiguous():
            raise ValueError(f"weights must be contiguous float32 or bfloat16 vectors of {d} on the queries' device")
    return Rotation(freq, q_weight.data_ptr(), k_weight.data_ptr(), rot, bool(interleaved),
                    q_weight.dtype is torch.bfloat16, bool(norm), eps)


def _heads(t, name, shape, dev):
    """The fa_heads of a view [B, H, N, d]."""
    stride = t.stride()
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor {list(shape)} on the queries' device")
    if stride[3] != 1:
        raise ValueError(f"{name}: heads must be contiguous")
    return Heads(t.data_ptr(), stride[0], stride[1], stride[2])


def _check_qk(q, k):
    """The shapes of queries [B, Hq, N, d] and keys [B, Hkv, N, d] and their device."""
    sq, sk, dev = q.shape, k.shape, q.get_device()
    if dev < 0 or len(sq) != 4 or len(sk) != 4 or sq[0] != sk[0] or sq[2:] != sk[2:]:
        raise ValueError("expected CUDA tensors q [B, Hq, N, d] and k [B, Hkv, N, d]")
    return sq, sk, dev


def _positions(positions, B, N, dev):
    """(pointer, stride between sequences) of positions [N] or [B, N]."""
    if positions is None:
        return None, 0
    shape, stride = positions.shape, positions.stride()
    if positions.dtype is not torch.int32 or positions.get_device() != dev or tuple(shape) not in ((N,), (B, N)) or \
            (stride[-1] != 1 and N > 1):
        raise ValueError(f"positions must be an int32 tensor [{N}] or [{B}, {N}] on the queries' device, rows contiguous")
    return positions.data_ptr(), stride[0] if len(shape) == 2 and B > 1 else 0


def _empty_as(t, stream):
    """A fresh tensor of t's shape, its tokens in front of its heads in memory where t's are."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _empty_as(t, None)
    shape = t.shape
    B, H, N, d = shape
    if t.stride(1) < t.stride(2):
        return t.new_empty_strided(shape, (N * H * d, d, H * d, 1))
    return t.new_empty(shape)


def norm_rotate(q, k, inv_freq, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                norm: bool = True, out=None, stream=None):
    """Queries and keys normed for each head and rotated by their positions: (q', k').

    q: bfloat16 [B, Hq, N, d], k: [B, Hkv, N, d], views with any outer strides that are multiples of 8 (such as
    transposed slices of a fused projection [B, N, heads, d]).  With r = 1 / sqrt(mean x^2 + eps) a head is
    y = weight * x * r, and its pairs i (entries i and i + rot / 2, or 2 i and 2 i + 1 where ``interleaved``) turn by
    position * inv_freq[i].  inv_freq: float64 [rot / 2], or None (the norm alone); rot is a multiple of 16.
    norm=False: the rotation alone.  positions: int32 [N] or [B, N]; None: 0, 1, ...
    q_weight, k_weight: float32 or bfloat16 [d]; None: ones.  out: the pair of tensors to write to (the inputs
    themselves are fine); else fresh contiguous ones, as the attention calls take them.
    """
    sq, sk, dev = _check_qk(q, k)
    plan = _rotation(inv_freq, sq[3], dev, q_weight, k_weight, eps, interleaved, norm)
    hq, hk = _heads(q, "q", sq, dev), _heads(k, "k", sk, dev)
    pos, pos_stride = _positions(positions, sq[0], sq[2], dev)
    if out is None:
        out = _empty(sq, torch.bfloat16, q, stream), _empty(sk, torch.bfloat16, k, stream)
    oq, ok = out
    hoq, hok = _heads(oq, "out", sq, dev), _heads(ok, "out", sk, dev)
    with _on_device(q):
        _check(load().fa_norm_rotate(plan, hq, hk, hoq, hok, sq[0], sq[1], sk[1], sq[2], sq[3], pos, pos_stride,
                                     _stream(stream)))
    return oq, ok


def norm_rotate_backward(q, k, dq_out, dk_out, inv_freq, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                         interleaved: bool = False, norm: bool = True, out=None, workspace=None, stream=None):
    """The backward of norm_rotate: (dq, dk, dq_weight, dk_weight).

    q, k: the forward's inputs; dq_out, dk_out: the gradients of its outputs (any strides); the other arguments are
    the forward's.  dq, dk have the inputs' order of tokens and heads in memory (out: the pair of tensors to
    write to, such as slices of a fused projection's gradient); dq_weight, dk_weight are float32 [d], or None without weights.
    workspace: fa_norm_rotate_bwd_workspace_size bytes, for calls that do not overlap; else allocated.
    """
    sq, sk, dev = _check_qk(q, k)
    B, Hq, N, d = sq
    plan = _rotation(inv_freq, d, dev, q_weight, k_weight, eps, interleaved, norm)
    hq, hk = _heads(q, "q", sq, dev), _heads(k, "k", sk, dev)
    hzq, hzk = _heads(dq_out, "dq_out", sq, dev), _heads(dk_out, "dk_out", sk, dev)
    pos, pos_stride = _positions(positions, B, N, dev)
    dq, dk = (_empty_as(q, stream), _empty_as(k, stream)) if out is None else out
    hdq, hdk = _heads(dq, "out", sq, dev), _heads(dk, "out", sk, dev)
    lib = load()
    dqw = dkw = ws = None
    nbytes = 0
    if q_weight is not None:
        dqw, dkw = _empty(d, torch.float32, q, stream), _empty(d, torch.float32, q, stream)
        if workspace is None:
            workspace = _empty(lib.fa_norm_rotate_bwd_workspace_size(B, Hq, sk[1], N, d), torch.uint8, q, stream)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the queries' device")
        ws, nbytes = workspace.data_ptr(), workspace.nbytes
    with _on_device(q):
        _check(lib.fa_norm_rotate_bwd(plan, hq, hk, hzq, hzk, hdq, hdk, _ptr(dqw), _ptr(dkw), B, Hq, sk[1], N, d, pos,
                                      pos_stride, ws, nbytes, _stream(stream)))
    return dq, dk, dqw, dkw


def fa_norm_rotate_bwd_workspace_size(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(load().fa_norm_rotate_bwd_workspace_size(B, Hq, Hkv, N, d))


def qkv_append(q, k_new, v_new, k_cache, v_cache, block_table, kv_len, q_indptr, inv_freq, positions=None, q_weight=None,
               k_weight=None, eps: float = 1e-6, interleaved: bool = False, norm: bool = True, k_scale=None, v_scale=None,
               out=None, stream=None):
    """norm_rotate and kv_append in one call, for packed rows: returns the queries normed and rotated, bfloat16 [T, Hq, d].

    q: bfloat16 [T, Hq, d]; k_new, v_new: [T, Hkv, d], rows strided alike (slices of a fused projection need no
    copy).  The keys are normed, rotated and written with the values into the cache, as kv_append writes them;
    see there for the cache's tensors, kv_len and q_indptr, and norm_rotate for the rest.
    positions: int32 [T], the tokens' positions for the rotation; None: their places in the cache.
    out: the tensor to write the queries to; rows behind the last sequence stay as they were (undefined in a fresh one).
    """
    kv = _paged(k_cache, v_cache, block_table, kv_len, k_scale, v_scale)
    dev, d = k_cache.get_device(), kv.d
    plan = _rotation(inv_freq, d, dev, q_weight, k_weight, eps, interleaved, norm)
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, d]")
    Hq = q.shape[1]
    T, q_stride = _check_rows(q, Hq, d, dev, "q")
    _, stride = rows = _check_rows(k_new, kv.Hkv, d, dev, "k_new")
    if _check_rows(v_new, kv.Hkv, d, dev, "v_new") != rows or rows[0] != T:
        raise ValueError("q, k_new and v_new must have the same rows, k_new and v_new the same row stride")
    indptr = _int32(q_indptr, kv.B + 1, "q_indptr", dev)
    pos = None if positions is None else _int32(positions, T, "positions", dev)
    if out is None:
        out = _empty_like(q, stream) if q.is_contiguous() else _empty((T, Hq, d), torch.bfloat16, q, stream)
    elif out.dtype is not torch.bfloat16 or out.shape != q.shape or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out must be a contiguous bfloat16 tensor of q's shape")
    if T:
        with _on_device(k_cache):
            _check(load().fa_qkv_append(kv, plan, q.data_ptr(), q_stride, out.data_ptr(), Hq, k_new.data_ptr(),
                                        v_new.data_ptr(), stride, indptr, pos, T, _stream(stream)))
    return out


# ----------------------------------------------------------------- accumulated attention weights, eviction

def fa_kv_accumulate_workspace_size(T: int, max_q: int, Hq: int, Hkv: int, d: int, dtype: int = FA_KV_BF16) -> int:
    return int(load().fa_kv_accumulate_workspace_size(T, _c_int(max_q), Hq, Hkv, d, dtype))


def _weights(weights, kv, k_cache):
    """(pointer, page stride) of a cache's accumulated weights."""
    shape, stride = k_cache.shape, weights.stride()
    if weights.dtype is not torch.float32 or weights.shape != shape[:3] or weights.get_device() != k_cache.get_device():
        raise ValueError("weights must be a float32 tensor [pages, Hkv, page_size] on the cache's device")
    if (shape[2] != 1 and stride[2] != 1) or (shape[1] != 1 and stride[1] != shape[2]):
        raise ValueError("weights: pages must be contiguous")
    return weights.data_ptr(), _outer(shape[0], stride[0], kv.Hkv * kv.page_size, "weights")


def kv_accumulate(weights, q, lse, k_cache, v_cache, block_table, kv_len, q_indptr, max_q, k_scale=None, v_scale=None,
                  scale=None, window=None, sinks: int = 0, workspace=None, stream=None):
    """Add to each cached key the attention weight that the new tokens give it (in place; returns weights).

    weights: float32 [pages, Hkv, page_size], one for each key of the cache.  For key j of a sequence and kv head:
    weights[j] = (0 if j is a new token's else weights[j]) + the sum over the new tokens i that see j and the
    query heads of the kv head of exp(scale q_i . k_j - lse_i).
    q, lse and the other arguments are those of forward_paged and its output; the cache holds the new keys.  Two
    sequences of one call must not share pages, as they may for forward_paged: a shared key's weight would lose one's sum.
    workspace: fa_kv_accumulate_workspace_size bytes, for calls that do not overlap; else allocated.
    """
    kv = _paged(k_cache, v_cache, block_table, kv_len, k_scale, v_scale)
    at, weight_stride = _weights(weights, kv, k_cache)
    if window is None:
        if sinks:
            raise ValueError("sinks need a window")
        window = 0
    elif window < 1:
        raise ValueError("window must be >= 1 (None: no window)")
    dev, d = k_cache.get_device(), kv.d
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, d]")
    Hq = q.shape[1]
    T, stride = _check_rows(q, Hq, d, dev, "q")
    if lse.dtype is not torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous() or lse.get_device() != dev:
        raise ValueError("lse must be a contiguous float32 tensor [T, Hq]")
    indptr = _int32(q_indptr, kv.B + 1, "q_indptr", dev)
    if T == 0:
        return weights
    lib, max_q = load(), _c_int(max_q)
    if workspace is None:
        n = lib.fa_kv_accumulate_workspace_size(T, max_q, Hq, kv.Hkv, d, kv.dtype)
        workspace = _empty(n, torch.uint8, q, stream) if n else None
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    ws, nbytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    with _on_device(k_cache):
        _check(lib.fa_kv_accumulate(kv, at, weight_stride, q.data_ptr(), stride, lse.data_ptr(), indptr, T, max_q, Hq,
                                    _c_int(window), _c_int(sinks), 1.0 / math.sqrt(d) if scale is None else float(scale),
                                    ws, nbytes, _stream(stream)))
    return weights


def kv_evict(weights, k_cache, v_cache, block_table, kv_len, keep, sinks: int = 0, recent: int = 0, table_out=None,
             k_scale=None, v_scale=None, kept_len=None, kept=None, stream=None):
    """Cut each sequence's cache to ``keep`` keys for each kv head: (kept_len, kept).

    The first ``sinks`` keys, the newest ``recent`` ones and, of the others, those with the largest weights (of equal
    ones the first) move in order, with their values, scales and weights, to the positions 0, 1, ... of the sequence
    in table_out: int32 [B, pages], free pages of the same pool (not a copy of block_table: keys that were to
    move within it are recorded, and do not); None: in place, where no two sequences share pages.
    weights: float32 [pages, Hkv, page_size] (kv_accumulate).
    kept_len: int32 [B], min(kv_len, keep): the lengths for the calls that follow (kv_len itself is not
    written).  kept: int32 [B, Hkv, keep], the kept keys' former positions, -1 behind kept_len.  Both are
    allocated unless given.  Later tokens keep their own rotation: pass their positions to qkv_append.
    """
    kv = _paged(k_cache, v_cache, block_table, kv_len, k_scale, v_scale)
    at, weight_stride = _weights(weights, kv, k_cache)
    dev = k_cache.get_device()
    out = out_stride = pages = 0
    if table_out is not None:
        rows = table_out.stride()
        if table_out.dtype is not torch.int32 or len(rows) != 2 or table_out.shape[0] != kv.B or \
                (rows[1] != 1 and table_out.shape[1] != 1) or table_out.get_device() != dev:
            raise ValueError("table_out must be an int32 tensor [B, pages] on the cache's device, rows contiguous")
        pages = table_out.shape[1]
        out, out_stride = table_out.data_ptr(), _outer(kv.B, rows[0], pages, "table_out")
    keep = int(keep)
    if not 1 <= keep < 2 ** 31:
        raise ValueError("keep must be from 1 to 2^31 - 1")
    if kept_len is None:
        kept_len = _empty(kv.B, torch.int32, k_cache, stream)
    else:
        _int32(kept_len, kv.B, "kept_len", dev)
    if kept is None:
        kept = _empty((kv.B, kv.Hkv, keep), torch.int32, k_cache, stream)
    elif kept.dtype is not torch.int32 or kept.shape != (kv.B, kv.Hkv, keep) or not kept.is_contiguous() or kept.get_device() != dev:
        raise ValueError("kept must be a contiguous int32 tensor [B, Hkv, keep] on the cache's device")
    with _on_device(k_cache):
        _check(load().fa_kv_evict(kv, at, weight_stride, out or None, out_stride, pages, keep, _c_int(sinks), _c_int(recent),
                                  kept_len.data_ptr(), kept.data_ptr(), _stream(stream)))
    return kept_len, kept


def device_status(stream=None):
    """Synchronise and raise if a kernel reported a device-side error."""
    _check(fa_device_status(stream))
