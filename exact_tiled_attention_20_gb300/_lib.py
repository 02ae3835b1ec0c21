"""ctypes binding of libfa.so -- argument marshalling only.

Every name here mirrors an entry point of include/fa.h.  Tensors are PyTorch CUDA tensors
(PyTorch provides device memory and streams); all arithmetic runs in the library's CUDA
kernels.  There is no CPU fallback: if libfa.so is missing or a call fails, an exception
is raised.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

from . import build as _build

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(6)
FA_BF16, FA_FP16 = 0, 1

_DTYPE = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}

_lock = threading.Lock()
_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {fa_status_string(status)} (status {status})")
        self.status = status


def library_path() -> str:
    return _build.LIB


def load():
    """Loads libfa.so (raising if it has not been built) and declares the signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, I, P]
        lib.fa_fwd.restype = I
        lib.fa_fwd_window.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, P]
        lib.fa_fwd_window.restype = I
        lib.fa_decode_workspace_bytes.argtypes = [I, I, I, I]
        lib.fa_decode_workspace_bytes.restype = SZ
        lib.fa_decode_default_splits.argtypes = [I, I, I, I]
        lib.fa_decode_default_splits.restype = I
        lib.fa_decode_splitkv.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, P, SZ, I, P]
        lib.fa_decode_splitkv.restype = I
        lib.fa_status_string.argtypes = [I]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_last_device_status.argtypes = []
        lib.fa_last_device_status.restype = I
        lib.fa_selftest_bounded_wait.argtypes = [P, P]
        lib.fa_selftest_bounded_wait.restype = I
        _lib = lib
        return lib


def _check_cuda(name, t, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _stream_handle(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def fa_status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


def fa_last_device_status() -> int:
    """Reads and clears the device status word (synchronises the device)."""
    return int(load().fa_last_device_status())


def fa_selftest_bounded_wait(result, stream=None) -> int:
    """Enqueues the bounded-wait self-test (see include/fa.h); result is a CUDA int32
    tensor of 3 elements.  Returns the launch status."""
    _check_cuda("result", result, torch.int32)
    if result.numel() < 3:
        raise ValueError("result needs 3 elements")
    return int(load().fa_selftest_bounded_wait(ctypes.c_void_p(result.data_ptr()),
                                               ctypes.c_void_p(_stream_handle(stream))))


def fa_fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
           return_lse: bool = True, stream=None, window=None):
    """Exact attention forward through fa_fwd (or fa_fwd_window when ``window=(left,
    right)`` is given; -1 = unbounded side).  q [B,Sq,Hq,D], k/v [B,Sk,Hkv,D].

    Returns (o, lse): o like q, lse fp32 [B, Hq, Sq] (None if return_lse is False and no
    lse buffer was given).  scale defaults to 1/sqrt(D).
    """
    if q.dtype not in _DTYPE:
        raise TypeError("q/k/v must be bf16 or fp16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_cuda(name, t, q.dtype)
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D:
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    if out is None:
        out = torch.empty_like(q)
    _check_cuda("out", out, q.dtype)
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have q's shape")
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check_cuda("lse", lse, torch.float32)
        if tuple(lse.shape) != (B, Hq, Sq):
            raise ValueError("lse must be [B, Hq, Sq]")
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        lp = lse.data_ptr() if lse is not None else None
        if window is None:
            st = load().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lp, B, Sq,
                               Sk, Hq, Hkv, D, sc, int(bool(causal)), _DTYPE[q.dtype],
                               _stream_handle(stream))
        else:
            st = load().fa_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lp,
                                      B, Sq, Sk, Hq, Hkv, D, sc, int(bool(causal)), int(window[0]),
                                      int(window[1]), _DTYPE[q.dtype], _stream_handle(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_window" if window is not None else "fa_fwd")
    return out, lse


def fa_decode_workspace_bytes(B: int, Hq: int, D: int, num_splits: int) -> int:
    return int(load().fa_decode_workspace_bytes(B, Hq, D, num_splits))


def fa_decode_default_splits(B: int, Hkv: int, max_kv_len: int, num_sms: int = 0) -> int:
    return int(load().fa_decode_default_splits(B, Hkv, max_kv_len, num_sms))


def fa_decode_splitkv(q, k_cache, v_cache, kv_lens, scale: float | None = None,
                      num_splits: int = 0, workspace=None, out=None, lse=None,
                      return_lse: bool = True, stream=None):
    """Split-KV decode through fa_decode_splitkv.

    q [B,1,Hq,D]; k_cache/v_cache [B,Smax,Hkv,D]; kv_lens int32 [B] on the device.
    workspace: a CUDA uint8 tensor of at least fa_decode_workspace_bytes(...) bytes, or
    None to allocate one with PyTorch.  Returns (o [B,1,Hq,D], lse [B,Hq]).
    """
    if q.dtype not in _DTYPE:
        raise TypeError("q/k_cache/v_cache must be bf16 or fp16")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        _check_cuda(name, t, q.dtype)
    _check_cuda("kv_lens", kv_lens, torch.int32)
    if q.dim() == 3:
        q = q.unsqueeze(1)
    B, one, Hq, D = q.shape
    if one != 1:
        raise ValueError("decode takes one query token per sequence: q [B, 1, Hq, D]")
    Bk, Smax, Hkv, Dk = k_cache.shape
    if tuple(v_cache.shape) != tuple(k_cache.shape) or Bk != B or Dk != D:
        raise ValueError("cache shape mismatch")
    if kv_lens.numel() != B:
        raise ValueError("kv_lens must hold B lengths")
    lib = load()
    with torch.cuda.device(q.device):
        ns = int(num_splits) if num_splits and num_splits > 0 else \
            lib.fa_decode_default_splits(B, Hkv, Smax, 0)
        if ns <= 0:
            raise FaError(FA_ERR_CUDA, "fa_decode_default_splits")
        ns = min(ns, Smax)
        need = lib.fa_decode_workspace_bytes(B, Hq, D, ns)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _check_cuda("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
        if out is None:
            out = torch.empty_like(q)
        _check_cuda("out", out, q.dtype)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
        if lse is not None:
            _check_cuda("lse", lse, torch.float32)
        sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
        st = lib.fa_decode_splitkv(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                   kv_lens.data_ptr(), out.data_ptr(),
                                   lse.data_ptr() if lse is not None else None, B, Hq, Hkv, D,
                                   Smax, sc, ns, workspace.data_ptr(), ws_bytes, _DTYPE[q.dtype],
                                   _stream_handle(stream))
    if st != FA_OK:
        raise FaError(st, "fa_decode_splitkv")
    return out, lse


_noalloc_declared = False


def fa_decode_splitkv_noalloc(q, k_cache, v_cache, kv_lens, scale: float | None = None,
                              num_splits: int = 0, out=None, lse=None, stream=None):
    """fa_decode_splitkv_noalloc: split-KV decode without a caller workspace, for callers
    that cannot allocate device memory (the partials go to a fixed scratch array inside
    the library; see include/fa.h for its size limit and sharing rules).  Output tensors
    must be given or are created here with PyTorch."""
    global _noalloc_declared
    lib = load()
    if not _noalloc_declared:
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.fa_decode_splitkv_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, I, P]
        lib.fa_decode_splitkv_noalloc.restype = I
        _noalloc_declared = True
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        _check_cuda(name, t, q.dtype)
    _check_cuda("kv_lens", kv_lens, torch.int32)
    B, _, Hq, D = q.shape
    _, Smax, Hkv, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        st = lib.fa_decode_splitkv_noalloc(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                           kv_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), B,
                                           Hq, Hkv, D, Smax, sc, int(num_splits), _DTYPE[q.dtype],
                                           _stream_handle(stream))
    if st != FA_OK:
        raise FaError(st, "fa_decode_splitkv_noalloc")
    return out, lse


_paged_declared = False


def fa_decode_splitkv_paged(q, k_pages, v_pages, block_table, kv_lens, scale: float | None = None,
                            num_splits: int = 0, workspace=None, out=None, lse=None, stream=None):
    """Split-KV decode over a paged cache through fa_decode_splitkv_paged.

    q [B,1,Hq,D]; k_pages/v_pages [num_pages, page_size, Hkv, D]; block_table int32
    [B, max_pages_per_seq] and kv_lens int32 [B] on the device.  Returns (o, lse)."""
    global _paged_declared
    lib = load()
    if not _paged_declared:
        P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_decode_splitkv_paged.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P,
                                                SZ, I, P]
        lib.fa_decode_splitkv_paged.restype = I
        _paged_declared = True
    if q.dtype not in _DTYPE:
        raise TypeError("q/k_pages/v_pages must be bf16 or fp16")
    for name, t in (("q", q), ("k_pages", k_pages), ("v_pages", v_pages)):
        _check_cuda(name, t, q.dtype)
    _check_cuda("block_table", block_table, torch.int32)
    _check_cuda("kv_lens", kv_lens, torch.int32)
    B, _, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_pages.shape
    max_pages = block_table.shape[1]
    with torch.cuda.device(q.device):
        ns = int(num_splits) if num_splits and num_splits > 0 else \
            lib.fa_decode_default_splits(B, Hkv, page_size * max_pages, 0)
        if ns <= 0:
            raise FaError(FA_ERR_CUDA, "fa_decode_default_splits")
        ns = min(ns, page_size * max_pages)
        if workspace is None:
            workspace = torch.empty(lib.fa_decode_workspace_bytes(B, Hq, D, ns), dtype=torch.uint8,
                                    device=q.device)
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
        sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
        st = lib.fa_decode_splitkv_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                         block_table.data_ptr(), kv_lens.data_ptr(), out.data_ptr(),
                                         lse.data_ptr(), B, Hq, Hkv, D, num_pages, page_size,
                                         max_pages, sc, ns, workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(),
                                         _DTYPE[q.dtype], _stream_handle(stream))
    if st != FA_OK:
        raise FaError(st, "fa_decode_splitkv_paged")
    return out, lse


_varlen_declared = False


def fa_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, causal: bool = False,
                  scale: float | None = None, window=(-1, -1), out=None, lse=None, stream=None):
    """Variable-length batch through fa_fwd_varlen: q [total_q, Hq, D], k/v [total_k, Hkv, D],
    cu_seqlens_q/k int32 [B+1] on the device.  Returns (o [total_q, Hq, D], lse [Hq, total_q])."""
    global _varlen_declared
    lib = load()
    if not _varlen_declared:
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.fa_fwd_varlen.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, P]
        lib.fa_fwd_varlen.restype = I
        _varlen_declared = True
    if q.dtype not in _DTYPE:
        raise TypeError("q/k/v must be bf16 or fp16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_cuda(name, t, q.dtype)
    _check_cuda("cu_seqlens_q", cu_seqlens_q, torch.int32)
    _check_cuda("cu_seqlens_k", cu_seqlens_k, torch.int32)
    total_q, Hq, D = q.shape
    total_k, Hkv, _ = k.shape
    B = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != B + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have B + 1 entries")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               lse.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B,
                               total_q, total_k, Hq, Hkv, D, sc, int(bool(causal)), int(window[0]),
                               int(window[1]), _DTYPE[q.dtype], _stream_handle(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_varlen")
    return out, lse


_multi_declared = False


def fa_decode_splitkv_multi(q, k_cache, v_cache, kv_lens, causal: bool = True,
                            scale: float | None = None, num_splits: int = 0, workspace=None,
                            out=None, lse=None, stream=None):
    """Several query tokens per sequence through fa_decode_splitkv_multi.
    q [B, Sq, Hq, D]; returns (o [B, Sq, Hq, D], lse [B, Hq, Sq])."""
    global _multi_declared
    lib = load()
    if not _multi_declared:
        P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_decode_splitkv_multi.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, P, SZ,
                                                I, P]
        lib.fa_decode_splitkv_multi.restype = I
        _multi_declared = True
    if q.dtype not in _DTYPE:
        raise TypeError("q/k_cache/v_cache must be bf16 or fp16")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        _check_cuda(name, t, q.dtype)
    _check_cuda("kv_lens", kv_lens, torch.int32)
    B, Sq, Hq, D = q.shape
    _, Smax, Hkv, _ = k_cache.shape
    with torch.cuda.device(q.device):
        ns = int(num_splits) if num_splits and num_splits > 0 else \
            lib.fa_decode_default_splits(B, Hkv, Smax, 0)
        ns = min(ns, Smax)
        if workspace is None:
            workspace = torch.empty(lib.fa_decode_workspace_bytes(B * Sq, Hq, D, ns),
                                    dtype=torch.uint8, device=q.device)
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
        sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
        st = lib.fa_decode_splitkv_multi(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                         kv_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Sq,
                                         Hq, Hkv, D, Smax, sc, int(bool(causal)), ns,
                                         workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(),
                                         _DTYPE[q.dtype], _stream_handle(stream))
    if st != FA_OK:
        raise FaError(st, "fa_decode_splitkv_multi")
    return out, lse


# ---- 8-bit paged KV cache.  A decode step runs these for every layer and token and its
# kernels take a few microseconds, so a call asks for all it checks in one expression; only
# where that fails does _refuse find out what to say.
_F8, _U8, _I32, _F32 = torch.float8_e4m3fn, torch.uint8, torch.int32, torch.float32
_fp8_lib = None


def _public_raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# The handle of a device's current stream, and the current device: what torch's own generated code
# asks for them (0.1 us, where the public calls take 1), or those calls where a build lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _load_fp8():
    global _fp8_lib
    if _fp8_lib is None:
        lib = load()
        P, I, F, SZ, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
        lib.fa_kv_append_paged_fp8.argtypes = [P, P, L, L, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P]
        lib.fa_kv_append_paged_fp8.restype = I
        lib.fa_kv_read_paged_fp8.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P]
        lib.fa_kv_read_paged_fp8.restype = I
        lib.fa_decode_splitkv_paged_fp8.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I,
                                                    I, P, SZ, I, P]
        lib.fa_decode_splitkv_paged_fp8.restype = I
        _fp8_lib = lib
    return _fp8_lib


def _refuse(*wanted):
    """Raises for the first of (name, tensor, dtype, device index, shape or None) that is not
    a contiguous CUDA tensor of that type and shape on that device."""
    for name, t, dtype, device, shape in wanted:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise AssertionError("a check failed that finds nothing wrong")


def _fp8_pool(k_pages, v_pages, k_scales, v_scales, block_table):
    """Checks the pool's tensors; returns (device index, num_pages, Hkv, page_size, D, B, max_pages)."""
    try:
        device, shape = k_pages.get_device(), k_pages.shape
        num_pages, Hkv, page, D = shape
        B, max_pages = block_table.shape
        rows = (num_pages, Hkv, page)
        if (device >= 0 and v_pages.get_device() == device and k_scales.get_device() == device
                and v_scales.get_device() == device and block_table.get_device() == device
                and k_pages.dtype is _F8 and v_pages.dtype is _F8 and k_scales.dtype is _U8
                and v_scales.dtype is _U8 and block_table.dtype is _I32 and v_pages.shape == shape
                and k_scales.shape == rows and v_scales.shape == rows and k_pages.is_contiguous()
                and v_pages.is_contiguous() and k_scales.is_contiguous() and v_scales.is_contiguous()
                and block_table.is_contiguous()):
            return device, num_pages, Hkv, page, D, B, max_pages
    except (AttributeError, ValueError):  # no tensors, or of other dimensions
        for t in (k_pages, v_pages, k_scales, v_scales, block_table):
            if not isinstance(t, torch.Tensor):
                raise TypeError("the pool, its scales and block_table must be CUDA tensors") from None
        raise ValueError("k_pages must be [num_pages, Hkv, page_size, D] and block_table "
                         "[B, max_pages_per_seq]") from None
    _refuse(("k_pages", k_pages, _F8, device, shape), ("v_pages", v_pages, _F8, device, shape),
            ("k_scales", k_scales, _U8, device, rows), ("v_scales", v_scales, _U8, device, rows),
            ("block_table", block_table, _I32, device, None))


def _is(t, dtype, device, shape):
    """Whether t is a contiguous tensor of this type and shape (None: any) on this device."""
    try:
        return (t.dtype is dtype and t.get_device() == device and (shape is None or t.shape == shape)
                and t.is_contiguous())
    except AttributeError:
        return False


def _stream_on(device, stream):
    """(handle of `stream` or of the device's current stream, the stream where it is not the
    current one)."""
    current = _raw_stream(device)
    if stream is None:
        return current, None
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, not on cuda:{device}")
    return stream.cuda_stream, (None if stream.cuda_stream == current else stream)


def _made(shape, dtype, device, other, returned=True):
    """A tensor made for a call on `other`, or on the current stream where that is None.  Its memory is
    of the call's stream: what was freed there, and is still in use there, is in use by work that
    comes before the call; memory of the current stream's could still be in use by work that
    nothing orders before it.  A `returned` tensor is read on the current stream, and its memory is
    not reused before the work queued there when it is freed is done."""
    if other is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _call_on(device, fn, *args):
    """Calls a C entry point with the device of this index current."""
    if _current_device() == device:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st != FA_OK:
        raise FaError(st, fn.__name__)


def _new_rows(name, t, dtype, device, Hkv, D):
    """A tensor of new rows [..., Hkv, D] whose heads are dense: (its tokens, their stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    shape = t.shape
    if len(shape) not in (3, 4) or shape[-2] != Hkv or shape[-1] != D:
        raise ValueError(f"{name} must be [B, n, {Hkv}, {D}] or [total, {Hkv}, {D}], got {tuple(shape)}")
    tokens = shape[0] if len(shape) == 3 else shape[0] * shape[1]
    if t.is_contiguous():
        return tokens, Hkv * D
    strides = t.stride()
    if strides[-1] != 1 or (Hkv > 1 and strides[-2] != D):
        raise ValueError(f"{name}: the heads of a token must be dense")
    if tokens <= 1:
        return tokens, Hkv * D
    if len(shape) == 3 or shape[1] == 1:
        return tokens, strides[0]
    if shape[0] > 1 and strides[0] != shape[1] * strides[1]:
        raise ValueError(f"{name}: the tokens of the batch must have one stride")
    return tokens, strides[1]


def fa_kv_append_paged_fp8(k_new, v_new, k_pages, v_pages, k_scales, v_scales, block_table, kv_lens,
                           cu_seqlens_new=None, stream=None):
    """Quantises new K/V rows into the 8-bit paged cache through fa_kv_append_paged_fp8.

    k_new/v_new bf16 or fp16: [B, n, Hkv, D] (n new tokens for each sequence), or packed
    [total, Hkv, D] with cu_seqlens_new int32 [B+1]; the tokens may be strided (a slice of a
    fused projection), the heads of a token dense. k_pages/v_pages float8_e4m3fn
    [num_pages, Hkv, page_size, D], k_scales/v_scales uint8 [num_pages, Hkv, page_size],
    block_table int32 [B, max_pages_per_seq]; kv_lens int32 [B] counts the new tokens: they
    become the last keys of their sequences.  Writes the pool in place; returns None."""
    lib = _fp8_lib or _load_fp8()
    device, num_pages, Hkv, page, D, B, max_pages = _fp8_pool(k_pages, v_pages, k_scales, v_scales, block_table)
    dtype = k_new.dtype if isinstance(k_new, torch.Tensor) else None
    if dtype not in _DTYPE:
        raise TypeError("k_new/v_new must be bf16 or fp16 tensors")
    total, k_stride = _new_rows("k_new", k_new, dtype, device, Hkv, D)
    v_stride = _new_rows("v_new", v_new, dtype, device, Hkv, D)[1]
    shape = k_new.shape
    if v_new.shape != shape:
        raise ValueError("k_new and v_new must have one shape")
    if not _is(kv_lens, _I32, device, (B,)):
        _refuse(("kv_lens", kv_lens, _I32, device, (B,)))
    cu = None
    if cu_seqlens_new is not None:
        if not _is(cu_seqlens_new, _I32, device, (B + 1,)):
            _refuse(("cu_seqlens_new", cu_seqlens_new, _I32, device, (B + 1,)))
        if len(shape) != 3:
            raise ValueError("with cu_seqlens_new, k_new and v_new are packed [total, Hkv, D]")
        cu = cu_seqlens_new.data_ptr()
    elif len(shape) != 4 or shape[0] != B:
        raise ValueError("without cu_seqlens_new, k_new and v_new are [B, n, Hkv, D]")
    _call_on(device, lib.fa_kv_append_paged_fp8, k_new.data_ptr(), v_new.data_ptr(), k_stride, v_stride, cu,
             block_table.data_ptr(), kv_lens.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
             k_scales.data_ptr(), v_scales.data_ptr(), B, total, Hkv, D, num_pages, page, max_pages,
             _DTYPE[dtype], _stream_on(device, stream)[0])


def fa_kv_read_paged_fp8(k_pages, v_pages, k_scales, v_scales, block_table, cu_seqlens, total=None,
                         kv_starts=None, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """Reads rows of the 8-bit paged cache back through fa_kv_read_paged_fp8.

    Packed rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 receive keys kv_starts[b] (0), ... of
    sequence b; cu_seqlens int32 [B+1], kv_starts int32 [B], on the device.  k_out/v_out
    [total, Hkv, D] are given, or made here from ``total`` and ``dtype``; rows behind the last
    sequence are not written.  Returns (k, v)."""
    lib = _fp8_lib or _load_fp8()
    device, num_pages, Hkv, page, D, B, max_pages = _fp8_pool(k_pages, v_pages, k_scales, v_scales, block_table)
    if not _is(cu_seqlens, _I32, device, (B + 1,)):
        _refuse(("cu_seqlens", cu_seqlens, _I32, device, (B + 1,)))
    if kv_starts is not None and not _is(kv_starts, _I32, device, (B,)):
        _refuse(("kv_starts", kv_starts, _I32, device, (B,)))
    given = k_out if k_out is not None else v_out
    if given is not None:
        dtype = given.dtype
        if total is None:
            total = given.shape[0]
    elif total is None:
        raise ValueError("give total, the packed rows, or k_out and v_out")
    if dtype not in _DTYPE:
        raise TypeError("k/v are read as bf16 or fp16")
    handle, other = _stream_on(device, stream)
    shape = (int(total), Hkv, D)
    if k_out is None:
        k_out = _made(shape, dtype, k_pages.device, other)
    if v_out is None:
        v_out = _made(shape, dtype, k_pages.device, other)
    if not (_is(k_out, dtype, device, shape) and _is(v_out, dtype, device, shape)):
        _refuse(("k_out", k_out, dtype, device, shape), ("v_out", v_out, dtype, device, shape))
    _call_on(device, lib.fa_kv_read_paged_fp8, k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
             v_scales.data_ptr(), block_table.data_ptr(), None if kv_starts is None else kv_starts.data_ptr(),
             cu_seqlens.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), B, shape[0], Hkv, D, num_pages, page,
             max_pages, _DTYPE[dtype], handle)
    return k_out, v_out


def fa_decode_splitkv_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, kv_lens,
                                causal: bool = True, scale: float | None = None, num_splits: int = 0,
                                workspace=None, out=None, lse=None, stream=None):
    """Split-KV decode over the 8-bit paged cache through fa_decode_splitkv_paged_fp8.

    q [B, Sq, Hq, D] bf16 or fp16; the pool as fa_kv_append_paged_fp8 writes it; kv_lens
    int32 [B].  workspace: a CUDA uint8 tensor of at least fa_decode_workspace_bytes(B * Sq,
    Hq, D, num_splits) bytes, or None to allocate one.  Returns (o like q, lse fp32
    [B, Hq, Sq])."""
    lib = _fp8_lib or _load_fp8()
    device, num_pages, Hkv, page, D, B, max_pages = _fp8_pool(k_pages, v_pages, k_scales, v_scales, block_table)
    dtype = q.dtype if isinstance(q, torch.Tensor) else None
    if dtype not in _DTYPE:
        raise TypeError("q must be a bf16 or fp16 tensor")
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != D:
        raise ValueError(f"q must be [{B}, Sq, Hq, {D}], got {tuple(shape)}")
    Sq, Hq = shape[1], shape[2]
    if not (_is(q, dtype, device, shape) and _is(kv_lens, _I32, device, (B,))):
        _refuse(("q", q, dtype, device, shape), ("kv_lens", kv_lens, _I32, device, (B,)))
    handle, other = _stream_on(device, stream)
    ns = int(num_splits)
    if workspace is None:
        room = ns
        if room <= 0:
            # Sizes the workspace and is not passed on: the default may be 1, and a caller's 1
            # forbids cutting.
            with torch.cuda.device(device):
                room = lib.fa_decode_default_splits(B, Hkv, page * max_pages, 0)
        workspace = _made(max(16, lib.fa_decode_workspace_bytes(B * Sq, Hq, D, room)), _U8, q.device, other,
                          returned=False)
    elif not _is(workspace, _U8, device, None):
        _refuse(("workspace", workspace, _U8, device, None))
    if out is None:
        out = _made(shape, dtype, q.device, other)
    elif not _is(out, dtype, device, shape):
        _refuse(("out", out, dtype, device, shape))
    if lse is None:
        lse = _made((B, Hq, Sq), _F32, q.device, other)
    elif not _is(lse, _F32, device, (B, Hq, Sq)):
        _refuse(("lse", lse, _F32, device, (B, Hq, Sq)))
    _call_on(device, lib.fa_decode_splitkv_paged_fp8, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
             k_scales.data_ptr(), v_scales.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(),
             out.data_ptr(), lse.data_ptr(), B, Sq, Hq, Hkv, D, num_pages, page, max_pages,
             1.0 / math.sqrt(D) if scale is None else float(scale), 1 if causal else 0, ns,
             workspace.data_ptr(), workspace.numel(), _DTYPE[dtype], handle)
    return out, lse
