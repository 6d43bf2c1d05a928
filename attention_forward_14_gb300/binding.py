"""ctypes binding of libattn_fwd.so (the C ABI in include/attn_fwd.h).

Argument marshalling only: every step of the forward and backward runs in the
library's CUDA kernels.  PyTorch provides device memory and streams.  If the library is
missing or cannot be loaded, every call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(HERE, "libattn_fwd.so")
CHECKED_LIB_PATH = os.path.join(HERE, "libattn_fwd_checked.so")  # every computed index bounds-checked
_lib = None
_lock = threading.Lock()

FP16, BF16 = 0, 1
ERRORS = {
    0: "ATTN_OK", -1: "ATTN_ERR_NULL", -2: "ATTN_ERR_SHAPE", -3: "ATTN_ERR_HEADDIM", -4: "ATTN_ERR_DTYPE",
    -5: "ATTN_ERR_SCALE", -6: "ATTN_ERR_ALIGN", -7: "ATTN_ERR_ARCH", -8: "ATTN_ERR_CUDA", -9: "ATTN_ERR_WATCHDOG",
    -10: "ATTN_ERR_BUILD",
}
# Every function include/attn_fwd.h declares.
EXPORTS = ["attn_fwd", "attn_fwd_host", "attn_fwd_varlen", "attn_fwd_fp8", "attn_fwd_splitkv", "attn_fwd_splitkv_workspace_bytes",
           "attn_fwd_splitkv_default_splits", "attn_fwd_splitkv_noalloc", "attn_last_error", "attn_fwd_status", "attn_fwd_status_clear",
           "attn_fwd_debug_status", "attn_fwd_sched_pin_slot", "attn_fwd_bounds_selftest", "attn_bwd_bounds_selftest",
           "attn_fwd_watchdog_selftest", "attn_bwd_watchdog_selftest", "attn_version", "attn_bwd", "attn_bwd_workspace_bytes", "attn_bwd_varlen",
           "attn_bwd_varlen_workspace_bytes", "attn_fwd_kvcache", "attn_fwd_kvcache_paged", "attn_qk_norm_rope",
           "attn_qk_norm_rope_bwd", "attn_qk_norm_rope_bwd_workspace_bytes", "attn_kvcache_append_paged",
           "attn_fwd_kvcache_paged_fp8", "attn_fwd_kvcache_paged_fp8_workspace_bytes"]


class AttnError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{ERRORS.get(code, code)}: {message}")
        self.code = code


def lib_path() -> str:
    return _LIB_PATH


def _bind(lib):
    i64, vp, c_int, c_float = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.attn_fwd.restype = c_int
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int, c_float, c_int, vp]
    lib.attn_fwd_host.restype = c_int
    lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                  i64, i64, i64, i64, i64, c_int, c_float, c_int, vp]
    lib.attn_fwd_fp8.restype = c_int
    lib.attn_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int, c_float, c_float, c_float,
                                 c_float, vp]
    lib.attn_fwd_varlen.restype = c_int
    lib.attn_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, c_int, c_float,
                                    c_int, vp]
    lib.attn_fwd_splitkv.restype = c_int
    lib.attn_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int, c_float, c_int, c_int,
                                     vp, i64, vp]
    lib.attn_fwd_splitkv_workspace_bytes.restype = i64
    lib.attn_fwd_splitkv_workspace_bytes.argtypes = [i64, i64, i64, i64, c_int]
    lib.attn_fwd_splitkv_default_splits.restype = c_int
    lib.attn_fwd_splitkv_default_splits.argtypes = [i64, i64, i64, i64, i64, c_int]
    lib.attn_fwd_splitkv_noalloc.restype = c_int
    lib.attn_fwd_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int, c_float, c_int,
                                             c_int, vp]
    lib.attn_fwd_kvcache.restype = c_int
    lib.attn_fwd_kvcache.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, c_int, c_float,
                                     c_int, c_int, vp, i64, vp]
    lib.attn_fwd_kvcache_paged.restype = c_int
    lib.attn_fwd_kvcache_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64,
                                           i64, c_int, c_float, c_int, c_int, vp, i64, vp]
    lib.attn_last_error.restype = ctypes.c_char_p
    lib.attn_last_error.argtypes = []
    lib.attn_fwd_status.restype = c_int
    lib.attn_fwd_status.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.attn_fwd_status_clear.restype = c_int
    lib.attn_fwd_status_clear.argtypes = []
    lib.attn_fwd_debug_status.restype = c_int
    lib.attn_fwd_debug_status.argtypes = []
    lib.attn_fwd_sched_pin_slot.restype = c_int
    lib.attn_fwd_sched_pin_slot.argtypes = [c_int]
    lib.attn_fwd_bounds_selftest.restype = c_int
    lib.attn_fwd_bounds_selftest.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_float, c_int, vp]
    lib.attn_bwd_watchdog_selftest.restype = c_int
    lib.attn_bwd_watchdog_selftest.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int,
                                               c_float, c_int, vp, i64, c_int, c_int, vp]
    lib.attn_bwd_bounds_selftest.restype = c_int
    lib.attn_bwd_bounds_selftest.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_float,
                                             c_int, vp, i64, vp]
    lib.attn_fwd_watchdog_selftest.restype = c_int
    lib.attn_fwd_watchdog_selftest.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int, c_float,
                                               c_int, c_int, c_int, vp]
    lib.attn_version.restype = ctypes.c_char_p
    lib.attn_version.argtypes = []
    lib.attn_bwd.restype = c_int
    lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int, c_float, c_int,
                             vp, i64, vp]
    lib.attn_bwd_workspace_bytes.restype = i64
    lib.attn_bwd_workspace_bytes.argtypes = [i64, i64, i64, i64]
    lib.attn_bwd_varlen.restype = c_int
    lib.attn_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64,
                                    c_int, c_float, c_int, vp, i64, vp]
    lib.attn_bwd_varlen_workspace_bytes.restype = i64
    lib.attn_bwd_varlen_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    lib.attn_qk_norm_rope.restype = c_int
    lib.attn_qk_norm_rope.argtypes = [vp] * 13 + [i64] * 8 + [c_int, c_float, c_int, vp]
    lib.attn_qk_norm_rope_bwd.restype = c_int
    lib.attn_qk_norm_rope_bwd.argtypes = [vp] * 19 + [i64] * 8 + [c_int, c_float, c_int, vp, i64, vp]
    lib.attn_qk_norm_rope_bwd_workspace_bytes.restype = i64
    lib.attn_qk_norm_rope_bwd_workspace_bytes.argtypes = [i64]
    lib.attn_kvcache_append_paged.restype = c_int
    lib.attn_kvcache_append_paged.argtypes = [vp] * 13 + [i64] * 10 + [c_int, c_int, vp]
    lib.attn_fwd_kvcache_paged_fp8.restype = c_int
    lib.attn_fwd_kvcache_paged_fp8.argtypes = [vp] * 9 + [i64] * 9 + [c_int, c_float, c_int, vp, i64, vp]
    lib.attn_fwd_kvcache_paged_fp8_workspace_bytes.restype = i64
    lib.attn_fwd_kvcache_paged_fp8_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    return lib


def load(path: str | None = None):
    """Load (once) and bind the C ABI.  Raises if the library is absent."""
    global _lib
    if path is None and _lib is not None:  # the common case: no lock
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _LIB_PATH
        if not os.path.exists(p):
            raise AttnError(-8, f"{p} not built; run python -m attention_forward_14_gb300.build")
        lib = _bind(ctypes.CDLL(p))
        if path is None:
            _lib = lib
        return lib


def _check(rc: int, lib) -> int:
    if rc < 0:
        raise AttnError(rc, lib.attn_last_error().decode(errors="replace"))
    return rc


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return FP16
    if t.dtype == torch.bfloat16:
        return BF16
    raise AttnError(-4, f"unsupported dtype {t.dtype}")


def _stream_handle(stream, device):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(stream, device):
    """The same as a number, without building torch's stream object for the
    current one (2 us of the 20 that a small call takes on the host)."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    current = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if current is None:
        return torch.cuda.current_stream(device).cuda_stream
    return current(device.index)


class _OnDevice:
    """Make `device` current for the call (the library works on the current
    device); does nothing when it already is."""
    __slots__ = ("ctx",)

    def __init__(self, device):
        import torch
        idx = device.index if device.index is not None else torch.cuda.current_device()
        self.ctx = None if idx == torch.cuda.current_device() else torch.cuda.device(idx)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def attn_fwd(q, k, v, causal: bool = False, scale: float | None = None, o=None, lse=None,
             return_lse: bool = True, stream=None):
    """O = softmax(scale * Q K^T [+ causal]) V on the GPU.

    q: [b, h, sq, d], k/v: [b, h, sk, d] contiguous CUDA tensors (fp16 or
    bf16, same dtype and device).  ``scale`` defaults to 1/sqrt(d).  ``o``
    and ``lse`` may be given (preallocated outputs); otherwise they are
    allocated with torch.  Returns (o, lse) -- lse is None when
    ``return_lse`` is False and no ``lse`` was given.
    """
    import torch
    lib = load()
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise AttnError(-2, "q, k, v must be 4-D [b, h, s, d]")
    b, h, sq, d = q.shape
    sk = k.shape[2]
    if tuple(k.shape) != (b, h, sk, d) or tuple(v.shape) != (b, h, sk, d):
        raise AttnError(-2, f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    if not (q.dtype == k.dtype == v.dtype):
        raise AttnError(-4, "q, k, v dtypes differ")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError(-2, f"{name} must be a contiguous CUDA tensor")
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((b, h, sq), dtype=torch.float32, device=q.device)
    if o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous():
        raise AttnError(-2, "o must be a contiguous tensor shaped and typed like q")
    if lse is not None and (tuple(lse.shape) != (b, h, sq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise AttnError(-2, "lse must be contiguous fp32 [b, h, sq]")
    with _OnDevice(q.device):
        rc = lib.attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                          lse.data_ptr() if lse is not None else None,
                          b, h, sq, sk, d, int(bool(causal)), float(scale), _dtype_code(q),
                          _stream_handle(stream, q.device))
    _check(rc, lib)
    return o, lse


def attn_fwd_fp8(q, k, v, causal: bool = False, scale: float | None = None, descale_q: float = 1.0,
                 descale_k: float = 1.0, descale_v: float = 1.0, o=None, lse=None, stream=None):
    """e4m3 inputs [b, h, s, d], d = 64 or 128 (torch.float8_e4m3fn CUDA tensors) with
    per-tensor descales; returns (o bf16 [b, h, sq, d], lse fp32)."""
    import torch
    lib = load()
    b, h, sq, d = q.shape
    sk = k.shape[2]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float8_e4m3fn:
            raise AttnError(-4, f"{name} must be a contiguous CUDA float8_e4m3fn tensor")
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    if o is None:
        o = torch.empty((b, h, sq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((b, h, sq), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib.attn_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), b, h, sq, sk,
                              d, int(bool(causal)), float(scale), float(descale_q), float(descale_k),
                              float(descale_v), _stream_handle(stream, q.device))
    _check(rc, lib)
    return o, lse


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                    causal: bool = False, scale: float | None = None, o=None, lse=None, stream=None):
    """Packed variable-length forward.  q: [total_q, h, d], k/v: [total_k,
    h, d] CUDA tensors; cu_seqlens_*: int32 CUDA tensors [batch + 1].
    Returns (o [total_q, h, d], lse [h, total_q])."""
    import torch
    lib = load()
    total_q, h, d = q.shape
    total_k = k.shape[0]
    batch = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != batch + 1:
        raise AttnError(-2, "cu_seqlens_q and cu_seqlens_k sizes differ")
    for name, t in (("q", q), ("k", k), ("v", v), ("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError(-2, f"{name} must be a contiguous CUDA tensor")
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32:
        raise AttnError(-4, "cu_seqlens must be int32")
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((h, total_q), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib.attn_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                 cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), batch, h, total_q, total_k,
                                 int(max_seqlen_q), int(max_seqlen_k), d, int(bool(causal)), float(scale),
                                 _dtype_code(q), _stream_handle(stream, q.device))
    _check(rc, lib)
    return o, lse


def splitkv_workspace_bytes(b, h, sq, d, num_splits) -> int:
    lib = load()
    return _check(int(lib.attn_fwd_splitkv_workspace_bytes(b, h, sq, d, num_splits)), lib)


def splitkv_default_splits(b, h, sq, sk, d, causal=False) -> int:
    lib = load()
    return _check(int(lib.attn_fwd_splitkv_default_splits(b, h, sq, sk, d, int(bool(causal)))), lib)


def attn_fwd_splitkv(q, k, v, causal: bool = False, scale: float | None = None, num_splits: int | None = None,
                     o=None, lse=None, workspace=None, stream=None):
    """Split-KV forward (same result as attn_fwd).  ``num_splits`` defaults
    to the library's choice for the device; ``workspace`` (a CUDA uint8
    tensor) is allocated with torch when not given.  Returns (o, lse)."""
    import torch
    lib = load()
    b, h, sq, d = q.shape
    sk = k.shape[2]
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    if num_splits is None:
        with torch.cuda.device(q.device):
            num_splits = splitkv_default_splits(b, h, sq, sk, d, causal)
    need = splitkv_workspace_bytes(b, h, sq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((b, h, sq), dtype=torch.float32, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("lse", lse)):
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError(-2, f"{name} must be a contiguous CUDA tensor")
    with torch.cuda.device(q.device):
        rc = lib.attn_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                  b, h, sq, sk, d, int(bool(causal)), float(scale), _dtype_code(q), int(num_splits),
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream, q.device))
    _check(rc, lib)
    return o, lse


def attn_fwd_kvcache(q, k_cache, v_cache, cache_seqlens, k_new=None, v_new=None, causal: bool = False,
                     scale: float | None = None, num_splits: int | None = None, o=None, lse=None, workspace=None,
                     stream=None):
    """Attention of q [b, h, sq, d] against a KV cache [b, h, s_cache, d]
    whose batch element i holds cache_seqlens[i] valid tokens (int32 CUDA
    tensor [b]).  With k_new / v_new [b, h, s_new, d] the new rows are
    first written into the cache at each element's length (the caches are
    updated in place; cache_seqlens is not) and attended to as well.
    ``num_splits`` defaults to the library's split-KV choice for s_cache.
    Returns (o, lse)."""
    import torch
    lib = load()
    b, h, sq, d = q.shape
    s_cache = k_cache.shape[2]
    if tuple(k_cache.shape) != (b, h, s_cache, d) or tuple(v_cache.shape) != (b, h, s_cache, d):
        raise AttnError(-2, f"cache shapes {tuple(k_cache.shape)} / {tuple(v_cache.shape)} do not match q")
    if (k_new is None) != (v_new is None):
        raise AttnError(-1, "k_new and v_new must both be given or both be None")
    s_new = 0 if k_new is None else k_new.shape[2]
    if k_new is not None and (tuple(k_new.shape) != (b, h, s_new, d) or tuple(v_new.shape) != (b, h, s_new, d)):
        raise AttnError(-2, "k_new / v_new must be [b, h, s_new, d]")
    if cache_seqlens.dtype != torch.int32 or cache_seqlens.numel() != b:
        raise AttnError(-4, "cache_seqlens must be an int32 tensor of b elements")
    tensors = [("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("cache_seqlens", cache_seqlens)]
    if k_new is not None:
        tensors += [("k_new", k_new), ("v_new", v_new)]
    for name, t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError(-2, f"{name} must be a contiguous CUDA tensor")
        if name != "cache_seqlens" and t.dtype != q.dtype:
            raise AttnError(-4, f"{name} dtype differs from q")
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    if num_splits is None:
        with torch.cuda.device(q.device):
            num_splits = splitkv_default_splits(b, h, sq, max(s_cache, 1), d, causal)
        num_splits = max(1, min(num_splits, (s_cache + 127) // 128))
    need = splitkv_workspace_bytes(b, h, sq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((b, h, sq), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib.attn_fwd_kvcache(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                  k_new.data_ptr() if k_new is not None else None,
                                  v_new.data_ptr() if v_new is not None else None,
                                  cache_seqlens.data_ptr(), o.data_ptr(), lse.data_ptr(), b, h, sq, s_cache, s_new,
                                  d, int(bool(causal)), float(scale), _dtype_code(q), int(num_splits),
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream, q.device))
    _check(rc, lib)
    return o, lse


def attn_fwd_kvcache_paged(q, k_pool, v_pool, cache_seqlens, block_table, k_new=None, v_new=None,
                           causal: bool = False, scale: float | None = None, num_splits: int | None = None, o=None,
                           lse=None, workspace=None, stream=None):
    """attn_fwd_kvcache over a paged cache: k_pool / v_pool [num_pages,
    page_size, h, d], block_table int32 [b, pages_per_seq] (CUDA tensors).
    Returns (o, lse)."""
    import torch
    lib = load()
    b, h, sq, d = q.shape
    num_pages, page_size = k_pool.shape[0], k_pool.shape[1]
    if tuple(k_pool.shape) != (num_pages, page_size, h, d) or tuple(v_pool.shape) != tuple(k_pool.shape):
        raise AttnError(-2, f"pool shapes {tuple(k_pool.shape)} / {tuple(v_pool.shape)} do not match q")
    if block_table.dim() != 2 or block_table.shape[0] != b or block_table.dtype != torch.int32:
        raise AttnError(-2, "block_table must be int32 [b, pages_per_seq]")
    pages_per_seq = block_table.shape[1]
    if (k_new is None) != (v_new is None):
        raise AttnError(-1, "k_new and v_new must both be given or both be None")
    s_new = 0 if k_new is None else k_new.shape[2]
    if k_new is not None and (tuple(k_new.shape) != (b, h, s_new, d) or tuple(v_new.shape) != (b, h, s_new, d)):
        raise AttnError(-2, "k_new / v_new must be [b, h, s_new, d]")
    if cache_seqlens.dtype != torch.int32 or cache_seqlens.numel() != b:
        raise AttnError(-4, "cache_seqlens must be an int32 tensor of b elements")
    tensors = [("q", q), ("k_pool", k_pool), ("v_pool", v_pool), ("cache_seqlens", cache_seqlens),
               ("block_table", block_table)]
    if k_new is not None:
        tensors += [("k_new", k_new), ("v_new", v_new)]
    for name, t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError(-2, f"{name} must be a contiguous CUDA tensor")
        if name not in ("cache_seqlens", "block_table") and t.dtype != q.dtype:
            raise AttnError(-4, f"{name} dtype differs from q")
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    cap = pages_per_seq * page_size
    if num_splits is None:
        with torch.cuda.device(q.device):
            num_splits = splitkv_default_splits(b, h, sq, max(cap, 1), d, causal)
        num_splits = max(1, min(num_splits, (cap + 127) // 128))
    need = splitkv_workspace_bytes(b, h, sq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((b, h, sq), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib.attn_fwd_kvcache_paged(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                        k_new.data_ptr() if k_new is not None else None,
                                        v_new.data_ptr() if v_new is not None else None,
                                        cache_seqlens.data_ptr(), block_table.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                        b, h, sq, num_pages, page_size, pages_per_seq, s_new, d, int(bool(causal)),
                                        float(scale), _dtype_code(q), int(num_splits), workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), _stream_handle(stream, q.device))
    _check(rc, lib)
    return o, lse


def attn_fwd_host(q_host, k_host, v_host, o_host, lse_host, q_dev, k_dev, v_dev, o_dev, lse_dev,
                  causal: bool = False, scale: float | None = None, stream=None):
    """End-to-end call on host (ideally pinned) tensors through the C ABI:
    host->device copies, the forward, device->host copies, all enqueued on
    ``stream``.  The caller synchronises the stream before reading o_host."""
    import torch
    lib = load()
    b, h, sq, d = q_host.shape
    sk = k_host.shape[2]
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    with torch.cuda.device(q_dev.device):
        rc = lib.attn_fwd_host(q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(), o_host.data_ptr(),
                               lse_host.data_ptr() if lse_host is not None else None,
                               q_dev.data_ptr(), k_dev.data_ptr(), v_dev.data_ptr(), o_dev.data_ptr(),
                               lse_dev.data_ptr() if lse_dev is not None else None,
                               b, h, sq, sk, d, int(bool(causal)), float(scale), _dtype_code(q_host),
                               _stream_handle(stream, q_dev.device))
    _check(rc, lib)


def status():
    """(code, block, warp, site) of the device watchdog (synchronises)."""
    lib = load()
    out = (ctypes.c_uint32 * 4)()
    _check(lib.attn_fwd_status(out), lib)
    return tuple(int(x) for x in out)


def status_clear():
    lib = load()
    _check(lib.attn_fwd_status_clear(), lib)


def watchdog_selftest(q, k, v, o, lse, causal, scale, withheld_load: int, timeout_ms: int):
    """Run the forward with one K/V load withheld; returns the recorded code."""
    import torch
    lib = load()
    b, h, sq, d = q.shape
    sk = k.shape[2]
    with torch.cuda.device(q.device):
        rc = lib.attn_fwd_watchdog_selftest(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                            lse.data_ptr() if lse is not None else None,
                                            b, h, sq, sk, d, int(bool(causal)), float(scale), _dtype_code(q),
                                            int(withheld_load), int(timeout_ms),
                                            _stream_handle(None, q.device))
    return _check(rc, lib)


def bwd_watchdog_selftest(q, k, v, o, dout, lse, causal, scale, withheld_load: int, timeout_ms: int):
    """Run the backward with one query-tile load withheld in every CTA;
    returns the recorded code.  The gradients are not meaningful."""
    import torch
    lib = load()
    b, h, sq, d = q.shape
    sk = k.shape[2]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = bwd_workspace_bytes(b, h, sq, d)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib.attn_bwd_watchdog_selftest(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                                            lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                            b, h, sq, sk, d, int(bool(causal)), float(scale), _dtype_code(q),
                                            ws.data_ptr(), nbytes, int(withheld_load), int(timeout_ms),
                                            _stream_handle(None, q.device))
    return _check(rc, lib)


def bwd_workspace_bytes(b: int, h: int, sq: int, d: int) -> int:
    lib = load()
    return _check(int(lib.attn_bwd_workspace_bytes(b, h, sq, d)), lib)


def attn_bwd(q, k, v, o, dout, lse, causal: bool = False, scale: float | None = None, dq=None, dk=None, dv=None,
             workspace=None, stream=None):
    """Gradients (dq, dk, dv) of attn_fwd for the output gradient ``dout``.

    q, o, dout: [b, h, sq, 128]; k, v: [b, h, sk, 128] contiguous CUDA
    tensors of one dtype (fp16 or bf16); lse: fp32 [b, h, sq] from the
    forward.  Outputs and the workspace (a CUDA uint8 tensor of at least
    bwd_workspace_bytes bytes) are allocated with torch when not given."""
    import torch
    lib = load()
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise AttnError(-2, "q, k, v must be 4-D [b, h, s, d]")
    b, h, sq, d = q.shape
    sk = k.shape[2]
    if tuple(k.shape) != (b, h, sk, d) or tuple(v.shape) != (b, h, sk, d) or o.shape != q.shape or \
            dout.shape != q.shape or tuple(lse.shape) != (b, h, sq):
        raise AttnError(-2, "shape mismatch among q, k, v, o, dout, lse")
    if not (q.dtype == k.dtype == v.dtype == o.dtype == dout.dtype) or lse.dtype != torch.float32:
        raise AttnError(-4, "q, k, v, o, dout must share a dtype; lse must be fp32")
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    if dq is None:
        dq = torch.empty_like(q)
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    if workspace is None:
        with torch.cuda.device(q.device):
            need = bwd_workspace_bytes(b, h, sq, d)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("lse", lse), ("dq", dq), ("dk", dk),
                    ("dv", dv), ("workspace", workspace)):
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError(-2, f"{name} must be a contiguous CUDA tensor")
    with torch.cuda.device(q.device):
        rc = lib.attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), b, h, sq, sk, d, int(bool(causal)),
                          float(scale), _dtype_code(q), workspace.data_ptr(),
                          workspace.numel() * workspace.element_size(), _stream_handle(stream, q.device))
    _check(rc, lib)
    return dq, dk, dv


def attn_bwd_varlen(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                    causal: bool = False, scale: float | None = None, dq=None, dk=None, dv=None, workspace=None,
                    stream=None):
    """Gradients (dq, dk, dv) of attn_fwd_varlen.  q, o, dout: [total_q, h, d];
    k, v: [total_k, h, d] of one dtype; lse: fp32 [h, total_q];
    cu_seqlens_q / _k: int32 CUDA tensors [batch + 1]."""
    import torch
    lib = load()
    total_q, h, d = q.shape
    total_k = k.shape[0]
    batch = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != batch + 1 or tuple(k.shape) != (total_k, h, d) or tuple(v.shape) != (total_k, h, d) \
            or o.shape != q.shape or dout.shape != q.shape or tuple(lse.shape) != (h, total_q):
        raise AttnError(-2, "shape mismatch among q, k, v, o, dout, lse, cu_seqlens")
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        need = _check(int(lib.attn_bwd_varlen_workspace_bytes(batch, h, total_q, max_seqlen_q, d)), lib)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("lse", lse), ("dq", dq), ("dk", dk),
                    ("dv", dv), ("workspace", workspace), ("cu_seqlens_q", cu_seqlens_q),
                    ("cu_seqlens_k", cu_seqlens_k)):
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError(-2, f"{name} must be a contiguous CUDA tensor")
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32:
        raise AttnError(-4, "cu_seqlens must be int32")
    with torch.cuda.device(q.device):
        rc = lib.attn_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                                 lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), cu_seqlens_q.data_ptr(),
                                 cu_seqlens_k.data_ptr(), batch, h, total_q, total_k, int(max_seqlen_q),
                                 int(max_seqlen_k), d, int(bool(causal)), float(scale), _dtype_code(q),
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 _stream_handle(stream, q.device))
    _check(rc, lib)
    return dq, dk, dv


_Strides = ctypes.c_int64 * 3


def _as_dense(name, t):
    """A [b, h, s, d] tensor, or a packed [total, h, d] one as b = 1: its shape and its strides (b, head, token)."""
    shape, st = t.shape, t.stride()
    if len(shape) == 4:
        b, h, s, d = shape
        sb, sh, ss, sd = st
    elif len(shape) == 3:
        s, h, d = shape
        ss, sh, sd = st
        b, sb = 1, 0
    else:
        raise AttnError(-2, f"{name} must be [b, h, s, d] or [total, h, d]")
    if sd != 1 and d > 1 and t.numel() > 0:
        raise AttnError(-2, f"the {d} values of a head of {name} must be contiguous")
    # an axis of one has no stride of its own
    return b, h, s, d, _Strides(sb if b > 1 else 0, sh if h > 1 else 0, ss if s > 1 else 0)


def _output(name, t, ref):
    """An output shaped and typed like its input `ref`: allocated (contiguous) or checked; its strides as above."""
    import torch
    if t is None:
        t = torch.empty_like(ref, memory_format=torch.contiguous_format)
    elif t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
        raise AttnError(-2, f"{name} must be shaped and typed like its input, on its device")
    return t, _as_dense(name, t)[4]


def _rotation(cos, sin, device):
    """(pointer, pointer, rot, table_len) of the rotation's tables; nothing for none."""
    import torch
    if cos is None or sin is None:
        if cos is not sin:
            raise AttnError(-1, "cos and sin must both be given or both be None")
        return None, None, 0, 0
    if cos.dim() != 2 or cos.shape != sin.shape:
        raise AttnError(-2, "cos and sin must be [table_len, rot / 2]")
    if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.device != device or sin.device != device or \
            not (cos.is_contiguous() and sin.is_contiguous()):
        raise AttnError(-4, "cos and sin must be contiguous fp32 tensors on the inputs' device")
    length, half = cos.shape
    return cos.data_ptr(), sin.data_ptr(), 2 * half, length


def _positions(positions, b, s, packed, cos, device):
    """(pointer, stride over b) of the positions of a dense [b, s] or packed [total] batch."""
    import torch
    if positions is None:
        if packed and cos is not None:
            raise AttnError(-1, "a packed batch needs positions: they start again in every sequence")
        return None, 0
    shape = positions.shape
    if positions.dtype != torch.int32 or positions.device != device or \
            not (shape == (s,) or (not packed and shape == (b, s))):
        raise AttnError(-4, f"positions must be int32 of {s} or (not packed) {b} x {s} on the inputs' device")
    st = positions.stride()
    if st[-1] != 1 and s > 1:
        raise AttnError(-2, "the positions of a sequence must be contiguous")
    return positions.data_ptr(), st[0] if len(st) == 2 and b > 1 else 0


def _norm_inputs(q, k, q_weight, k_weight):
    """Shapes and strides of q and k, and the pointers of their weights."""
    b, h, s, d, qs = _as_dense("q", q)
    bk, hkv, sk, dk, ks = _as_dense("k", k)
    if bk != b or sk != s or dk != d or q.dim() != k.dim():
        raise AttnError(-2, f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)}")
    dt, dev = q.dtype, q.device
    if not q.is_cuda or k.dtype != dt or k.device != dev:
        raise AttnError(-4, "q and k must be CUDA tensors of one dtype on one device")
    for w in (q_weight, k_weight):
        if w is not None and (w.shape != (d,) or w.dtype != dt or w.device != dev or not w.is_contiguous()):
            raise AttnError(-2, f"norm weights must be contiguous [{d}] tensors typed like q, on its device")
    return (b, h, hkv, s, d, qs, ks, q_weight.data_ptr() if q_weight is not None else None,
            k_weight.data_ptr() if k_weight is not None else None)


def _used_on(stream, *tensors):
    """Tensors allocated here for a call on a stream that was given: their
    memory is not handed out again before that stream is done with them."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def attn_qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps: float = 1e-6,
                      interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and the rotary rotation, in one
    pass, into the layout the attention reads.

    q: [b, h, s, d] and k: [b, h_kv, s, d], or packed [total, h, d] and
    [total, h_kv, d]; fp16 or bf16, any strides (multiples of 8 elements) with
    contiguous heads, so views of a fused projection need no copy.
    ``q_weight`` / ``k_weight`` [d] (None: no norm); ``cos`` / ``sin`` fp32
    [table_len, rot / 2] (None: no rotation); ``positions`` int32 [b, s], [s]
    or (packed) [total], None: 0..s-1.  ``interleaved``: adjacent pairs turn
    instead of pairs (i, i + rot/2).  Negative positions are padding (zeros).
    Returns (q_out, k_out), contiguous unless given."""
    lib = load()
    b, h, hkv, s, d, qs, ks, wq, wk = _norm_inputs(q, k, q_weight, k_weight)
    dt, dev = _dtype_code(q), q.device
    c, sn, rot, length = _rotation(cos, sin, dev)
    pos, pos_b = _positions(positions, b, s, q.dim() == 3, cos, dev)
    q_out, qos = _output("q_out", q_out, q)
    k_out, kos = _output("k_out", k_out, k)
    with _OnDevice(dev):
        rc = lib.attn_qk_norm_rope(q.data_ptr(), k.data_ptr(), wq, wk, c, sn, pos, q_out.data_ptr(), k_out.data_ptr(),
                                   qs, ks, qos, kos, b, h, hkv, s, d, rot, length, pos_b, 1 if interleaved else 0, eps,
                                   dt, _raw_stream(stream, dev))
    if rc < 0:
        _check(rc, lib)
    _used_on(stream, q_out, k_out)
    return q_out, k_out


def attn_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of attn_qk_norm_rope for the gradients of its outputs:
    (dq, dk, dq_weight, dk_weight); the weights' gradients are fp32 [d], None
    for a weight that is None.  ``dq`` / ``dk`` may be given (for example
    slices of the fused projection's gradient), with any strides; ``workspace``
    is a CUDA uint8 tensor of qk_norm_rope_bwd_workspace_bytes(d) bytes."""
    import torch
    lib = load()
    b, h, hkv, s, d, qs, ks, wq, wk = _norm_inputs(q, k, q_weight, k_weight)
    dt, dev = _dtype_code(q), q.device
    c, sn, rot, length = _rotation(cos, sin, dev)
    pos, pos_b = _positions(positions, b, s, q.dim() == 3, cos, dev)
    dq_out, gqs = _output("dq_out", dq_out, q)
    dk_out, gks = _output("dk_out", dk_out, k)
    dq, dqs = _output("dq", dq, q)
    dk, dks = _output("dk", dk, k)
    dwq = torch.empty(d, dtype=torch.float32, device=dev) if wq is not None else None
    dwk = torch.empty(d, dtype=torch.float32, device=dev) if wk is not None else None
    if workspace is None and (wq is not None or wk is not None):
        workspace = torch.empty(qk_norm_rope_bwd_workspace_bytes(d), dtype=torch.uint8, device=dev)
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise AttnError(-2, "workspace must be a contiguous tensor on the inputs' device")
    with _OnDevice(dev):
        rc = lib.attn_qk_norm_rope_bwd(dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), wq, wk, c, sn,
                                       pos, dq.data_ptr(), dk.data_ptr(), dwq.data_ptr() if wq is not None else None,
                                       dwk.data_ptr() if wk is not None else None, gqs, gks, qs, ks, dqs, dks, b, h,
                                       hkv, s, d, rot, length, pos_b, 1 if interleaved else 0, eps, dt,
                                       workspace.data_ptr() if workspace is not None else None,
                                       workspace.nbytes if workspace is not None else 0, _raw_stream(stream, dev))
    if rc < 0:
        _check(rc, lib)
    _used_on(stream, dq, dk, dwq, dwk, workspace)
    return dq, dk, dwq, dwk


def qk_norm_rope_bwd_workspace_bytes(d: int) -> int:
    lib = load()
    return _check(int(lib.attn_qk_norm_rope_bwd_workspace_bytes(d)), lib)


def _check_pools(k_pool, v_pool, k_scale, v_scale, block_table, cache_seqlens, b, hkv, d):
    """The checks of a paged cache that need the tensors; returns (num_pages, page_size, pages_per_seq, scale_block)."""
    import torch
    dev, shape = k_pool.device, k_pool.shape
    if len(shape) != 4 or shape[2] != hkv or shape[3] != d or v_pool.shape != shape or v_pool.dtype != k_pool.dtype:
        raise AttnError(-2, f"pools {tuple(shape)} / {tuple(v_pool.shape)} must be [num_pages, page_size, {hkv}, {d}]")
    num_pages, page_size = shape[0], shape[1]
    table = block_table.shape
    if len(table) != 2 or table[0] != b or block_table.dtype != torch.int32:
        raise AttnError(-2, "block_table must be int32 [b, pages_per_seq]")
    if cache_seqlens.shape != (b,) or cache_seqlens.dtype != torch.int32:
        raise AttnError(-4, "cache_seqlens must be an int32 tensor of b elements")
    if not k_pool.is_cuda or v_pool.device != dev or block_table.device != dev or cache_seqlens.device != dev or \
            not (k_pool.is_contiguous() and v_pool.is_contiguous() and block_table.is_contiguous() and
                 cache_seqlens.is_contiguous()):
        raise AttnError(-2, "pools, block_table and cache_seqlens must be contiguous CUDA tensors on one device")
    if k_scale is None or v_scale is None:
        if k_scale is not v_scale:
            raise AttnError(-1, "k_scale and v_scale must both be given or both be None")
        return num_pages, page_size, table[1], 0
    if k_pool.dtype != torch.float8_e4m3fn:
        raise AttnError(-4, "a cache with scales must be float8_e4m3fn")
    scales = k_scale.shape
    if len(scales) != 3 or scales[0] != num_pages or scales[1] != hkv or scales[2] < 1 or page_size % scales[2] != 0 or \
            v_scale.shape != scales:
        raise AttnError(-2, "scales must be [num_pages, h_kv, page_size / scale_block]")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or k_scale.device != dev or \
            v_scale.device != dev or not (k_scale.is_contiguous() and v_scale.is_contiguous()):
        raise AttnError(-4, "scales must be contiguous fp32 tensors on the pools' device")
    return num_pages, page_size, table[1], page_size // scales[2]


def attn_kvcache_append_paged(k_new, v_new, k_pool, v_pool, cache_seqlens, block_table, cos=None, sin=None,
                              interleaved: bool = False, k_scale=None, v_scale=None, new_seqlens=None, stream=None):
    """Write new keys, rotated by their positions on the way, and values into
    a paged cache, in place.

    k_new / v_new: [b, h_kv, s_new, d] fp16 or bf16, any strides (multiples of
    8 elements) with contiguous heads; k_pool / v_pool: [num_pages, page_size,
    h_kv, d] of their dtype (the cache of attn_fwd_kvcache_paged), or
    float8_e4m3fn with ``k_scale`` / ``v_scale`` fp32 [num_pages, h_kv,
    page_size / scale_block] (the cache of attn_fwd_kvcache_paged_fp8).  Token
    t of element e goes to position cache_seqlens[e] + t; ``new_seqlens`` int32
    [b] says how many of a padded batch's tokens are there.  ``cos`` / ``sin``
    fp32 [at least the capacity, rot / 2]; None: no rotation.  cache_seqlens is
    not updated."""
    import torch
    lib = load()
    if k_new.dim() != 4 or k_new.shape != v_new.shape:
        raise AttnError(-2, f"k_new{tuple(k_new.shape)} and v_new{tuple(v_new.shape)} must be [b, h_kv, s_new, d]")
    b, hkv, s, d, ks = _as_dense("k_new", k_new)
    vs = _as_dense("v_new", v_new)[4]
    dt, dev = _dtype_code(k_new), k_pool.device
    num_pages, page_size, pps, block = _check_pools(k_pool, v_pool, k_scale, v_scale, block_table, cache_seqlens, b,
                                                    hkv, d)
    if v_new.dtype != k_new.dtype or (block == 0 and k_pool.dtype != k_new.dtype):
        raise AttnError(-4, "k_new, v_new and a cache without scales must have one dtype")
    if k_new.device != dev or v_new.device != dev:
        raise AttnError(-2, "k_new, v_new and the pools must be on one device")
    if new_seqlens is not None and (new_seqlens.shape != (b,) or new_seqlens.dtype != torch.int32 or
                                    new_seqlens.device != dev or not new_seqlens.is_contiguous()):
        raise AttnError(-4, "new_seqlens must be an int32 tensor of b elements on the pools' device")
    c, sn, rot, length = _rotation(cos, sin, dev)
    with _OnDevice(dev):
        rc = lib.attn_kvcache_append_paged(k_new.data_ptr(), v_new.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                           k_scale.data_ptr() if block else None,
                                           v_scale.data_ptr() if block else None, cache_seqlens.data_ptr(),
                                           new_seqlens.data_ptr() if new_seqlens is not None else None,
                                           block_table.data_ptr(), c, sn, ks, vs, b, hkv, s, num_pages, page_size, pps,
                                           block, d, rot, length, 1 if interleaved else 0, dt, _raw_stream(stream, dev))
    if rc < 0:
        _check(rc, lib)


def kvcache_paged_fp8_workspace_bytes(b, h, h_kv, sq, d) -> int:
    lib = load()
    return _check(int(lib.attn_fwd_kvcache_paged_fp8_workspace_bytes(b, h, h_kv, sq, d)), lib)


def attn_fwd_kvcache_paged_fp8(q, k_pool, v_pool, k_scale, v_scale, cache_seqlens, block_table, causal: bool = False,
                               scale: float | None = None, o=None, lse=None, workspace=None, stream=None):
    """Attention of q [b, h, sq, d] (fp16 or bf16) over an e4m3 paged cache:
    k_pool / v_pool float8_e4m3fn [num_pages, page_size, h_kv, d] with k_scale
    / v_scale fp32 [num_pages, h_kv, page_size / scale_block], block_table
    int32 [b, pages_per_seq].  Element e attends to its first cache_seqlens[e]
    tokens (the new ones among them: append first); h / h_kv query heads share
    a key head.  ``workspace``: a CUDA uint8 tensor of
    kvcache_paged_fp8_workspace_bytes bytes.  Returns (o, lse)."""
    import torch
    lib = load()
    if q.dim() != 4 or k_pool.dim() != 4:
        raise AttnError(-2, "q must be [b, h, sq, d] and the pools [num_pages, page_size, h_kv, d]")
    b, h, sq, d = q.shape
    hkv = k_pool.shape[2]
    dt, dev = _dtype_code(q), q.device
    if k_scale is None or v_scale is None:
        raise AttnError(-1, "k_scale and v_scale must be given")
    num_pages, page_size, pps, block = _check_pools(k_pool, v_pool, k_scale, v_scale, block_table, cache_seqlens, b,
                                                    hkv, d)
    if not q.is_contiguous() or dev != k_pool.device:
        raise AttnError(-2, "q must be contiguous, on the pools' device")
    if o is None:
        o = torch.empty_like(q)
    elif o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous() or o.device != dev:
        raise AttnError(-2, "o must be a contiguous tensor shaped and typed like q, on its device")
    if lse is None:
        lse = torch.empty((b, h, sq), dtype=torch.float32, device=dev)
    elif lse.shape != (b, h, sq) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != dev:
        raise AttnError(-2, "lse must be contiguous fp32 [b, h, sq] on q's device")
    if workspace is None:
        workspace = torch.empty(kvcache_paged_fp8_workspace_bytes(b, h, hkv, sq, d), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise AttnError(-2, "workspace must be a contiguous tensor on q's device")
    with _OnDevice(dev):
        rc = lib.attn_fwd_kvcache_paged_fp8(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(),
                                            v_scale.data_ptr(), cache_seqlens.data_ptr(), block_table.data_ptr(),
                                            o.data_ptr(), lse.data_ptr(), b, h, hkv, sq, num_pages, page_size, pps,
                                            block, d, 1 if causal else 0, d ** -0.5 if scale is None else scale, dt,
                                            workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, dev))
    if rc < 0:
        _check(rc, lib)
    _used_on(stream, o, lse, workspace)
    return o, lse
