"""GB300-native ALiBi attention: Python binding of the C ABI (include/alibi.h).

Argument marshalling only: every step of the computation runs in the CUDA
library ``_build/libalibi_gb300.so``. There is no CPU fallback; if the library
is missing or fails to load, every call raises.

The functions carry the names of the C entry points. Tensors are torch CUDA
tensors (torch supplies device memory and streams); ``stream`` defaults to
torch's current stream on the tensors' device.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import numpy as np

from . import _build

__all__ = [
    "AlibiError", "load", "lib_path", "exported_symbols", "alibi_version", "alibi_status_str", "alibi_slopes",
    "alibi_attn_fwd", "alibi_attn_fwd_ex", "alibi_attn_skip_plan", "alibi_attn_fwd_f32", "alibi_attn_decode", "alibi_attn_decode_splits", "alibi_attn_probs_f32",
    "alibi_attn_underflow_bf16", "alibi_check_error", "alibi_attn_decode_noalloc", "alibi_selftest_timeout",
    "alibi_selftest_fwd_timeout", "alibi_decode_underflow_bf16",
    "alibi_slopes_explicit", "alibi_attn_probs_f32_ex", "AlibiFwdOptions", "alibi_attn_bwd", "alibi_attn_bwd_f32",
    "alibi_kv_block_norms", "alibi_attn_decode_skip",
    "alibi_kv4_block_bytes", "alibi_kv4_cache", "alibi_kv4_write", "alibi_kv4_read", "alibi_attn_decode_kv4",
    "AlibiPages", "AlibiRows", "AlibiRotation", "alibi_pages", "alibi_paged_append", "alibi_attn_decode_paged",
    "alibi_attn_fwd_paged", "alibi_selftest_fwd_paged_timeout", "alibi_selftest_decode_paged_timeout",
]

ALIBI_OK, ALIBI_ERR_INVALID, ALIBI_ERR_UNSUPPORTED, ALIBI_ERR_CUDA, ALIBI_ERR_TIMEOUT, ALIBI_ERR_CHECK = 0, -1, -2, -3, -4, -5
ALIBI_ERR_RANGE = -6
ALIBI_FWD_SKIP_UNDERFLOW, ALIBI_FWD_CLAMP, ALIBI_FWD_LOGDIST, ALIBI_FWD_SOFTCAP = 1, 2, 4, 8
ALIBI_FWD_NOMINAL_ORDER = 16

_lock = threading.Lock()
_lib = None


class AlibiFwdOptions(ctypes.Structure):
    """The C struct alibi_fwd_options (include/alibi.h)."""
    _fields_ = [("flags", ctypes.c_uint), ("clamp_min", ctypes.c_float), ("softcap_z", ctypes.c_float),
                ("slopes", ctypes.POINTER(ctypes.c_float))]


class AlibiPages(ctypes.Structure):
    """The C struct alibi_pages (include/alibi.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v")]
                + [(n, ctypes.c_longlong) for n in ("k_page", "k_head", "k_slot", "v_page", "v_head", "v_slot")]
                + [("table", ctypes.c_void_p)] + [(n, ctypes.c_int) for n in ("pages", "heads", "slots", "width", "d")])


class AlibiRows(ctypes.Structure):
    """The C struct alibi_rows (include/alibi.h)."""
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_longlong) for n in ("batch", "head", "token")]


class AlibiRotation(ctypes.Structure):
    """The C struct alibi_rotation (include/alibi.h)."""
    _fields_ = [("dims", ctypes.c_int), ("interleaved", ctypes.c_int), ("base", ctypes.c_double),
                ("freqs", ctypes.POINTER(ctypes.c_double))]


class AlibiError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {alibi_status_str(status)} ({status})")


def checks_build() -> bool:
    """True when ALIBI_CHECKS=1 selects the debug-checks library (every TMA coordinate,
    TMEM address and shared-memory operand tested in the kernels; slower)."""
    return os.environ.get("ALIBI_CHECKS", "0") == "1"


def lib_path() -> str:
    return _build.LIB_CHECKS if checks_build() else _build.LIB


def load(build_if_missing: bool = False):
    """Load the CUDA library (optionally building it first). Raises if it cannot be loaded."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if build_if_missing and not os.path.exists(path):
            _build.build(checks=checks_build())
        if not os.path.exists(path):
            raise RuntimeError(f"ALiBi CUDA library not built ({path}); run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        vp, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.alibi_version.restype = I
        lib.alibi_status_str.argtypes = [I]
        lib.alibi_status_str.restype = ctypes.c_char_p
        lib.alibi_slopes.argtypes = [I, ctypes.POINTER(F)]
        lib.alibi_attn_fwd.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, vp]
        lib.alibi_attn_fwd_f32.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, vp]
        lib.alibi_attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, ctypes.POINTER(AlibiFwdOptions), vp]
        lib.alibi_slopes_explicit.argtypes = [I, ctypes.c_double, ctypes.c_double, ctypes.c_double, I,
                                              ctypes.POINTER(F)]
        lib.alibi_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I,
                                        ctypes.POINTER(AlibiFwdOptions), vp]
        lib.alibi_attn_bwd_f32.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I, vp]
        lib.alibi_kv_block_norms.argtypes = [vp, vp, I, I, I, I, I, vp]
        lib.alibi_attn_decode_skip.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, vp]
        lib.alibi_attn_probs_f32_ex.argtypes = [vp, vp, vp, vp, I, I, I, I, I, vp]
        lib.alibi_attn_fwd_ex.restype = I
        lib.alibi_attn_skip_plan.argtypes = [vp, vp, I, I, I, I, ctypes.POINTER(F), vp, vp]
        lib.alibi_attn_skip_plan.restype = I
        lib.alibi_attn_decode.argtypes = [vp, vp, vp, vp, I, I, I, I, vp]
        lib.alibi_attn_probs_f32.argtypes = [vp, vp, vp, vp, I, I, I, I, vp]
        lib.alibi_attn_decode_splits.argtypes = [I, I, I, I]
        lib.alibi_attn_decode_noalloc.argtypes = [vp, vp, vp, vp, I, I, I, I, vp]
        lib.alibi_attn_decode_noalloc.restype = I
        lib.alibi_attn_underflow_bf16.argtypes = [vp, vp, I, I, I, I, F, vp, vp]
        lib.alibi_check_error.argtypes = [vp]
        lib.alibi_selftest_timeout.argtypes = [vp]
        lib.alibi_selftest_timeout.restype = I
        lib.alibi_selftest_fwd_timeout.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, vp]
        lib.alibi_selftest_fwd_timeout.restype = I
        lib.alibi_decode_underflow_bf16.argtypes = [vp, vp, I, I, I, I, F, vp, vp]
        lib.alibi_decode_underflow_bf16.restype = I
        lib.alibi_kv4_block_bytes.argtypes = [I]
        lib.alibi_kv4_block_bytes.restype = I
        lib.alibi_kv4_write.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, vp]
        lib.alibi_kv4_write.restype = I
        lib.alibi_kv4_read.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, I, vp]
        lib.alibi_kv4_read.restype = I
        lib.alibi_attn_decode_kv4.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, I, I, I, ctypes.POINTER(F), vp]
        lib.alibi_attn_decode_kv4.restype = I
        pages, rows = ctypes.POINTER(AlibiPages), ctypes.POINTER(AlibiRows)
        lib.alibi_paged_append.argtypes = [rows, rows, pages, vp, vp, I, I, ctypes.POINTER(AlibiRotation), rows, vp, I, vp]
        lib.alibi_paged_append.restype = I
        lib.alibi_attn_decode_paged.argtypes = [vp, pages, vp, vp, vp, I, I, I, I, ctypes.POINTER(F), vp]
        lib.alibi_attn_decode_paged.restype = I
        lib.alibi_attn_fwd_paged.argtypes = [vp, pages, vp, vp, vp, vp, I, I, I, I, ctypes.POINTER(F), vp]
        lib.alibi_attn_fwd_paged.restype = I
        lib.alibi_selftest_fwd_paged_timeout.argtypes = [vp, pages, vp, vp, vp, vp, I, I, I, I, I, I, vp]
        lib.alibi_selftest_fwd_paged_timeout.restype = I
        lib.alibi_selftest_decode_paged_timeout.argtypes = [vp, pages, vp, vp, vp, I, I, I, I, I, vp]
        lib.alibi_selftest_decode_paged_timeout.restype = I
        for name in ("alibi_attn_fwd", "alibi_attn_fwd_f32", "alibi_attn_decode", "alibi_attn_decode_splits",
                     "alibi_attn_probs_f32",
                     "alibi_attn_underflow_bf16", "alibi_check_error", "alibi_slopes"):
            getattr(lib, name).restype = I
        _lib = lib
        return lib


def exported_symbols(names) -> dict:
    """Which of ``names`` the loaded library exports (no device work)."""
    lib = load()
    return {n: hasattr(lib, n) for n in names}


def _check(status: int, where: str):
    if status != ALIBI_OK:
        raise AlibiError(status, where)


def _stream(stream, device):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, dtype, shape, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# --------------------------------------------------------------------- entry points

def alibi_version() -> int:
    return load().alibi_version()


def alibi_status_str(status: int) -> str:
    try:
        return load().alibi_status_str(int(status)).decode()
    except Exception:  # library unavailable while formatting an error
        return f"status {status}"


def alibi_slopes(H: int) -> np.ndarray:
    """fp32 ALiBi slopes for H heads (host computation in the library)."""
    out = np.empty(H, dtype=np.float32)
    _check(load().alibi_slopes(int(H), out.ctypes.data_as(ctypes.POINTER(ctypes.c_float))), "alibi_slopes")
    return out


def alibi_attn_fwd(q, k, v, out=None, lse=None, causal: bool = True, stream=None, want_lse: bool = True,
                   skip_underflow: bool = False):
    """bf16 prefill on the tensor cores (causal, or symmetric bias over all keys).
    q, k, v: [B, H, N, d] bf16 CUDA tensors.

    ``skip_underflow`` leaves out KV tiles whose weights provably flush to zero
    (alibi_attn_fwd_ex with ALIBI_FWD_SKIP_UNDERFLOW); the result is bit-identical.
    """
    import torch
    _need(q, torch.bfloat16, None, "q")
    B, H, N, d = q.shape
    _need(k, torch.bfloat16, q.shape, "k")
    _need(v, torch.bfloat16, q.shape, "v")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.bfloat16, q.shape, "out")
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, torch.float32, (B, H, N), "lse")
    if skip_underflow:
        opt = AlibiFwdOptions(ALIBI_FWD_SKIP_UNDERFLOW, 0.0, 0.0, None)
        _check(load().alibi_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d,
                                        int(bool(causal)), ctypes.byref(opt), _stream(stream, q.device)),
               "alibi_attn_fwd_ex")
    else:
        _check(load().alibi_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d,
                                     int(bool(causal)), _stream(stream, q.device)), "alibi_attn_fwd")
    return out, lse


def alibi_attn_fwd_ex(q, k, v, out=None, lse=None, causal: bool = True, flags: int = 0, clamp_min: float = -87.0,
                      softcap_z: float = 50.0, slopes=None, stream=None):
    """Prefill with options (ALIBI_FWD_* flags): exact underflow skipping, or the
    clamp / log-distance / soft-cap mitigations with their parameters, and
    optionally caller-chosen per-head slopes (H values, natural-log units)."""
    import torch
    _need(q, torch.bfloat16, None, "q")
    B, H, N, d = q.shape
    _need(k, torch.bfloat16, q.shape, "k")
    _need(v, torch.bfloat16, q.shape, "v")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _need(out, torch.bfloat16, q.shape, "out")
    _need(lse, torch.float32, (B, H, N), "lse")
    m = None
    if slopes is not None:
        m = np.ascontiguousarray(slopes, dtype=np.float32)
        if m.shape != (H,):
            raise ValueError(f"slopes: expected shape ({H},), got {m.shape}")
    opt = AlibiFwdOptions(int(flags), float(clamp_min), float(softcap_z),
                          None if m is None else m.ctypes.data_as(ctypes.POINTER(ctypes.c_float)))
    _check(load().alibi_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d, int(bool(causal)),
                                    ctypes.byref(opt), _stream(stream, q.device)),
           "alibi_attn_fwd_ex")
    return out, lse


def alibi_slopes_explicit(H: int, delta_first: float, delta_last: float, tau: float | None = None,
                          log_distance: bool = False) -> np.ndarray:
    """fp32 slopes whose zero-logit blindness distances run geometrically from
    delta_first (head 0) to delta_last (head H-1); tau defaults to ln 2^-126."""
    tau = -126.0 * math.log(2.0) if tau is None else tau
    out = np.empty(H, dtype=np.float32)
    _check(load().alibi_slopes_explicit(int(H), float(delta_first), float(delta_last), float(tau),
                                        int(bool(log_distance)), out.ctypes.data_as(ctypes.POINTER(ctypes.c_float))),
           "alibi_slopes_explicit")
    return out


def alibi_attn_bwd(q, k, v, out, lse, dout, dq=None, dk=None, dv=None, causal: bool = True, slopes=None,
                   flags: int = 0, clamp_min: float = -87.0, softcap_z: float = 50.0, stream=None):
    """bf16 backward on the tensor cores: (dq, dk, dv) of sum(dout * out) for the
    forward's out and lse. All tensors [B, H, N, d] bf16 CUDA tensors, lse fp32.
    flags / clamp_min / softcap_z / slopes must be those the forward ran with."""
    import torch
    _need(q, torch.bfloat16, None, "q")
    B, H, N, d = q.shape
    for t, name in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, torch.bfloat16, q.shape, name)
    _need(lse, torch.float32, (B, H, N), "lse")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for t, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, torch.bfloat16, q.shape, name)
    m = None
    if slopes is not None:
        m = np.ascontiguousarray(slopes, dtype=np.float32)
        if m.shape != (H,):
            raise ValueError(f"slopes: expected shape ({H},), got {m.shape}")
    opt = AlibiFwdOptions(int(flags), float(clamp_min), float(softcap_z),
                          None if m is None else m.ctypes.data_as(ctypes.POINTER(ctypes.c_float)))
    _check(load().alibi_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                 _ptr(dv), B, H, N, d, int(bool(causal)), ctypes.byref(opt),
                                 _stream(stream, q.device)), "alibi_attn_bwd")
    return dq, dk, dv


def alibi_attn_bwd_f32(q, k, v, out, lse, dout, causal: bool = True, stream=None):
    """fp32 backward (reference precision). All tensors fp32 CUDA tensors."""
    import torch
    _need(q, torch.float32, None, "q")
    B, H, N, d = q.shape
    for t, name in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, torch.float32, q.shape, name)
    _need(lse, torch.float32, (B, H, N), "lse")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    _check(load().alibi_attn_bwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                                     _ptr(dk), _ptr(dv), B, H, N, d, int(bool(causal)), _stream(stream, q.device)),
           "alibi_attn_bwd_f32")
    return dq, dk, dv


def alibi_attn_skip_plan(q, k, first_tile=None, slopes=None, stream=None):
    """Per work item (b*H + h, 256-row block): the first 128-key tile the skipping
    prefill computes. Returns an int32 CUDA tensor [B*H*ceil(N/256)]."""
    import torch
    _need(q, torch.bfloat16, None, "q")
    B, H, N, d = q.shape
    _need(k, torch.bfloat16, q.shape, "k")
    items = B * H * ((N + 255) // 256)
    if first_tile is None:
        first_tile = torch.empty(items, dtype=torch.int32, device=q.device)
    _need(first_tile, torch.int32, (items,), "first_tile")
    m = None if slopes is None else np.ascontiguousarray(slopes, dtype=np.float32)
    if m is not None and m.shape != (H,):
        raise ValueError(f"slopes: expected shape ({H},), got {m.shape}")
    _check(load().alibi_attn_skip_plan(_ptr(q), _ptr(k), B, H, N, d,
                                       None if m is None else m.ctypes.data_as(ctypes.POINTER(ctypes.c_float)),
                                       _ptr(first_tile), _stream(stream, q.device)),
           "alibi_attn_skip_plan")
    return first_tile


def alibi_attn_fwd_f32(q, k, v, out=None, lse=None, causal: bool = True, stream=None):
    """fp32 prefill (reference precision), causal or symmetric. q, k, v: [B, H, N, d] fp32 CUDA tensors."""
    import torch
    _need(q, torch.float32, None, "q")
    B, H, N, d = q.shape
    _need(k, torch.float32, q.shape, "k")
    _need(v, torch.float32, q.shape, "v")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.float32, q.shape, "out")
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _need(lse, torch.float32, (B, H, N), "lse")
    _check(load().alibi_attn_fwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d,
                                     int(bool(causal)), _stream(stream, q.device)), "alibi_attn_fwd_f32")
    return out, lse


def alibi_attn_decode(q, kcache, vcache, out=None, stream=None):
    """bf16 decode: q [B, H, d] at position L-1 against caches [B, H, L, d]."""
    import torch
    _need(kcache, torch.bfloat16, None, "kcache")
    B, H, L, d = kcache.shape
    _need(vcache, torch.bfloat16, kcache.shape, "vcache")
    _need(q, torch.bfloat16, (B, H, d), "q")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.bfloat16, (B, H, d), "out")
    _check(load().alibi_attn_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(out), B, H, L, d,
                                    _stream(stream, q.device)), "alibi_attn_decode")
    return out


def alibi_kv_block_norms(kcache, knorm=None, blk_begin: int = 0, stream=None):
    """Maximum key norm per 64-key block of a bf16 cache [B, H, L, d] -> fp32 [B, H, ceil(L/64)].
    Only blocks >= blk_begin are recomputed (refresh the tail after appending keys)."""
    import torch
    _need(kcache, torch.bfloat16, None, "kcache")
    B, H, L, d = kcache.shape
    nblk = (L + 63) // 64
    if knorm is None:
        knorm = torch.empty((B, H, nblk), dtype=torch.float32, device=kcache.device)
    _need(knorm, torch.float32, (B, H, nblk), "knorm")
    _check(load().alibi_kv_block_norms(_ptr(kcache), _ptr(knorm), B, H, L, d, int(blk_begin),
                                       _stream(stream, kcache.device)), "alibi_kv_block_norms")
    return knorm


def alibi_attn_decode_skip(q, kcache, vcache, knorm, out=None, stream=None):
    """Decode that skips cache rows whose weights are provably below 2^-127 of the
    largest (needs the cache's block norms from alibi_kv_block_norms)."""
    import torch
    _need(kcache, torch.bfloat16, None, "kcache")
    B, H, L, d = kcache.shape
    _need(vcache, torch.bfloat16, kcache.shape, "vcache")
    _need(q, torch.bfloat16, (B, H, d), "q")
    _need(knorm, torch.float32, (B, H, (L + 63) // 64), "knorm")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.bfloat16, (B, H, d), "out")
    _check(load().alibi_attn_decode_skip(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(knorm), _ptr(out), B, H, L, d,
                                         _stream(stream, q.device)), "alibi_attn_decode_skip")
    return out


def alibi_attn_decode_noalloc(q, kcache, vcache, out, stream=None):
    """Decode without any device allocation (for callers that cannot allocate).

    Same result as alibi_attn_decode, but the split-K partials live in a fixed
    4 MiB buffer inside the library, so ``out`` must be supplied by the caller.
    Calls that overlap on the GPU share that buffer and race: order them.
    """
    import torch
    _need(kcache, torch.bfloat16, None, "kcache")
    B, H, L, d = kcache.shape
    _need(vcache, torch.bfloat16, kcache.shape, "vcache")
    _need(q, torch.bfloat16, (B, H, d), "q")
    _need(out, torch.bfloat16, (B, H, d), "out")
    _check(load().alibi_attn_decode_noalloc(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(out), B, H, L, d,
                                            _stream(stream, q.device)), "alibi_attn_decode_noalloc")
    return out


def alibi_kv4_block_bytes(d: int) -> int:
    """Bytes of one 32-token block of the 4-bit KV cache for head size d."""
    n = load().alibi_kv4_block_bytes(max(-1, min(int(d), 1 << 30)))
    if n < 0:
        raise AlibiError(n, "alibi_kv4_block_bytes")
    return n


def alibi_kv4_cache(B: int, H: int, C: int, d: int, device=None):
    """An empty 4-bit KV cache for B sequences of up to C tokens (a multiple of 32) and H KV heads of
    size d: uint8 [B, H, C / 32, alibi_kv4_block_bytes(d)], uninitialised (rows are used once written)."""
    import torch
    if C < 1 or C % 32 != 0:
        raise ValueError(f"C must be a positive multiple of 32, got {C}")
    return torch.empty((B, H, C // 32, alibi_kv4_block_bytes(d)), dtype=torch.uint8,
                       device="cuda" if device is None else device)


# The 4-bit cache's calls are made once per layer and token, so they check their arguments in one expression and leave it to
# _explain_kv4 to say what is wrong, and look up what they use of torch once (host time of a write
# 6.0 -> 5.5 us, of a decode into given outputs 7.3 -> 6.7).
_names = None


def _current_stream_handle(index: int) -> int:
    import torch
    return torch.cuda.current_stream(index).cuda_stream


def _kv4_names():
    """(bfloat16, uint8, int32, float32, handle of a device's current stream, current device, the library)"""
    global _names
    if _names is None:
        import torch
        # torch's own shortcuts, where it has them, take 0.06 and 0.1 us; its documented calls, 1.1 and 0.2 us, do the same
        raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _current_stream_handle
        current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _names = (torch.bfloat16, torch.uint8, torch.int32, torch.float32, raw_stream, current, load())
    return _names


def _need_on(t, dtype, shape, name, index):
    """_need, and on CUDA device `index`."""
    _need(t, dtype, shape, name)
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _explain_kv4(dtype, first, others, cache, H, ints):
    """Raise what is wrong with a call on the 4-bit cache. first: (tensor, name, dimensions); others: (tensor, name, dtype,
    shape) like it; ints: (tensor or None, name) of int32 [B]."""
    import torch
    t, name, dims = first
    _need(t, dtype, None, name)
    if t.dim() not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions, got shape {tuple(t.shape)}")
    B, d, index = t.shape[0], t.shape[-1], t.get_device()
    for o, oname, odtype, shape in others:
        _need_on(o, odtype, shape, oname, index)
    _need_on(cache, torch.uint8, None, "cache", index)
    s = tuple(cache.shape)
    if len(s) != 4 or s[0] != B or s[3] != 36 * max(d, 32) or H not in (None, s[1]):
        raise ValueError(f"cache must have shape ({B}, {'heads' if H is None else H}, C / 32, {36 * max(d, 32)}), got {s}")
    for o, oname in ints:
        if o is not None:
            _need_on(o, torch.int32, (B,), oname, index)


def _empty_on(stream, index, shape, dtype):
    """An uninitialised tensor whose memory belongs to the stream that will write it: memory of another stream may still
    be in use there."""
    import torch
    device, raw_stream = torch.device("cuda", index), _kv4_names()[4]
    if not isinstance(stream, int):
        stream = stream.cuda_stream
    if stream == raw_stream(index):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _call_kv4(index, fn, where, stream, *args):
    """fn(*args, stream) with the tensors' device current, on `stream` (None: torch's current one)."""
    _, _, _, _, raw_stream, current, _ = _kv4_names()
    if stream is None:
        stream = raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if current() == index:
        status = fn(*args, stream)
    else:
        import torch
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != ALIBI_OK:
        raise AlibiError(status, where)


def _kv4_sizes(n, C, where):
    """What the library refuses of n tokens and a capacity of C, here, where a number beyond 32 bits is still itself."""
    if not 0 < n <= C:
        raise AlibiError(ALIBI_ERR_INVALID, where)
    if C > 1 << 24:
        raise AlibiError(ALIBI_ERR_UNSUPPORTED, where)


def _kv4_rows_ok(k, v, dtype, cache, pos, count) -> bool:
    _, uint8, int32, _, _, _, _ = _kv4_names()
    try:
        shape, c, index = k.shape, cache.shape, k.get_device()
        B, H, _, d = shape
        return (k.dtype is dtype and v.dtype is dtype and cache.dtype is uint8
                and index == v.get_device() == cache.get_device() >= 0 and v.shape == shape
                and len(c) == 4 and c[0] == B and c[1] == H and c[3] == (36 * d if d > 32 else 1152)
                and k.is_contiguous() and v.is_contiguous() and cache.is_contiguous()
                and (pos is None or (pos.dtype is int32 and pos.shape == (B,) and pos.get_device() == index
                                     and pos.is_contiguous()))
                and (count is None or (count.dtype is int32 and count.shape == (B,)
                                       and count.get_device() == index and count.is_contiguous())))
    except (AttributeError, TypeError, ValueError):
        return False


def alibi_kv4_write(k, v, cache, pos=None, count=None, stream=None) -> None:
    """Quantise new keys and values [B, H, T, d] (bf16) and write them into the 4-bit cache
    (alibi_kv4_cache): token t < count[b] of sequence b to row pos[b] + t. pos and count are int32
    CUDA tensors [B] (None: 0 and T). Sequences that do not fit are left out and reported by
    alibi_check_error."""
    bfloat16, _, _, _, _, _, lib = _kv4_names()
    if not _kv4_rows_ok(k, v, bfloat16, cache, pos, count):
        _explain_kv4(bfloat16, (k, "k", (4,)), [(v, "v", bfloat16, getattr(k, "shape", None))], cache,
                     k.shape[1] if hasattr(k, "shape") and len(k.shape) == 4 else None, [(pos, "pos"), (count, "count")])
    B, H, T, d = k.shape
    C = cache.shape[2] * 32
    if not 0 < T <= C <= 1 << 24:
        _kv4_sizes(T, C, "alibi_kv4_write")
    _call_kv4(k.get_device(), lib.alibi_kv4_write, "alibi_kv4_write", stream, k.data_ptr(), v.data_ptr(),
              cache.data_ptr(), None if pos is None else pos.data_ptr(), None if count is None else count.data_ptr(),
              B, H, T, C, d)


def alibi_kv4_read(cache, k, v, pos=None, count=None, stream=None):
    """Read rows of the 4-bit cache back into k and v [B, H, T, d] (both bf16, or both fp32 for the
    held values exactly): row pos[b] + t of sequence b to token t < count[b]; other tokens of k and v
    are left as they were. pos and count as in alibi_kv4_write. Returns (k, v)."""
    bfloat16, _, _, float32, _, _, lib = _kv4_names()
    dtype = float32 if getattr(k, "dtype", None) is float32 else bfloat16
    if not _kv4_rows_ok(k, v, dtype, cache, pos, count):
        _explain_kv4(dtype, (k, "k", (4,)), [(v, "v", dtype, getattr(k, "shape", None))], cache,
                     k.shape[1] if hasattr(k, "shape") and len(k.shape) == 4 else None, [(pos, "pos"), (count, "count")])
    B, H, T, d = k.shape
    C = cache.shape[2] * 32
    if not 0 < T <= C <= 1 << 24:
        _kv4_sizes(T, C, "alibi_kv4_read")
    _call_kv4(k.get_device(), lib.alibi_kv4_read, "alibi_kv4_read", stream, cache.data_ptr(), k.data_ptr(),
              v.data_ptr(), None if pos is None else pos.data_ptr(), None if count is None else count.data_ptr(),
              B, H, T, C, d, int(dtype is float32))
    return k, v


def alibi_attn_decode_kv4(q, cache, lens=None, L=None, out=None, lse=None, slopes=None, stream=None):
    """ALiBi attention of the newest T tokens of each sequence over the 4-bit cache that holds them.
    q: bf16 [B, H, T, d], or [B, H, d] for one token; cache: uint8 [B, H_kv, C / 32, bytes], H a multiple
    of H_kv and at most 384; lens: int32 CUDA tensor [B] of lengths (None: all L); L: a bound on them (None: the
    capacity C); slopes: H values (None: alibi_slopes(H)). Returns (out, lse): bf16 like q, fp32
    without the last dimension; those made here belong to `stream`."""
    bfloat16, uint8, int32, float32, raw_stream, current, lib = _kv4_names()
    try:
        shape, c, index = q.shape, cache.shape, q.get_device()
        dims, B, H, d = len(shape), shape[0], shape[1], shape[-1]
        good = (3 <= dims <= 4 and q.dtype is bfloat16 and cache.dtype is uint8
                and index == cache.get_device() >= 0 and len(c) == 4 and c[0] == B and c[3] == (36 * d if d > 32 else 1152)
                and q.is_contiguous() and cache.is_contiguous()
                and (lens is None or (lens.dtype is int32 and lens.shape == (B,) and lens.get_device() == index
                                      and lens.is_contiguous()))
                and (out is None or (out.dtype is bfloat16 and out.shape == shape and out.get_device() == index
                                     and out.is_contiguous()))
                and (lse is None or (lse.dtype is float32 and lse.shape == shape[:-1] and lse.get_device() == index
                                     and lse.is_contiguous())))
    except (AttributeError, IndexError, TypeError, ValueError):
        good = False
    import torch
    if not good:
        given = [(out, "out", bfloat16, getattr(q, "shape", None))] if out is not None else []
        given += [(lse, "lse", float32, getattr(q, "shape", (0,))[:-1])] if lse is not None else []
        _explain_kv4(bfloat16, (q, "q", (3, 4)), given, cache, None, [(lens, "lens")])
    if out is None:
        out = (torch.empty(shape, dtype=bfloat16, device=q.device) if stream is None
               else _empty_on(stream, index, shape, bfloat16))
    if lse is None:
        lse = (torch.empty(shape[:-1], dtype=float32, device=q.device) if stream is None
               else _empty_on(stream, index, shape[:-1], float32))
    m = None
    if slopes is not None:
        m = np.ascontiguousarray(slopes, dtype=np.float32)
        if m.shape != (H,):
            raise ValueError(f"slopes: expected shape ({H},), got {m.shape}")
    C = c[2] * 32
    L = C if L is None else int(L)
    if not 0 < L <= C <= 1 << 24:
        _kv4_sizes(L, C, "alibi_attn_decode_kv4")
    args = (q.data_ptr(), cache.data_ptr(), None if lens is None else lens.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H,
            c[1], shape[2] if dims == 4 else 1, L, C, d,
            None if m is None else m.ctypes.data_as(ctypes.POINTER(ctypes.c_float)))
    if stream is None and current() == index:  # as _call_kv4 does it, without its 0.6 us
        status = lib.alibi_attn_decode_kv4(*args, raw_stream(index))
        if status != ALIBI_OK:
            raise AlibiError(status, "alibi_attn_decode_kv4")
    else:
        _call_kv4(index, lib.alibi_attn_decode_kv4, "alibi_attn_decode_kv4", stream, *args)
    return out, lse


def alibi_pages(P: int, H: int, S: int, d: int, device=None):
    """Pools for a paged KV cache of P pages of S tokens (a power of two in [8, 1024]) and H KV heads of size d: k_pages
    and v_pages, bf16 [P, H, S, d], uninitialised (rows are used once written). The paged calls take any tensors of that
    shape whose last dimension is contiguous and whose other strides are multiples of 8."""
    import torch
    device = "cuda" if device is None else device
    return tuple(torch.empty((P, H, S, d), dtype=torch.bfloat16, device=device) for _ in range(2))


def _row_strides(shape, stride, name):
    """Strides of all dimensions but the last; of one that has a single index any will do, and it gets that of a dense row."""
    if stride[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return [s if n > 1 else -(-shape[-1] // 8) * 8 for n, s in zip(shape[:-1], stride)]


def _strided(t, dtype, dims, name, index=None):
    """_need without contiguity: a CUDA tensor of `dims` dimensions, on device `index` where one is given."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _paged_ints(t, B, index, name):
    """The address of int32 [B], or None."""
    if t is None:
        return None
    try:
        good = t.dtype is _kv4_names()[2] and t.shape == (B,) and t.get_device() == index and t.is_contiguous()
    except AttributeError:
        good = False
    if not good:
        _need_on(t, _kv4_names()[2], (B,), name, index)
    return t.data_ptr()


_pack_pages = struct.Struct("=QQqqqqqqQiiiii").pack_into


def _paged_cache(k_pages, v_pages, table, B, d, index):
    """The C struct of a paged cache, its tensors checked; its heads, and the tokens that the table has room for."""
    bfloat16, _, int32, _, _, _, _ = _kv4_names()
    try:
        shape, M = k_pages.shape, table.shape
        P, H, S, dk = shape
        good = (k_pages.dtype is bfloat16 and v_pages.dtype is bfloat16 and table.dtype is int32 and v_pages.shape == shape
                and dk == d and len(M) == 2 and M[0] == B and index == k_pages.get_device() == v_pages.get_device()
                == table.get_device() >= 0 and table.is_contiguous() and P < 1 << 31 and H < 1 << 31 and S < 1 << 31 and M[1] < 1 << 31)
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _explain_paged(k_pages, v_pages, table, B, d, index)
    if k_pages.is_contiguous():
        kp, kh, ks = H * S * d, S * d, d
    else:
        kp, kh, ks = _row_strides(shape, k_pages.stride(), "k_pages")
    if v_pages.is_contiguous():
        vp, vh, vs = H * S * d, S * d, d
    else:
        vp, vh, vs = _row_strides(shape, v_pages.stride(), "v_pages")
    pages = AlibiPages()
    try:  # field by field this would take 1.2 us more
        _pack_pages(pages, 0, k_pages.data_ptr(), v_pages.data_ptr(), kp, kh, ks, vp, vh, vs, table.data_ptr(), P, H, S, M[1], d)
    except struct.error:  # d beyond 32 bits
        raise AlibiError(ALIBI_ERR_UNSUPPORTED, "paged cache") from None
    return pages, H, M[1] * S


def _explain_paged(k_pages, v_pages, table, B, d, index):
    """Raise what is wrong with a paged cache."""
    bfloat16, _, int32, _, _, _, _ = _kv4_names()
    _strided(k_pages, bfloat16, 4, "k_pages", index)
    _strided(v_pages, bfloat16, 4, "v_pages", index)
    shape = k_pages.shape
    if v_pages.shape != shape or shape[3] != d:
        raise ValueError(f"k_pages and v_pages must have one shape (pages, heads, slots, {d}), got {tuple(shape)} and "
                         f"{tuple(v_pages.shape)}")
    _need_on(table, int32, None, "table", index)
    if table.dim() != 2 or table.shape[0] != B:
        raise ValueError(f"table must have shape ({B}, pages of a sequence), got {tuple(table.shape)}")
    raise AlibiError(ALIBI_ERR_UNSUPPORTED, "paged cache")


_pack_rows = struct.Struct("=Qqqq").pack_into


def _rows_struct(t, shape, name):
    """The C struct of rows [B, H, T, d]."""
    rows = AlibiRows()
    if t.is_contiguous():
        n = shape[2] * shape[3]
        _pack_rows(rows, 0, t.data_ptr(), shape[1] * n, n, shape[3])
    else:
        _pack_rows(rows, 0, t.data_ptr(), *_row_strides(shape, t.stride(), name))
    return rows


def _is_rows(t, dtype, shape, index) -> bool:
    try:
        return t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0
    except AttributeError:
        return False


def alibi_paged_append(k, v, k_pages, v_pages, table, pos=None, count=None, rotate: int = 0, base: float = 10000.0, freqs=None,
                       interleaved: bool = False, q=None, q_out=None, stream=None):
    """Append new keys and values [B, H_kv, T, d] (bf16, any strides that are multiples of 8) to the pages of a pool: token
    t < count[b] of sequence b to row pos[b] + t, which is slot j % S of page table[b, j // S]. k_pages, v_pages: [P, H_kv, S, d]
    (alibi_pages); table: int32 [B, pages of a sequence]; pos and count: int32 CUDA tensors [B] (None: 0 and T).
    rotate > 0 turns the first `rotate` elements (a multiple of 16) of the keys by their positions, and those of
    the queries q [B, H, T, d] into q_out, which is returned; frequencies base^(-2 i / rotate), or freqs (rotate / 2 numbers,
    radians per token); pairs of elements i and i + rotate / 2, or 2 i and 2 i + 1 (interleaved). Sequences that do not fit
    and tokens without a page are left out and reported by alibi_check_error."""
    bfloat16, _, _, _, _, _, lib = _kv4_names()
    try:
        shape, index = k.shape, k.get_device()
        B, H, T, d = shape
        good = k.dtype is bfloat16 and _is_rows(v, bfloat16, shape, index)
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _strided(k, bfloat16, 4, "k")
        _strided(v, bfloat16, 4, "v", k.get_device())
        raise ValueError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
    pages, heads, _ = _paged_cache(k_pages, v_pages, table, B, d, index)
    if heads != H:
        raise ValueError(f"k_pages must have {H} heads, got {heads}")
    if B >= 1 << 31 or T >= 1 << 31:
        raise AlibiError(ALIBI_ERR_INVALID, "alibi_paged_append")
    rotation = f = None
    if rotate:
        if not 0 < rotate <= d or rotate % 16:
            raise ValueError(f"rotate must be a multiple of 16 and at most {d}, got {rotate}")
        if freqs is not None:
            f = np.ascontiguousarray(freqs, dtype=np.float64)
            if f.shape != (rotate // 2,):
                raise ValueError(f"freqs: expected shape ({rotate // 2},), got {f.shape}")
            f = f.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
        rotation = AlibiRotation(rotate, int(bool(interleaved)), base, f)
    rows = None
    if q is None:
        if q_out is not None:
            raise ValueError("q_out needs q")
    else:
        if not rotate:
            raise ValueError("q needs rotate")
        try:
            qs = q.shape
            good = _is_rows(q, bfloat16, (B, qs[1], T, d), index)
        except (AttributeError, IndexError):
            good = False
        if not good:
            _strided(q, bfloat16, 4, "q", index)
            raise ValueError(f"q must have shape ({B}, heads, {T}, {d}), got {tuple(q.shape)}")
        rows = _rows_struct(q, qs, "q")
        if q_out is None:
            import torch
            q_out = (torch.empty(qs, dtype=bfloat16, device=q.device) if stream is None
                     else _empty_on(stream, index, qs, bfloat16))
        elif not (_is_rows(q_out, bfloat16, qs, index) and q_out.is_contiguous()):
            _need_on(q_out, bfloat16, qs, "q_out", index)
    _call_kv4(index, lib.alibi_paged_append, "alibi_paged_append", stream, _rows_struct(k, shape, "k"), _rows_struct(v, shape, "v"),
              pages, _paged_ints(pos, B, index, "pos"), _paged_ints(count, B, index, "count"), B, T, rotation, rows,
              None if q is None else q_out.data_ptr(), 0 if q is None else q.shape[1])
    return q_out


def _slope_array(slopes, H):
    """A ctypes pointer to H slopes; it keeps the array."""
    m = np.ascontiguousarray(slopes, dtype=np.float32)
    if m.shape != (H,):
        raise ValueError(f"slopes: expected shape ({H},), got {m.shape}")
    return m.ctypes.data_as(ctypes.POINTER(ctypes.c_float))


def _paged_bound(L, C, where):
    """The bound on the lengths: L, or C, what the table has room for."""
    L = C if L is None else int(L)
    if not 0 < L <= C <= 1 << 24:
        raise AlibiError(ALIBI_ERR_UNSUPPORTED if 0 < L <= C else ALIBI_ERR_INVALID, where)
    return L


def _paged_query(q, dims):
    """Shape and device index of queries of so many dimensions."""
    bfloat16 = _kv4_names()[0]
    try:
        shape, index = q.shape, q.get_device()
        good = q.dtype is bfloat16 and len(shape) in dims and index >= 0 and q.is_contiguous()
    except (AttributeError, TypeError):
        good = False
    if not good:
        _need(q, bfloat16, None, "q")
        raise ValueError(f"q must have {' or '.join(map(str, dims))} dimensions, got shape {tuple(q.shape)}")
    return shape, index


def _paged_outputs(out, lse, q, shape, index, stream):
    """out and lse of the queries q, made where they are not given."""
    import torch
    bfloat16, _, _, float32, _, _, _ = _kv4_names()
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty_on(stream, index, shape, bfloat16)
    elif not (_is_rows(out, bfloat16, shape, index) and out.is_contiguous()):
        _need_on(out, bfloat16, shape, "out", index)
    if lse is None:
        lse = (torch.empty(shape[:-1], dtype=float32, device=q.device) if stream is None
               else _empty_on(stream, index, shape[:-1], float32))
    elif not (_is_rows(lse, float32, shape[:-1], index) and lse.is_contiguous()):
        _need_on(lse, float32, shape[:-1], "lse", index)
    return out, lse


def alibi_attn_decode_paged(q, k_pages, v_pages, table, lens=None, L=None, out=None, lse=None, slopes=None, stream=None):
    """ALiBi attention of the newest T tokens (at most 16) of each sequence over the pages that hold them. q: bf16 [B, H, T, d],
    or [B, H, d] for one token; k_pages, v_pages: [P, H_kv, S, d], H a multiple of H_kv and at most 384; table: int32 [B, pages of
    a sequence]; lens: int32 CUDA tensor [B] of lengths (None: all L); L: a bound on them (None: what the table has
    room for); slopes: H values (None: alibi_slopes(H)). Returns (out, lse): bf16 like q, fp32 without the last
    dimension; those made here belong to `stream`."""
    _, _, _, _, raw_stream, current, lib = _kv4_names()
    shape, index = _paged_query(q, (3, 4))
    B, H, d = shape[0], shape[1], shape[-1]
    pages, _, C = _paged_cache(k_pages, v_pages, table, B, d, index)
    L = _paged_bound(L, C, "alibi_attn_decode_paged")
    out, lse = _paged_outputs(out, lse, q, shape, index, stream)
    args = (q.data_ptr(), pages, _paged_ints(lens, B, index, "lens"), out.data_ptr(), lse.data_ptr(), B, H,
            shape[2] if len(shape) == 4 else 1, L, None if slopes is None else _slope_array(slopes, H))
    if stream is None and current() == index:  # as _call_kv4 does it, without its 0.6 us
        status = lib.alibi_attn_decode_paged(*args, raw_stream(index))
        if status != ALIBI_OK:
            raise AlibiError(status, "alibi_attn_decode_paged")
    else:
        _call_kv4(index, lib.alibi_attn_decode_paged, "alibi_attn_decode_paged", stream, *args)
    return out, lse


def alibi_attn_fwd_paged(q, k_pages, v_pages, table, lens=None, count=None, L=None, out=None, lse=None, slopes=None, stream=None):
    """ALiBi attention of up to T new tokens of each sequence, a prompt or a part of one, over the pages that hold them
    and what came before. q: bf16 [B, H, T, d]; count: int32 CUDA tensor [B], the new tokens of each sequence (None: T); lens:
    their lengths, the new tokens included; k_pages, v_pages, table, L and slopes as in alibi_attn_decode_paged. Query t <
    count[b] has position lens[b] - count[b] + t; out and lse of tokens from count[b] on are left as they were, and a
    sequence with a count of 0 is not looked at, whatever its length.
    Returns (out, lse): bf16 [B, H, T, d] and fp32 [B, H, T]; those made here belong to `stream`."""
    lib = _kv4_names()[6]
    shape, index = _paged_query(q, (4,))
    B, H, T, d = shape
    pages, _, C = _paged_cache(k_pages, v_pages, table, B, d, index)
    L = _paged_bound(L, C, "alibi_attn_fwd_paged")
    out, lse = _paged_outputs(out, lse, q, shape, index, stream)
    _call_kv4(index, lib.alibi_attn_fwd_paged, "alibi_attn_fwd_paged", stream, q.data_ptr(), pages,
              _paged_ints(lens, B, index, "lens"), _paged_ints(count, B, index, "count"), out.data_ptr(), lse.data_ptr(), B, H, T, L,
              None if slopes is None else _slope_array(slopes, H))
    return out, lse


def alibi_attn_decode_splits(B: int, H: int, L: int, d: int) -> int:
    """KV splits alibi_attn_decode uses for this shape (1 = single kernel, no partials)."""
    s = load().alibi_attn_decode_splits(int(B), int(H), int(L), int(d))
    if s < 0:
        raise AlibiError(s, "alibi_attn_decode_splits")
    return s


def alibi_attn_probs_f32(q, k, lse, P=None, stream=None):
    """fp32 causal attention weights [B, H, N, N] from the LSE of alibi_attn_fwd_f32."""
    return alibi_attn_probs_f32_ex(q, k, lse, P, causal=True, stream=stream)


def alibi_attn_probs_f32_ex(q, k, lse, P=None, causal: bool = True, stream=None):
    """fp32 attention weights [B, H, N, N] from the LSE of alibi_attn_fwd_f32 (either mask)."""
    import torch
    _need(q, torch.float32, None, "q")
    B, H, N, d = q.shape
    _need(k, torch.float32, q.shape, "k")
    _need(lse, torch.float32, (B, H, N), "lse")
    if P is None:
        P = torch.empty((B, H, N, N), dtype=torch.float32, device=q.device)
    _need(P, torch.float32, (B, H, N, N), "P")
    _check(load().alibi_attn_probs_f32_ex(_ptr(q), _ptr(k), _ptr(lse), _ptr(P), B, H, N, d, int(bool(causal)),
                                          _stream(stream, q.device)), "alibi_attn_probs_f32_ex")
    return P


def alibi_attn_underflow_bf16(q, k, tau: float, counts=None, stream=None):
    """Per-head counts of causal pairs whose max-subtracted exponent is <= tau."""
    import torch
    _need(q, torch.bfloat16, None, "q")
    B, H, N, d = q.shape
    _need(k, torch.bfloat16, q.shape, "k")
    if counts is None:
        counts = torch.empty((H,), dtype=torch.int64, device=q.device)
    _need(counts, torch.int64, (H,), "counts")
    _check(load().alibi_attn_underflow_bf16(_ptr(q), _ptr(k), B, H, N, d, ctypes.c_float(tau), _ptr(counts),
                                            _stream(stream, q.device)), "alibi_attn_underflow_bf16")
    return counts


def alibi_decode_underflow_bf16(q, kcache, tau: float, counts=None, stream=None):
    """Per-head counts of cached keys whose max-subtracted exponent at the decode row is <= tau."""
    import torch
    _need(q, torch.bfloat16, None, "q")
    B, H, d = q.shape
    _need(kcache, torch.bfloat16, None, "kcache")
    if kcache.dim() != 4 or tuple(kcache.shape[:2]) != (B, H) or kcache.shape[3] != d:
        raise ValueError("kcache must be [B, H, L, d] matching q [B, H, d]")
    L = kcache.shape[2]
    if counts is None:
        counts = torch.empty((H,), dtype=torch.int64, device=q.device)
    _need(counts, torch.int64, (H,), "counts")
    _check(load().alibi_decode_underflow_bf16(_ptr(q), _ptr(kcache), B, H, L, d, ctypes.c_float(tau), _ptr(counts),
                                              _stream(stream, q.device)), "alibi_decode_underflow_bf16")
    return counts


def alibi_selftest_timeout(stream=None) -> None:
    """Launch the failure-path self-test (a bounded wait that must time out)."""
    import torch
    _check(load().alibi_selftest_timeout(_stream(stream, torch.cuda.current_device())), "alibi_selftest_timeout")


def alibi_selftest_fwd_timeout(q, k, v, wait_us: int = 20000, out=None, lse=None, stream=None):
    """Run the prefill kernel with one Q load left out and a short wait limit (failure-path self-test)."""
    import torch
    _need(q, torch.bfloat16, None, "q")
    B, H, N, d = q.shape
    _need(k, torch.bfloat16, q.shape, "k")
    _need(v, torch.bfloat16, q.shape, "v")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check(load().alibi_selftest_fwd_timeout(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d,
                                             int(wait_us), _stream(stream, q.device)), "alibi_selftest_fwd_timeout")
    return out, lse


def alibi_selftest_decode_paged_timeout(q, k_pages, v_pages, table, lens=None, L=None, out=None, lse=None, wait_us: int = 20000,
                                        stream=None):
    """Run the decode over pages with a wait of every CTA that must run out and a short limit (failure-path self-test)."""
    shape, index = _paged_query(q, (4,))
    B, H, T, d = shape
    pages, _, C = _paged_cache(k_pages, v_pages, table, B, d, index)
    L = _paged_bound(L, C, "alibi_selftest_decode_paged_timeout")
    out, lse = _paged_outputs(out, lse, q, shape, index, stream)
    _call_kv4(index, load().alibi_selftest_decode_paged_timeout, "alibi_selftest_decode_paged_timeout", stream, q.data_ptr(), pages,
              _paged_ints(lens, B, index, "lens"), out.data_ptr(), lse.data_ptr(), B, H, T, L, int(wait_us))
    return out, lse


def alibi_selftest_fwd_paged_timeout(q, k_pages, v_pages, table, barrier: int, lens=None, count=None, L=None, out=None, lse=None,
                                     wait_us: int = 20000, stream=None):
    """Run the prefill over pages with a barrier that waits for an arrival that nobody makes (alibi.h has their numbers) and a short
    wait limit (failure-path self-test)."""
    shape, index = _paged_query(q, (4,))
    B, H, T, d = shape
    pages, _, C = _paged_cache(k_pages, v_pages, table, B, d, index)
    L = _paged_bound(L, C, "alibi_selftest_fwd_paged_timeout")
    out, lse = _paged_outputs(out, lse, q, shape, index, stream)
    _call_kv4(index, load().alibi_selftest_fwd_paged_timeout, "alibi_selftest_fwd_paged_timeout", stream, q.data_ptr(), pages,
              _paged_ints(lens, B, index, "lens"), _paged_ints(count, B, index, "count"), out.data_ptr(), lse.data_ptr(), B, H, T, L,
              int(barrier), int(wait_us))
    return out, lse


def alibi_check_error(stream=None, device=None) -> None:
    """Synchronise and raise if a kernel recorded a device-side failure."""
    _check(load().alibi_check_error(_stream(stream, device)), "alibi_check_error")
