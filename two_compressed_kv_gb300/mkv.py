"""Thin Python binding of the C ABI in include/mkv.h (ctypes).

Argument marshalling only: every step of compression and decode runs in the
CUDA library libmkv.so.  Functions keep the C names.  Tensor arguments are
torch tensors on the ctx's device; the CUDA stream defaults to torch's current
stream.  A missing library is an ImportError, never a fallback.
"""
from __future__ import annotations

import ctypes
import itertools
import os
from ctypes import (POINTER, Structure, c_char_p, c_double, c_float, c_int, c_int32, c_int64,
                    c_uint8, c_uint16, c_uint32, c_uint64, c_void_p)

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmkv.so")

MKV_OK = 0
MKV_ERR_INVALID_ARG = 1
MKV_ERR_STATE = 2
MKV_ERR_OOM = 3
MKV_ERR_CUDA = 4
MKV_ERR_DEVICE_CHECK = 5
MKV_ERR_TIMEOUT = 6

MKV_STRATEGY_SM, MKV_STRATEGY_PV, MKV_STRATEGY_DENSE, MKV_STRATEGY_PVB = 0, 1, 2, 3
MKV_FLAG_KERNEL_TIMING = 1
MKV_FLAG_SCORE_TIMING = 2
MKV_FLAG_NO_PDL = 4
MKV_FLAG_BITMASK_PV = 8
MKV_BASIS_STATIC_MAX_BYTES = 16 << 20
(MKV_KERNEL_QROT, MKV_KERNEL_SCORE, MKV_KERNEL_TOPK, MKV_KERNEL_ATTN, MKV_KERNEL_MERGE,
 MKV_KERNEL_GRAM, MKV_KERNEL_EIG, MKV_KERNEL_ANALYZE, MKV_KERNEL_LAYOUT, MKV_KERNEL_PACK) = range(10)
KERNEL_NAMES = ["qrot", "score", "topk", "attn", "merge"]          # decode kernels
COMPRESS_KERNEL_NAMES = ["gram", "eig", "analyze", "layout", "pack"]  # ids 5..9


class mkv_config(Structure):
    _fields_ = [("batch", c_int32), ("n_kv_heads", c_int32), ("n_q_heads", c_int32),
                ("head_dim", c_int32), ("max_ctx", c_int64), ("segment", c_int32),
                ("c", c_int32), ("tau", c_float), ("top_k", c_int32), ("attn_chunk", c_int32),
                ("max_pool_bytes", c_uint64), ("flags", c_uint32), ("device", c_int32)]


class mkv_segment_header(Structure):
    _fields_ = [("off16", c_uint32), ("strategy", c_uint8), ("reserved", c_uint8),
                ("rows", c_uint16)]


class mkv_stats_t(Structure):
    _fields_ = [("ctx_len", c_int64), ("n_segments", c_int64),
                ("strategy_count", (c_int64 * 4) * 2), ("payload_bytes", c_uint64 * 2),
                ("header_bytes", c_uint64), ("uncompressed_bytes", c_uint64),
                ("pool_capacity", c_uint64), ("decode_calls", c_int64),
                ("kernel_launches", c_int64)]


HEADER_NP = np.dtype([("off16", "<u4"), ("strategy", "u1"), ("rsv", "u1"), ("rows", "<u2")])


MKV_DT_F16, MKV_DT_BF16, MKV_DT_F32, MKV_DT_E4M3 = range(4)
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}
MKV_ROPE_MAX_PAIRS = 128


class mkv_rope_config(Structure):
    _fields_ = [("head_dim", c_int32), ("rot_dim", c_int32), ("interleaved", c_int32),
                ("scaling", c_int32), ("base", c_double), ("factor", c_double),
                ("original", c_double), ("low_freq", c_double), ("high_freq", c_double),
                ("beta_fast", c_double), ("beta_slow", c_double), ("attn_factor", c_double)]


class MkvRopePlan(Structure):
    """A rotation ready to use (mkv_rope_plan_init): plain host data."""
    _fields_ = [("turn", c_uint64 * MKV_ROPE_MAX_PAIRS), ("mult", c_float),
                ("head_dim", c_int32), ("rot_dim", c_int32), ("interleaved", c_int32)]

    @property
    def address(self) -> int:
        return ctypes.addressof(self)


class mkv_rope_args(Structure):
    _fields_ = [("x", c_void_p), ("out", c_void_p), ("pos", c_void_p), ("x_stride", c_int64 * 3),
                ("out_stride", c_int64 * 3), ("pos_stride", c_int64), ("tokens", c_int64),
                ("batch", c_int32), ("heads", c_int32), ("dtype", c_int32),
                ("first_pos", c_int32), ("transposed", c_int32)]


class mkv_paged_cache(Structure):
    _fields_ = [("k_pages", c_void_p), ("v_pages", c_void_p), ("page_table", c_void_p),
                ("k_scale", c_void_p), ("v_scale", c_void_p), ("status", c_void_p),
                ("table_stride", c_int64), ("dtype", c_int32), ("batch", c_int32),
                ("n_kv_heads", c_int32), ("head_dim", c_int32), ("page_size", c_int32),
                ("n_pages", c_int32), ("max_pages", c_int32)]


class mkv_paged_append_args(Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("q", c_void_p), ("q_out", c_void_p),
                ("seq", c_void_p), ("slot", c_void_p), ("pos", c_void_p), ("acc", c_void_p),
                ("pos_meta", c_void_p), ("k_stride", c_int64 * 2), ("v_stride", c_int64 * 2),
                ("q_stride", c_int64 * 2), ("q_out_stride", c_int64 * 2), ("meta_stride", c_int64),
                ("n", c_int64), ("n_q_heads", c_int32), ("in_dtype", c_int32)]


class mkv_paged_decode_args(Structure):
    _fields_ = [("q", c_void_p), ("out", c_void_p), ("lse", c_void_p), ("seq_lens", c_void_p),
                ("acc", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_uint64),
                ("q_stride", c_int64 * 2), ("acc_stride", c_int64), ("max_len", c_int64),
                ("n_q_heads", c_int32), ("q_dtype", c_int32), ("out_dtype", c_int32),
                ("scale", c_float)]


class mkv_paged_evict_args(Structure):
    _fields_ = [("acc", c_void_p), ("pos", c_void_p), ("acc_out", c_void_p),
                ("pos_out", c_void_p), ("seq_lens", c_void_p), ("next_pos", c_void_p),
                ("lens_out", c_void_p), ("src", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_uint64), ("meta_stride", c_int64), ("out_stride", c_int64),
                ("max_len", c_int64), ("budget", c_int32), ("sink", c_int32), ("recent", c_int32)]


ROPE_ORDERS = {"blocks": 0, "cyclic": 1}
MKV_ROPE_MAX_AXES = 4


class mkv_rope_axes(Structure):
    _fields_ = [("n_axes", c_int32), ("axis", c_uint8 * MKV_ROPE_MAX_PAIRS)]


class MkvRopeAxes:
    """A rotation with several axes ready to use (mkv_rope_axes_init): plain host data."""

    def __init__(self):
        self.plan, self.axes = MkvRopePlan(), mkv_rope_axes()
        self.address, self.axes_address = self.plan.address, ctypes.addressof(self.axes)


class mkv_norm_rope_args(Structure):
    _fields_ = [("x", c_void_p * 2), ("out", c_void_p * 2), ("grad", c_void_p * 2),
                ("weight", c_void_p * 2), ("weight_grad", c_void_p * 2), ("pos", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_uint64),
                ("x_stride", c_int64 * 3 * 2), ("out_stride", c_int64 * 3 * 2),
                ("grad_stride", c_int64 * 3 * 2), ("pos_stride", c_int64),
                ("pos_axis_stride", c_int64), ("tokens", c_int64), ("batch", c_int32),
                ("heads", c_int32 * 2), ("dtype", c_int32), ("weight_dtype", c_int32),
                ("first_pos", c_int32), ("eps", c_float), ("weight_offset", c_float)]


class mkv_prefill_args(Structure):
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("out", c_void_p),
                ("lse", c_void_p), ("q_lens", c_void_p), ("kv_lens", c_void_p),
                ("prefix", c_void_p), ("docs", c_void_p), ("slopes", c_void_p), ("status", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_uint64), ("q_stride", c_int64 * 3),
                ("k_stride", c_int64 * 3), ("v_stride", c_int64 * 3), ("out_stride", c_int64 * 3),
                ("docs_stride", c_int64), ("q_tokens", c_int64), ("kv_tokens", c_int64),
                ("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32),
                ("head_dim", c_int32), ("dtype", c_int32), ("causal", c_int32),
                ("window", c_int32), ("scale", c_float), ("cap", c_float)]


class mkv_paged_attend_args(Structure):
    _fields_ = [("q", c_void_p), ("out", c_void_p), ("lse", c_void_p), ("seq_lens", c_void_p),
                ("new_lens", c_void_p), ("tree", c_void_p), ("slopes", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_uint64), ("q_stride", c_int64 * 3),
                ("max_len", c_int64), ("n", c_int32), ("n_q_heads", c_int32), ("q_dtype", c_int32),
                ("window", c_int32), ("scale", c_float), ("cap", c_float)]


class MkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {mkv_status_string(status)}"
        if status in (MKV_ERR_CUDA, MKV_ERR_OOM) or where.startswith(("mkv_rope", "mkv_paged", "mkv_norm", "mkv_prefill")):
            msg += f" ({mkv_last_error_string()})"
        super().__init__(msg)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run two_compressed_kv_gb300.build_lib.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P = c_void_p
    sig = {
        "mkv_validate_config": (c_int, [POINTER(mkv_config)]),
        "mkv_segment_bytes": (c_uint64, [c_int, c_int, c_int]),
        "mkv_create": (c_int, [POINTER(mkv_config), POINTER(P)]),
        "mkv_compress": (c_int, [P, P, P, c_int64, P]),
        "mkv_decode": (c_int, [P, P, P, P, P]),
        "mkv_decode_layers": (c_int, [P, c_int, P, P, P, P]),
        "mkv_free": (None, [P]),
        "mkv_status_string": (c_char_p, [c_int]),
        "mkv_last_error_string": (c_char_p, []),
        "mkv_stats": (c_int, [P, POINTER(mkv_stats_t)]),
        "mkv_export": (c_int, [P, c_int, c_int, c_int, P, P, P, P, POINTER(c_uint64)]),
        "mkv_kernel_time": (c_int, [P, c_int, POINTER(c_double), POINTER(c_int64), c_int]),
        "mkv_check_device": (c_int, [P]),
        "mkv_basis_static": (c_int, [P, P, c_int, c_int, c_int64, P, P, P]),
        "mkv_debug_wait_test": (c_int, [P, c_uint64, P]),
        "mkv_append": (c_int, [P, P, P, c_int32, P]),
        "mkv_set_flags": (c_int, [P, c_uint32]),
        "mkv_debug_set_pdl": (c_int, [P, c_uint32]),
        "mkv_debug_set_check_extent": (c_int, [P, c_uint64]),
        "mkv_rope_plan_init": (c_int, [P, P]),
        "mkv_rope": (c_int, [P, P, P]),
        "mkv_paged_validate": (c_int, [P]),
        "mkv_paged_append": (c_int, [P, P, P, P]),
        "mkv_paged_decode_workspace": (c_uint64, [P, P]),
        "mkv_paged_decode": (c_int, [P, P, P]),
        "mkv_paged_evict_workspace": (c_uint64, [P, P]),
        "mkv_paged_evict": (c_int, [P, P, P]),
        "mkv_paged_check": (c_int, [P]),
        "mkv_rope_axes_init": (c_int, [P, P, c_int32, c_int32, c_int32, P, P]),
        "mkv_rope_multi": (c_int, [P, P, P, c_int64, P]),
        "mkv_norm_rope": (c_int, [P, P, P, P]),
        "mkv_norm_rope_grad": (c_int, [P, P, P, P]),
        "mkv_norm_rope_grad_workspace": (c_uint64, [P, P]),
        "mkv_prefill_workspace": (c_uint64, [P]),
        "mkv_prefill": (c_int, [P, P]),
        "mkv_paged_attend_workspace": (c_uint64, [P, P]),
        "mkv_paged_attend": (c_int, [P, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()
lib = _lib


def _check(status: int, where: str):
    if status != MKV_OK:
        raise MkvError(status, where)


def _stream_ptr(stream, device=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dptr(t, dtype, name, shape=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def mkv_status_string(status: int) -> str:
    return _lib.mkv_status_string(status).decode()


def mkv_last_error_string() -> str:
    return _lib.mkv_last_error_string().decode()


def make_config(batch, n_kv_heads, n_q_heads, max_ctx, segment, c, tau, top_k,
                attn_chunk=0, max_pool_bytes=0, flags=0, device=0, head_dim=128) -> mkv_config:
    return mkv_config(batch=batch, n_kv_heads=n_kv_heads, n_q_heads=n_q_heads, head_dim=head_dim,
                      max_ctx=max_ctx, segment=segment, c=c, tau=tau, top_k=top_k,
                      attn_chunk=attn_chunk, max_pool_bytes=max_pool_bytes, flags=flags,
                      device=device)


def mkv_validate_config(cfg: mkv_config) -> int:
    return _lib.mkv_validate_config(ctypes.byref(cfg))


def mkv_segment_bytes(strategy: int, rows: int, c: int) -> int:
    return int(_lib.mkv_segment_bytes(strategy, rows, c))


def mkv_create(cfg: mkv_config) -> c_void_p:
    h = c_void_p()
    _check(_lib.mkv_create(ctypes.byref(cfg), ctypes.byref(h)), "mkv_create")
    return h


def mkv_free(ctx) -> None:
    _lib.mkv_free(ctx)


def mkv_compress(ctx, k, v, ctx_len=None, stream=None) -> None:
    import torch
    ctx_len = k.shape[2] if ctx_len is None else ctx_len
    pk = _dptr(k, torch.float16, "k")
    pv = _dptr(v, torch.float16, "v", k.shape)
    _check(_lib.mkv_compress(ctx, pk, pv, ctx_len, _stream_ptr(stream, k.device)), "mkv_compress")


def mkv_decode(ctx, q, out, sel=None, stream=None) -> None:
    import torch
    pq = _dptr(q, torch.float16, "q")
    po = _dptr(out, torch.float32, "out", q.shape)
    ps = None if sel is None else _dptr(sel, torch.int32, "sel")
    _check(_lib.mkv_decode(ctx, pq, po, ps, _stream_ptr(stream, q.device)), "mkv_decode")


MKV_MAX_FUSED_LAYERS = 64


def mkv_decode_layers(ctxs, qs, outs, sels=None, stream=None) -> None:
    """mkv_decode of several ctxs (same shape and state) in one launch per
    decode kernel.  ctxs: ctx handles; qs, outs (and sels, or None): one
    tensor per ctx, as for mkv_decode."""
    import torch
    n = len(ctxs)
    if len(qs) != n or len(outs) != n or (sels is not None and len(sels) != n):
        raise ValueError("ctxs, qs, outs and sels must have the same length")
    devs = {t.device for t in list(qs) + list(outs) + list(sels or []) if t is not None}
    if len(devs) > 1:
        raise ValueError("all tensors of one call must be on one device")
    arr = lambda vals: (c_void_p * max(1, n))(*vals)
    pc = arr([c if isinstance(c, int) else getattr(c, "value", c) for c in ctxs])
    pq = arr([_dptr(q, torch.float16, "q") for q in qs])
    po = arr([_dptr(o, torch.float32, "out", q.shape) for o, q in zip(outs, qs)])
    ps = None if sels is None else arr([None if t is None else _dptr(t, torch.int32, "sel")
                                        for t in sels])
    dev = qs[0].device if n else None
    with torch.cuda.device(dev):
        _check(_lib.mkv_decode_layers(pc, n, pq, po, ps, _stream_ptr(stream, dev)),
               "mkv_decode_layers")


def mkv_decode_layers_raw(ctxs, n: int, q_ptrs, out_ptrs, sel_ptrs=None, stream_ptr: int = 0) -> int:
    """Pointer-level call (no checks beyond the library's own); returns the status.
    Any of the arrays may be None (a NULL array)."""
    arr = lambda vals: None if vals is None else (c_void_p * max(1, len(vals)))(*vals)
    return _lib.mkv_decode_layers(arr(ctxs), n, arr(q_ptrs), arr(out_ptrs), arr(sel_ptrs),
                                  stream_ptr or None)


def mkv_append(ctx, k, v, stream=None) -> None:
    """k, v: fp16 [B][H][n][128] new tokens of every stream."""
    import torch
    pk = _dptr(k, torch.float16, "k")
    pv = _dptr(v, torch.float16, "v", k.shape)
    _check(_lib.mkv_append(ctx, pk, pv, int(k.shape[2]), _stream_ptr(stream, k.device)),
           "mkv_append")


def mkv_decode_raw(ctx, q_ptr: int, out_ptr: int, sel_ptr: int = 0, stream_ptr: int = 0) -> int:
    """Pointer-level call (no checks beyond the library's own); returns the status."""
    return _lib.mkv_decode(ctx, q_ptr, out_ptr, sel_ptr or None, stream_ptr or None)


def mkv_stats(ctx) -> dict:
    st = mkv_stats_t()
    _check(_lib.mkv_stats(ctx, ctypes.byref(st)), "mkv_stats")
    return {
        "ctx_len": st.ctx_len, "n_segments": st.n_segments,
        "strategy_count": [[st.strategy_count[x][i] for i in range(4)] for x in range(2)],
        "payload_bytes": [st.payload_bytes[0], st.payload_bytes[1]],
        "header_bytes": st.header_bytes, "uncompressed_bytes": st.uncompressed_bytes,
        "pool_capacity": st.pool_capacity, "decode_calls": st.decode_calls,
        "kernel_launches": st.kernel_launches,
    }


def mkv_export(ctx, b: int, h: int, which: int, n_segments: int):
    """(basis [128,128] fp32, eigvals [128] fp32, headers (structured), payload bytes)."""
    basis = np.zeros((128, 128), dtype=np.float32)
    lam = np.zeros(128, dtype=np.float32)
    hdr = np.zeros(n_segments, dtype=HEADER_NP)
    nbytes = c_uint64(0)
    _check(_lib.mkv_export(ctx, b, h, which, None, None, None, None, ctypes.byref(nbytes)),
           "mkv_export(size)")
    payload = np.zeros(max(1, nbytes.value), dtype=np.uint8)
    _check(_lib.mkv_export(ctx, b, h, which, basis.ctypes.data, lam.ctypes.data,
                           hdr.ctypes.data, payload.ctypes.data, ctypes.byref(nbytes)),
           "mkv_export")
    return basis, lam, hdr, payload[:nbytes.value].tobytes()


def mkv_export_headers(ctx, b: int, h: int, which: int, n_segments: int) -> np.ndarray:
    """Only the segment headers of one stream (off16 relative to the stream)."""
    hdr = np.zeros(n_segments, dtype=HEADER_NP)
    nbytes = c_uint64(0)
    _check(_lib.mkv_export(ctx, b, h, which, None, None, hdr.ctypes.data, None,
                           ctypes.byref(nbytes)), "mkv_export(headers)")
    return hdr


def mkv_check_device(ctx) -> int:
    """MKV_OK, or MKV_ERR_TIMEOUT when a bounded device wait gave up (synchronous)."""
    return _lib.mkv_check_device(ctx)


def mkv_set_flags(ctx, flags: int) -> None:
    _check(_lib.mkv_set_flags(ctx, int(flags)), "mkv_set_flags")


def mkv_debug_set_pdl(ctx, mask: int) -> None:
    """Measurement hook: decode kernels launched with PDL (bit k), bit 8 = no early signal."""
    _check(_lib.mkv_debug_set_pdl(ctx, int(mask)), "mkv_debug_set_pdl")


def mkv_debug_wait_test(ctx, limit_ns: int, stream=None) -> None:
    """Test hook: one CTA waits on an mbarrier nobody arrives on, for limit_ns."""
    _check(_lib.mkv_debug_wait_test(ctx, int(limit_ns), _stream_ptr(stream)),
           "mkv_debug_wait_test")


def mkv_debug_set_check_extent(ctx, nbytes: int) -> None:
    """Test hook: check pool accesses against min(nbytes, pool size); 0 resets."""
    _check(_lib.mkv_debug_set_check_extent(ctx, int(nbytes)), "mkv_debug_set_check_extent")


def mkv_kernel_time(ctx, kernel_id: int, reset: bool = False):
    ms = c_double(0.0)
    n = c_int64(0)
    _check(_lib.mkv_kernel_time(ctx, kernel_id, ctypes.byref(ms), ctypes.byref(n), int(reset)),
           "mkv_kernel_time")
    return ms.value, n.value


def mkv_basis_static(k, v, basis, eigvals, stream=None) -> None:
    """Bases and eigenvalues of every K and V stream, with no ctx and no
    allocation inside the library (its scratch is a static device buffer).
    k, v: fp16 [B][H][T][128]; basis: fp32 [2][B*H][128][128]; eigvals: fp32
    [2][B*H][128], all on the current CUDA device."""
    import torch
    devs = {t.device for t in (k, v, basis, eigvals)}
    if len(devs) != 1:
        raise ValueError("k, v, basis and eigvals must be on one device, got "
                         f"{sorted(map(str, devs))}")
    B, H, T, _ = k.shape
    pk = _dptr(k, torch.float16, "k", (B, H, T, 128))
    pv = _dptr(v, torch.float16, "v", (B, H, T, 128))
    pb = _dptr(basis, torch.float32, "basis", (2, B * H, 128, 128))
    pe = _dptr(eigvals, torch.float32, "eigvals", (2, B * H, 128))
    # the library works on the current device: make it the tensors' own
    with torch.cuda.device(k.device):
        _check(_lib.mkv_basis_static(pk, pv, B, H, T, pb, pe, _stream_ptr(stream, k.device)),
               "mkv_basis_static")


# ---- rotary positions and the paged cache ----------------------------------------------------
#
# These calls come once a layer and token, and their kernels take a few microseconds where the
# batch is small, so the tensors are checked and the argument structs filled in C++ (_marshal,
# csrc/py_marshal.cpp).

_T = None                      # torch, once a call needs it
_M = None                      # the marshalling module


def _native():
    """The marshalling module; loaded with torch by the first call that needs it."""
    global _T, _M
    if _M is None:
        import torch

        try:
            from . import _marshal
        except ImportError as e:
            raise ImportError("the marshalling module _marshal.so is missing or was built for another Python or "
                              "torch: run python -m two_compressed_kv_gb300.build_lib") from e
        _marshal.bind(*(ctypes.cast(getattr(_lib, f), c_void_p).value for f in (
            "mkv_rope", "mkv_paged_append", "mkv_paged_decode_workspace", "mkv_paged_decode",
            "mkv_paged_evict_workspace", "mkv_paged_evict", "mkv_rope_multi", "mkv_norm_rope",
            "mkv_norm_rope_grad", "mkv_norm_rope_grad_workspace", "mkv_prefill",
            "mkv_prefill_workspace", "mkv_paged_attend", "mkv_paged_attend_workspace")))
        _T, _M = torch, _marshal
    return _M


def _address(stream):
    """A stream (torch.cuda.Stream or its address) as an address; None stays None."""
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _new(shape, dtype, dev, stream):
    """A tensor from torch's caching allocator whose memory belongs to the stream that uses it."""
    if stream is None:
        return _T.empty(shape, dtype=dtype, device=dev)
    if isinstance(stream, int):
        stream = _T.cuda.ExternalStream(stream, device=dev)
    with _T.cuda.stream(stream):
        return _T.empty(shape, dtype=dtype, device=dev)


def mkv_rope_plan(head_dim, rot_dim=None, base=10000.0, interleaved=False, scaling="none",
                  factor=1.0, original=0.0, low_freq=1.0, high_freq=4.0, beta_fast=32.0,
                  beta_slow=1.0, attn_factor=0.0) -> MkvRopePlan:
    """The rotation that mkv_rope and mkv_paged_append take.  scaling: "none", "linear", "ntk",
    "yarn" or "banded" (see mkv_rope_config in include/mkv.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    cfg = mkv_rope_config(head_dim, head_dim if rot_dim is None else rot_dim, int(interleaved),
                          ROPE_SCALINGS[scaling], base, factor, original, low_freq, high_freq,
                          beta_fast, beta_slow, attn_factor)
    plan = MkvRopePlan()
    _check(_lib.mkv_rope_plan_init(ctypes.byref(cfg), ctypes.byref(plan)), "mkv_rope_plan_init")
    return plan


def mkv_rope(plan, x, pos=None, out=None, transposed=False, first_pos=0, stream=None):
    """Rotates x [batch, tokens, heads, head_dim] (fp16, bf16 or fp32; any strides, the last
    dimension contiguous) by the positions pos (int32 [batch, tokens]; None: first_pos + token)
    into out (new where None; may be x; e.g. a transposed view of a [batch, heads, tokens,
    head_dim] tensor).  transposed: the gradient of the call.  Returns out, which like the results
    of all calls here carries no autograd history: a backward pass calls it with transposed=True."""
    m = _native()
    if out is None and isinstance(x, _T.Tensor):
        out = _new(x.shape, x.dtype, x.device, stream)
    _check(m.rope(plan.address, x, pos, out, transposed, first_pos, _address(stream)), "mkv_rope")
    return out


class MkvPaged:
    """A paged cache over the caller's tensors: k_pages, v_pages [n_pages, kv_heads, page_size,
    head_dim] (fp16, bf16 or float8_e4m3fn), page_table int32 [batch, max_pages] (rows may be
    strided), k_scale and v_scale fp32 [kv_heads] (float8 only).  Holds the tensors and a status
    word, so keep it until its calls have ended; check() reports what kernels found outside the
    cache."""

    def __init__(self, k_pages, v_pages, page_table, k_scale=None, v_scale=None):
        _native()
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages), ("page_table", page_table)):
            if not isinstance(t, _T.Tensor):
                raise TypeError(f"{name} must be a torch tensor")
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [n_pages, kv_heads, page_size, head_dim]")
        if page_table.dim() != 2:
            raise ValueError("page_table must be [batch, max_pages]")
        types = {_T.float16: MKV_DT_F16, _T.bfloat16: MKV_DT_BF16, _T.float8_e4m3fn: MKV_DT_E4M3}
        if k_pages.dtype not in types:
            raise TypeError(f"k_pages must be one of {list(types)}, got {k_pages.dtype}")
        v = self.view = mkv_paged_cache()
        v.dtype = types[k_pages.dtype]
        v.k_pages = _dptr(k_pages, k_pages.dtype, "k_pages")
        v.v_pages = _dptr(v_pages, k_pages.dtype, "v_pages", k_pages.shape)
        if page_table.dtype != _T.int32:
            raise TypeError(f"page_table must be torch.int32, got {page_table.dtype}")
        v.batch, v.max_pages = page_table.shape
        if page_table.stride(1) != 1 and v.max_pages > 1:
            raise ValueError("page_table must be contiguous in its last dimension")
        v.page_table = page_table.data_ptr()
        v.table_stride = max(page_table.stride(0), v.max_pages) if v.batch == 1 else page_table.stride(0)
        v.n_pages, v.n_kv_heads, v.page_size, v.head_dim = k_pages.shape
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None:
                setattr(v, name, _dptr(s, _T.float32, name, (v.n_kv_heads,)))
        for t in (v_pages, page_table, k_scale, v_scale):
            if t is not None and t.device != k_pages.device:
                raise ValueError(f"all tensors of a cache must be on {k_pages.device}, one is on {t.device}")
        self.device = k_pages.device
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        self.k_scale, self.v_scale = k_scale, v_scale
        self.status = _T.zeros(1, dtype=_T.int32, device=self.device)
        with _T.cuda.device(self.device):        # zero before a call on any stream may set a bit
            if not _T.cuda.is_current_stream_capturing():
                _T.cuda.current_stream().synchronize()
        v.status = self.status.data_ptr()
        _check(_lib.mkv_paged_validate(ctypes.byref(v)), "mkv_paged_validate")
        self._address, self._dev = ctypes.addressof(v), self.device.index
        self._capacity = v.max_pages * v.page_size

    @property
    def capacity(self) -> int:
        """Slots the page table has room for in a sequence."""
        return self._capacity

    def check(self) -> int:
        """What kernels reported since the last check (synchronous): MKV_ERR_TIMEOUT when a bounded
        wait for a copy gave up (outputs undefined), else MKV_ERR_DEVICE_CHECK when one met a page,
        slot, sequence or length outside the cache, else MKV_OK.  mkv_last_error_string() names
        both where both happened."""
        with _T.cuda.device(self.device):
            return _lib.mkv_paged_check(self.status.data_ptr())


def mkv_paged_append(cache, k, v, slot, seq=None, plan=None, pos=None, q=None, q_out=None,
                     acc=None, pos_meta=None, stream=None):
    """Writes n tokens into the cache: k, v [n, kv_heads, head_dim], slot (and seq, pos) int32 [n];
    keys are rotated by plan at pos (None: the slot).  A negative slot is padding.  q [n, q_heads,
    head_dim] is rotated into q_out (new where None), which is returned.  acc (fp32) and pos_meta
    (int32) [batch, kv_heads, slots]: set to 0 and to the position in the written slots."""
    if q_out is None and isinstance(q, _T.Tensor):
        q_out = _new(q.shape, q.dtype, q.device, stream)
    _check(_M.append(cache._address, cache._dev, None if plan is None else plan.address, k, v, slot, seq,
                    pos, q, q_out, acc, pos_meta, _address(stream)), "mkv_paged_append")
    return q_out


def mkv_paged_decode(cache, q, seq_lens, out=None, lse=None, acc=None, max_len=0, scale=0.0,
                     out_dtype=None, workspace=None, stream=None):
    """Attention of one new token per sequence, q [batch, q_heads, head_dim], over its seq_lens
    (int32 [batch]) cached tokens.  out: contiguous, of q's type or fp32 (new, of out_dtype,
    where None), returned.  lse: fp32 [batch, q_heads] or None.  acc: fp32 [batch, kv_heads,
    slots] or None; every token's weights are added.  max_len: a bound on seq_lens (0: the page
    table's capacity, or, with acc, its slots where those are fewer); one near the lengths is faster.
    workspace: a uint8 tensor of mkv_paged_decode_workspace bytes (None: taken from torch's
    allocator)."""
    if out is None and isinstance(q, _T.Tensor):
        out = _new(q.shape, out_dtype or q.dtype, q.device, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
    _check(_M.decode(cache._address, cache._dev, cache._capacity, q, seq_lens, out, lse, acc, max_len, scale,
                    workspace, _address(stream)), "mkv_paged_decode")
    return out


def mkv_paged_decode_workspace(cache, q_heads, max_len=0, weights=False) -> int:
    """Bytes of workspace of mkv_paged_decode for these sizes (weights: with acc)."""
    qt = MKV_DT_F16 if cache.view.dtype == MKV_DT_E4M3 else cache.view.dtype
    a = mkv_paged_decode_args(n_q_heads=q_heads, max_len=max_len, acc=1 if weights else None,
                              q_dtype=qt, out_dtype=qt)
    with _T.cuda.device(cache.device):
        n = _lib.mkv_paged_decode_workspace(ctypes.byref(cache.view), ctypes.byref(a))
    if n == 0:
        raise MkvError(MKV_ERR_INVALID_ARG, "mkv_paged_decode_workspace")
    return n


def mkv_paged_evict_workspace(cache, budget, max_len=0) -> int:
    """Bytes of workspace of mkv_paged_evict for these sizes (max_len: the call's bound; 0: the
    page table's capacity, which is enough for a call without a bound too)."""
    a = mkv_paged_evict_args(budget=budget, max_len=max_len, meta_stride=max_len or cache.capacity,
                             out_stride=budget)
    with _T.cuda.device(cache.device):
        n = _lib.mkv_paged_evict_workspace(ctypes.byref(cache.view), ctypes.byref(a))
    if n == 0:
        raise MkvError(MKV_ERR_INVALID_ARG, "mkv_paged_evict_workspace")
    return n


def mkv_paged_evict(cache, acc, pos, seq_lens, next_pos, budget, sink=0, recent=0, acc_out=None,
                    pos_out=None, lens_out=None, src=None, max_len=0, workspace=None, stream=None):
    """Cuts every (sequence, KV head) down to `budget` tokens by accumulated weight, in place in
    the pages: the pages of a sequence that is cut must be its own (copy a common prefix first).
    acc (fp32), pos (int32) [batch, kv_heads, slots]; acc_out and pos_out [batch, kv_heads,
    slots_out] (None: in place, acc and pos themselves); seq_lens, next_pos int32 [batch]; lens_out
    int32 [batch] (None: seq_lens); src int32 [batch, kv_heads, budget] (new where None): the slot
    each kept token came from.  max_len: a bound on seq_lens (0: acc's slots or the page table's
    capacity, the fewer); one near the lengths is faster.  workspace: a uint8 tensor of
    mkv_paged_evict_workspace bytes (None: taken from torch's allocator).  Returns src."""
    if src is None:
        v = cache.view
        src = _new((v.batch, v.n_kv_heads, max(0, budget)), _T.int32, cache.device, stream)
    _check(_M.evict(cache._address, cache._dev, cache._capacity, acc, pos, seq_lens, next_pos, budget, sink, recent,
                   acc_out, pos_out, lens_out, src, max_len, workspace, _address(stream)), "mkv_paged_evict")
    return src


# ---- between projections and caches -----------------------------------------------------------

def mkv_rope_axes_plan(head_dim, sections, order="blocks", restart=False, rot_dim=None, base=10000.0,
                       interleaved=False, scaling="none", factor=1.0, original=0.0, low_freq=1.0,
                       high_freq=4.0, beta_fast=32.0, beta_slow=1.0, attn_factor=0.0) -> MkvRopeAxes:
    """A rotation with several axes (time, height, width): sections[a] pairs turn by the position of
    axis a, in "blocks" or dealt in turn ("cyclic"); restart: every axis has frequencies of its own,
    from 1 down.  rot_dim: twice the sections' sum where None."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    if order not in ROPE_ORDERS:
        raise ValueError(f"order must be one of {sorted(ROPE_ORDERS)}, got {order!r}")
    cfg = mkv_rope_config(head_dim, 2 * sum(sections) if rot_dim is None else rot_dim,
                          int(interleaved), ROPE_SCALINGS[scaling], base, factor, original, low_freq,
                          high_freq, beta_fast, beta_slow, attn_factor)
    made = MkvRopeAxes()
    n = len(sections)
    _check(_lib.mkv_rope_axes_init(ctypes.byref(cfg), (c_int32 * max(1, n))(*sections), n,
                                   ROPE_ORDERS[order], int(restart), made.address,
                                   made.axes_address), "mkv_rope_axes_init")
    return made


def mkv_rope_multi(plan, x, pos, out=None, transposed=False, stream=None):
    """mkv_rope with a rotation of several axes (mkv_rope_axes_plan): pos int32 [axes, batch,
    tokens].  transposed: the gradient of the call."""
    m = _native()
    if out is None and isinstance(x, _T.Tensor):
        out = _new(x.shape, x.dtype, x.device, stream)
    _check(m.rope_multi(plan.address, plan.axes_address, x, pos, out, transposed, _address(stream)),
           "mkv_rope_multi")
    return out


def mkv_norm_rope(plan, q, q_weight=None, pos=None, k=None, k_weight=None, eps=1e-6,
                  weight_offset=0.0, q_out=None, k_out=None, first_pos=0, stream=None):
    """RMS norm over every head of q (and k) [batch, tokens, heads, head_dim] and its rotation, in
    one pass: y = R(pos) (x / sqrt(mean(x^2) + eps) * (weight + weight_offset)).  plan:
    mkv_rope_plan, with pos int32 [batch, tokens] or None (first_pos + token), or
    mkv_rope_axes_plan, with pos [axes, batch, tokens].  Weights [head_dim]: of q's type or fp32,
    or None (1).  Returns q_out, or (q_out, k_out) with k (new where None; may be q and k)."""
    m = _native()
    if q_out is None and isinstance(q, _T.Tensor):
        q_out = _new(q.shape, q.dtype, q.device, stream)
    if k_out is None and isinstance(k, _T.Tensor):
        k_out = _new(k.shape, k.dtype, k.device, stream)
    _check(m.norm_rope(plan.address, getattr(plan, "axes_address", None), pos, q, q_weight, q_out, k, k_weight,
                       k_out, eps, weight_offset, first_pos, _address(stream), None, None, None, None, None),
           "mkv_norm_rope")
    return q_out if k is None else (q_out, k_out)


def mkv_norm_rope_grad(plan, dq, q, q_weight=None, pos=None, dk=None, k=None, k_weight=None, eps=1e-6,
                       weight_offset=0.0, dq_out=None, dk_out=None, q_weight_grad=None,
                       k_weight_grad=None, first_pos=0, workspace=None, stream=None):
    """Gradients of mkv_norm_rope: dq, dk are those of its results; q, k and the rest are its own
    arguments.  Returns (gradient of q, gradient of q_weight), or with k (of q, of k, of q_weight,
    of k_weight); those of the weights are fp32, written and not added to (None without a weight).
    workspace: a uint8 tensor of mkv_norm_rope_grad_workspace bytes (None: taken from torch's
    allocator)."""
    m = _native()
    if dq is None:
        raise TypeError("dq must be a torch tensor")
    if dq_out is None and isinstance(q, _T.Tensor):
        dq_out = _new(q.shape, q.dtype, q.device, stream)
    if dk_out is None and isinstance(k, _T.Tensor):
        dk_out = _new(k.shape, k.dtype, k.device, stream)
    if q_weight_grad is None and isinstance(q_weight, _T.Tensor):
        q_weight_grad = _new(q_weight.shape, _T.float32, q_weight.device, stream)
    if k_weight_grad is None and isinstance(k_weight, _T.Tensor):
        k_weight_grad = _new(k_weight.shape, _T.float32, k_weight.device, stream)
    _check(m.norm_rope(plan.address, getattr(plan, "axes_address", None), pos, q, q_weight, dq_out, k, k_weight,
                       dk_out, eps, weight_offset, first_pos, _address(stream), dq, dk, q_weight_grad,
                       k_weight_grad, workspace), "mkv_norm_rope_grad")
    return (dq_out, q_weight_grad) if k is None else (dq_out, dk_out, q_weight_grad, k_weight_grad)


def mkv_norm_rope_grad_workspace(plan, device=None) -> int:
    """Bytes of workspace of mkv_norm_rope_grad with a weight on `device` (None: the current one)."""
    _native()
    p = plan.plan if isinstance(plan, MkvRopeAxes) else plan
    a = mkv_norm_rope_args(dtype=MKV_DT_F32, weight_dtype=MKV_DT_F32)
    a.weight_grad[0] = 1
    with _T.cuda.device(device):
        n = _lib.mkv_norm_rope_grad_workspace(p.address, ctypes.byref(a))
    if n == 0:
        raise MkvError(MKV_ERR_INVALID_ARG, "mkv_norm_rope_grad_workspace")
    return n


def mkv_prefill(q, k, v, out=None, lse=None, causal=True, window=0, prefix=None, docs=None, q_lens=None,
                kv_lens=None, scale=0.0, cap=0.0, slopes=None, status=None, workspace=None, stream=None):
    """Attention of a prompt: q [batch, tokens, q_heads, head_dim] over k, v [batch, kv_tokens,
    kv_heads, head_dim] (fp16 or bf16, strided; a transposed view of a [batch, heads, tokens,
    head_dim] tensor is as good).  The last query stands at the last key; q_lens, kv_lens int32
    [batch]: how many there are of each sequence.  causal, window (keys less than that far away),
    prefix (int32 [batch]: keys seen by all queries), docs (int32 [batch, kv_tokens]: only keys of
    the query's document): which keys a query sees.  cap: scores become cap * tanh(score / cap);
    slopes (fp32 [q_heads]): slope * distance is taken off.  lse: fp32 [batch, tokens, q_heads] or
    None.  status: int32 [1] or None: set where a bounded wait gave up (outputs undefined then).
    workspace: a uint8 tensor of mkv_prefill_workspace bytes (None: taken from torch's allocator):
    for more than 16384 keys it takes four bytes an element of q, with a cap or slopes for each part
    of 32768 keys.
    Returns out (new where None), of q's shape and type; rows behind q_lens are left as they were."""
    m = _native()
    if out is None and isinstance(q, _T.Tensor):
        out = _new(q.shape, q.dtype, q.device, stream)
    _check(m.prefill(q, k, v, out, lse, q_lens, kv_lens, prefix, docs, slopes, causal, window, scale, cap, workspace,
                     _address(stream), status), "mkv_prefill")
    return out


def mkv_prefill_workspace(batch, q_tokens, kv_tokens, q_heads, kv_heads, head_dim, window=0, docs=False,
                          device=None, causal=None, prefix=None, capped=None) -> int:
    """Bytes of workspace of mkv_prefill for these sizes on `device` (None: the current one); 0: it
    needs none.  causal, prefix, capped (or biased): whether the call is so; None: enough for either."""
    _native()
    most = 0
    for c, p, t in itertools.product((1, 0), (0, 1), (0, 1)):
        if p > c or any(x is not None and y != bool(x) for x, y in ((causal, c), (prefix, p), (capped, t))):
            continue
        a = mkv_prefill_args(batch=batch, q_tokens=q_tokens, kv_tokens=kv_tokens, n_q_heads=q_heads,
                             n_kv_heads=kv_heads, head_dim=head_dim, dtype=MKV_DT_F16, window=window,
                             docs=1 if docs else None, causal=c, prefix=p or None, cap=t)
        with _T.cuda.device(device):
            n = _lib.mkv_prefill_workspace(ctypes.byref(a))
        if n == 2**64 - 1:
            raise MkvError(MKV_ERR_INVALID_ARG, "mkv_prefill_workspace")
        most = max(most, n)
    return most


def mkv_paged_attend(cache, q, seq_lens, tree=None, new_lens=None, out=None, lse=None, max_len=0, window=0,
                     scale=0.0, cap=0.0, slopes=None, workspace=None, stream=None):
    """Attention of the last new_lens (int32 [batch]; None: all) tokens of every sequence, q [batch,
    new_tokens, q_heads, head_dim], over its seq_lens (int32 [batch]) cached tokens, their own among
    them.  tree: int64 [batch, new_tokens], up to 64 of them: bit j of row i says that token i sees
    token j (None: a chain).  window, cap, slopes: as in mkv_prefill.  max_len: a bound on seq_lens
    (0: the page table's capacity); one near the lengths is faster.  lse: fp32 [batch, new_tokens,
    q_heads] or None.  workspace: a uint8 tensor of mkv_paged_attend_workspace bytes (None: taken
    from torch's allocator).  Returns out (new where None); rows behind new_lens are left as they
    were."""
    if out is None and isinstance(q, _T.Tensor):
        out = _new(q.shape, q.dtype, q.device, stream)
    _check(_M.attend(cache._address, cache._dev, q, seq_lens, out, lse, new_lens, tree, slopes, max_len, window, scale,
                     cap, workspace, _address(stream)), "mkv_paged_attend")
    return out


def mkv_paged_attend_workspace(cache, new_tokens, q_heads, max_len=0, window=0, capped=None) -> int:
    """Bytes of workspace of mkv_paged_attend for these sizes; 0: it needs none.  capped: whether the
    call has a cap or slopes; None: enough for either."""
    qt = MKV_DT_F16 if cache.view.dtype == MKV_DT_E4M3 else cache.view.dtype
    most = 0
    for t in (0, 1) if capped is None else (int(bool(capped)),):
        a = mkv_paged_attend_args(n=new_tokens, n_q_heads=q_heads, max_len=max_len, q_dtype=qt,
                                  window=window, cap=t)
        with _T.cuda.device(cache.device):
            n = _lib.mkv_paged_attend_workspace(ctypes.byref(cache.view), ctypes.byref(a))
        if n == 2**64 - 1:
            raise MkvError(MKV_ERR_INVALID_ARG, "mkv_paged_attend_workspace")
        most = max(most, n)
    return most


class Mkv:
    """Owns one ctx (one layer); frees it on close()."""

    def __init__(self, cfg: mkv_config):
        self.cfg = cfg
        self.ctx = mkv_create(cfg)
        self.T = 0

    @property
    def group(self) -> int:
        return self.cfg.n_q_heads // self.cfg.n_kv_heads

    def compress(self, k, v, stream=None):
        mkv_compress(self.ctx, k, v, k.shape[2], stream)
        self.T = k.shape[2]

    def append(self, k, v, stream=None):
        mkv_append(self.ctx, k, v, stream)
        self.T += k.shape[2]

    def decode(self, q, out=None, sel=None, stream=None):
        import torch
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        mkv_decode(self.ctx, q, out, sel, stream)
        return out

    def n_segments(self) -> int:
        return int(mkv_stats(self.ctx)["n_segments"])

    def export(self, b, h, which):
        return mkv_export(self.ctx, b, h, which, self.n_segments())

    def stats(self):
        return mkv_stats(self.ctx)

    def close(self):
        if self.ctx is not None:
            mkv_free(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()
