"""MXFP4 paged indexer cache for MI355X (gfx950): Python binding of libmxidx.so.

Thin ctypes layer over the C ABI in ``include/mxidx.h``: it checks tensor
dtypes/devices/shapes, allocates outputs with torch when the caller passes
none, and hands raw device pointers and the current HIP stream to the
library.  Every step of the path runs in the HIP kernels; there is no CPU or
PyTorch fallback, and a missing library raises ``MxidxError``.

Build the library with ``python -m mxfp4_paged_cache_quant_amd.build``.
"""

import collections
import ctypes
import os
import struct

__all__ = [
    "MxidxError", "lib", "lib_path", "version", "init",
    "quantize", "insert", "insert_quantize", "gather", "logits_prefill", "logits_paged",
    "logits_paged_insert", "topk", "topk_workspace_bytes", "topk_workspace", "topk_ws",
    "topk_noalloc", "topk_merge", "TOPK_NOALLOC_MAX_WORKSPACE",
    "quantize_rope", "insert_quantize_rope", "logits_paged_insert_rope", "ROPE_NEOX",
    "ROPE_INTERLEAVED", "kpool_insert",
    "quantize_fp8", "insert_fp8", "gather_fp8", "logits_prefill_fp8", "logits_paged_fp8",
    "logits_paged_insert_fp8",
    "StepMap", "step_map", "norm_rope", "latent_insert", "attn_paged", "attn_workspace_bytes",
    "attn_workspace_max_bytes", "attn_workspace", "LATENT_ROPE", "LATENT_DIMS",
    "latent_insert_mxfp4", "latent_gather_mxfp4", "latent_mxfp4_row_bytes", "attn_paged_mxfp4",
    "attn_prompt", "attn_prompt_workspace_bytes", "attn_prompt_workspace", "PROMPT_DIMS",
    "FP8_ROW_BYTES", "FP8_SCALE_F32", "FP8_SCALE_POW2",
    "HEAD_DIM", "ROW_BYTES", "PAGE_SIZE", "TOPK_MAX", "EXPORTS",
]

HEAD_DIM = 128
CODE_BYTES = 64
SCALE_BYTES = 4
ROW_BYTES = 68
PAGE_SIZE = 64
TOPK_MAX = 2048
MAX_HEADS = 128
TOPK_NOALLOC_MAX_WORKSPACE = 36 << 20
FP8_ROW_BYTES = 132
FP8_SCALE_F32, FP8_SCALE_POW2 = 0, 1
ROPE_NEOX, ROPE_INTERLEAVED = 0, 1
LATENT_ROPE = 64
LATENT_DIMS = (128, 256, 512)
PROMPT_DIMS = ((64, 64), (128, 128), (192, 128))     # (dk, dv) of attn_prompt
PROMPT_MAX_WORKSPACE = 36 << 20

IDX_BF16, IDX_F32 = 0, 1


class _Rope(ctypes.Structure):
    """The C ABI's idx_rope block (include/mxidx.h)."""
    _fields_ = [("cos_table", ctypes.c_void_p), ("sin_table", ctypes.c_void_p),
                ("table_rows", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("rope_dim", ctypes.c_int), ("rope_mode", ctypes.c_int)]


class _Heads(ctypes.Structure):
    """The C ABI's idx_heads block (include/mxidx.h)."""
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int), ("norm", ctypes.c_int), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("eps", ctypes.c_float)]


_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libmxidx.so")

_c_void_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_float = ctypes.c_float
_double = ctypes.c_double

# name -> (restype, argtypes); must match include/mxidx.h
EXPORTS = {
    "idx_version": (_int, []),
    "idx_strerror": (ctypes.c_char_p, [_int]),
    "idx_init": (_int, [_int]),
    "idx_arch_supported": (_int, [ctypes.c_char_p]),
    "idx_quantize": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "idx_quantize_rope": (_int, [_c_void_p, _int, _i64, _int, _i64, _c_void_p, _c_void_p, _i64,
                                 _c_void_p, _int, _int, _c_void_p, _c_void_p, _c_void_p]),
    "idx_insert": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _i64, _int, _c_void_p]),
    "idx_insert_quantize": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _i64, _int,
                                   _c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "idx_insert_quantize_rope": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _i64,
                                        _int, _c_void_p, _int, _i64, _i64, _int, _c_void_p,
                                        _c_void_p, _c_void_p, _c_void_p]),
    "idx_gather": (_int, [_c_void_p, _i64, _int, _c_void_p, _i64, _c_void_p, _c_void_p, _int, _i64,
                          _i64, _c_void_p, _c_void_p, _c_void_p]),
    "idx_logits_prefill": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                  _c_void_p, _i64, _int, _i64, _c_void_p, _i64, _int, _c_void_p]),
    "idx_logits_paged": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _int, _c_void_p,
                                _i64, _c_void_p, _int, _int, _int, _i64, _c_void_p, _i64, _int,
                                _c_void_p]),
    "idx_logits_paged_insert": (_int, [_c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _i64, _int,
                                       _c_void_p, _i64, _c_void_p, _int, _int, _int, _i64,
                                       _c_void_p, _i64, _int, _c_void_p]),
    "idx_logits_paged_insert_rope": (_int, [_c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _i64,
                                            _int, _c_void_p, _i64, _c_void_p, _int, _int, _int,
                                            _i64, _c_void_p, _i64, _int, _c_void_p, _c_void_p]),
    "idx_quantize_fp8": (_int, [_c_void_p, _int, _i64, _i64, _int, _c_void_p, _c_void_p, _c_void_p,
                                _c_void_p, _c_void_p]),
    "idx_insert_fp8": (_int, [_c_void_p, _int, _i64, _i64, _int, _c_void_p, _c_void_p, _i64, _int,
                              _c_void_p]),
    "idx_gather_fp8": (_int, [_c_void_p, _i64, _int, _c_void_p, _i64, _c_void_p, _c_void_p, _int,
                              _i64, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "idx_logits_prefill_fp8": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                      _c_void_p, _i64, _int, _i64, _c_void_p, _i64, _int,
                                      _c_void_p]),
    "idx_logits_paged_fp8": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _int, _c_void_p, _i64,
                                    _c_void_p, _int, _int, _int, _i64, _c_void_p, _i64, _int,
                                    _c_void_p]),
    "idx_logits_paged_insert_fp8": (_int, [_c_void_p, _c_void_p, _int, _c_void_p, _int, _c_void_p,
                                           _i64, _int, _c_void_p, _i64, _c_void_p, _int, _int, _int,
                                           _i64, _c_void_p, _i64, _int, _c_void_p]),
    "idx_kpool_insert": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _int,
                                _int, _int, _c_void_p, _i64, _int, _c_void_p, _c_void_p]),
    "idx_topk": (_int, [_c_void_p, _i64, _i64, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p]),
    "idx_topk_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "idx_topk_ws": (_int, [_c_void_p, _i64, _i64, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p,
                           ctypes.c_size_t, _c_void_p]),
    "idx_topk_noalloc": (_int, [_c_void_p, _i64, _i64, _c_void_p, _c_void_p, _int, _c_void_p,
                                _c_void_p]),
    "idx_topk_merge": (_int, [_c_void_p, _c_void_p, _int, _i64, _int, _int, _int, _c_void_p,
                              _c_void_p]),
    "idx_step_map": (_int, [_c_void_p, _c_void_p, _int, _c_void_p, _i64, _i64, _c_void_p, _i64,
                            _c_void_p, _c_void_p, _int, _int, _i64, _c_void_p, _c_void_p, _c_void_p,
                            _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "idx_norm_rope": (_int, [_c_void_p, _c_void_p, _int, _i64, _c_void_p, _c_void_p]),
    "idx_latent_insert": (_int, [_c_void_p, _int, _i64, _i64, _int, _int, _c_void_p, _float,
                                 _c_void_p, _c_void_p, _c_void_p, _i64, _int, _c_void_p, _int, _i64,
                                 _i64, _c_void_p, _i64, _i64, _c_void_p]),
    "idx_latent_insert_mxfp4": (_int, [_c_void_p, _int, _i64, _i64, _int, _int, _c_void_p, _double,
                                       _c_void_p, _c_void_p, _c_void_p, _i64, _int, _c_void_p, _int,
                                       _i64, _i64, _c_void_p, _i64, _i64, _c_void_p]),
    "idx_latent_gather_mxfp4": (_int, [_c_void_p, _i64, _int, _int, _c_void_p, _i64, _c_void_p,
                                       _c_void_p, _int, _i64, _i64, _c_void_p, _i64, _c_void_p]),
    "idx_attn_workspace_bytes": (ctypes.c_size_t, [_i64, _int, _int, _i64]),
    "idx_attn_workspace_bytes_mxfp4": (ctypes.c_size_t, [_i64, _int, _int, _i64]),
    "idx_attn_workspace_max_bytes": (ctypes.c_size_t, [_i64, _int, _int, _i64]),
    "idx_attn_paged": (_int, [_c_void_p, _i64, _i64, _i64, _int, _int, _c_void_p, _i64, _int,
                              _c_void_p, _i64, _int, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                              _i64, _int, _i64, _float, _c_void_p, _i64, _i64, _c_void_p, _c_void_p,
                              ctypes.c_size_t, _c_void_p]),
    "idx_attn_paged_mxfp4": (_int, [_c_void_p, _i64, _i64, _i64, _int, _int, _c_void_p, _i64, _int,
                                    _c_void_p, _i64, _int, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _i64, _int, _i64, _float, _c_void_p, _i64, _i64, _c_void_p, _c_void_p,
                                    ctypes.c_size_t, _c_void_p]),
    "idx_attn_prompt_workspace_bytes": (ctypes.c_size_t, [_i64, _int, _int, _int, _int, _int, _i64]),
    "idx_attn_prompt": (_int, [_c_void_p, _i64, _i64, _i64, _int, _c_void_p, _i64, _i64, _c_void_p, _i64,
                               _i64, _i64, _int, _int, _int, _c_void_p, _c_void_p, _int, _i64, _int,
                               _float, _c_void_p, _i64, _i64, _c_void_p, _c_void_p, ctypes.c_size_t,
                               _c_void_p]),
    "idx_entry": (_int, [ctypes.c_char_p]),
    "idx_call": (_int, [_int, ctypes.c_char_p, _int]),
}


class MxidxError(RuntimeError):
    def __init__(self, what, status=None):
        self.status = status
        super().__init__(what)


_LIB = None


def lib():
    """The loaded ctypes library (raises MxidxError when it is not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(lib_path):
            raise MxidxError(f"{lib_path} is not built: run python -m mxfp4_paged_cache_quant_amd.build")
        handle = ctypes.CDLL(lib_path)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def _check(status, call):
    if status != 0:
        msg = lib().idx_strerror(status).decode()
        raise MxidxError(f"{call}: {msg} (status {status})", status)


def version():
    return lib().idx_version()


def init(device=0):
    _check(lib().idx_init(device), "idx_init")


# ---------------------------------------------------------------------------
# torch-facing wrappers (torch supplies device memory and the stream only)
# ---------------------------------------------------------------------------

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, name, dtype=None):
    if not t.is_cuda:
        raise MxidxError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise MxidxError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _rows_view(x, name):
    """[..., 128] tensor with unit inner stride -> (rows, row_stride, dtype code)."""
    torch = _torch()
    _dev(x, name)
    if x.dtype == torch.bfloat16:
        code = IDX_BF16
    elif x.dtype == torch.float32:
        code = IDX_F32
    else:
        raise MxidxError(f"{name} must be bfloat16 or float32")
    if x.dim() >= 1 and x.shape[-1] == HEAD_DIM and x.numel() == 0:
        return 0, HEAD_DIM, code                   # no rows: strides are irrelevant
    if x.shape[-1] != HEAD_DIM or x.stride(-1) != 1:
        raise MxidxError(f"{name} must be [..., 128] with a contiguous last dim")
    rows = x.numel() // HEAD_DIM
    if x.dim() == 1:
        stride = HEAD_DIM
    else:
        x2 = x.reshape(-1, HEAD_DIM) if x.dim() > 2 else x
        if x2.data_ptr() != x.data_ptr():
            raise MxidxError(f"{name} rows must be addressable with one row stride")
        stride = x2.stride(0) if rows > 1 else HEAD_DIM
    return rows, stride, code


def quantize(x, values=None, scales=None, stream=None):
    """MXFP4-encode rows of 128 values: returns (values u8 [..., 64], scales u8 [..., 4])."""
    torch = _torch()
    rows, stride, code = _rows_view(x, "x")
    lead = tuple(x.shape[:-1])
    if values is None:
        values = torch.empty(lead + (CODE_BYTES,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(lead + (SCALE_BYTES,), dtype=torch.uint8, device=x.device)
    _dev(values, "values", torch.uint8)
    _dev(scales, "scales", torch.uint8)
    if values.numel() != rows * CODE_BYTES or scales.numel() != rows * SCALE_BYTES or \
            not values.is_contiguous() or not scales.is_contiguous():
        raise MxidxError("values/scales must be contiguous [rows, 64] / [rows, 4]")
    _check(lib().idx_quantize(_ptr(x), code, rows, stride, _ptr(values), _ptr(scales), _stream(stream)),
           "idx_quantize")
    return values, scales


def _check_rope_tables(cos, sin, rope_dim, positions, tokens):
    torch = _torch()
    for name, t in (("cos", cos), ("sin", sin)):
        _dev(t, name, torch.float32)
        if not t.is_contiguous() or t.dim() != 2 or t.shape[1] != rope_dim // 2:
            raise MxidxError(f"{name} must be a contiguous fp32 [table_rows, rope_dim/2]")
    if cos.shape != sin.shape:
        raise MxidxError("cos and sin tables must have the same shape")
    if positions is not None:
        _dev(positions, "positions", torch.int64)
        if positions.numel() != tokens or not positions.is_contiguous():
            raise MxidxError(f"positions must be a contiguous int64 [{tokens}]")


def _rope_block(cos, sin, rope_dim, mode, positions):
    """The idx_rope block of a fused call (the tensors must outlive the call)."""
    return _Rope(_ptr(cos), _ptr(sin), cos.shape[0], _ptr(positions), rope_dim,
                 {"neox": ROPE_NEOX, "interleaved": ROPE_INTERLEAVED}[mode])


def quantize_rope(q, cos, sin, rope_dim, mode="neox", positions=None, values=None, scales=None,
                  stream=None):
    """RoPE on the first ``rope_dim`` dims of each head of q [T, H, 128] (cos / sin
    fp32 [table_rows, rope_dim/2], table row positions[t] or t; ``mode`` "neox" or
    "interleaved"), then MXFP4: returns (values u8 [T, H, 64], scales u8 [T, H, 4])."""
    torch = _torch()
    if q.dim() != 3:
        raise MxidxError("q must be [T, H, 128]")
    T, H = q.shape[0], q.shape[1]
    rows, stride, code = _rows_view(q, "q")
    _check_rope_tables(cos, sin, rope_dim, positions, T)
    if values is None:
        values = torch.empty((T, H, CODE_BYTES), dtype=torch.uint8, device=q.device)
    if scales is None:
        scales = torch.empty((T, H, SCALE_BYTES), dtype=torch.uint8, device=q.device)
    _dev(values, "values", torch.uint8)
    _dev(scales, "scales", torch.uint8)
    if values.numel() != rows * CODE_BYTES or scales.numel() != rows * SCALE_BYTES or \
            not values.is_contiguous() or not scales.is_contiguous():
        raise MxidxError("values/scales must be contiguous [T, H, 64] / [T, H, 4]")
    mode_code = {"neox": ROPE_NEOX, "interleaved": ROPE_INTERLEAVED}[mode]
    _check(lib().idx_quantize_rope(_ptr(q), code, T, H, stride, _ptr(cos), _ptr(sin), cos.shape[0],
                                   _ptr(positions), rope_dim, mode_code, _ptr(values), _ptr(scales),
                                   _stream(stream)), "idx_quantize_rope")
    return values, scales


def insert(k, slot_mapping, cache, stream=None):
    """Quantize K rows [N, 128] and scatter them into ``cache`` [num_pages, 64*68] (in place)."""
    torch = _torch()
    rows, stride, code = _rows_view(k, "k")
    _dev(slot_mapping, "slot_mapping", torch.int64)
    _dev(cache, "cache", torch.uint8)
    if slot_mapping.numel() != rows or not slot_mapping.is_contiguous():
        raise MxidxError("slot_mapping must be a contiguous int64 [N]")
    if not cache.is_contiguous() or cache.numel() % (PAGE_SIZE * ROW_BYTES) != 0:
        raise MxidxError("cache must be a contiguous uint8 [num_pages, 64*68]")
    num_pages = cache.numel() // (PAGE_SIZE * ROW_BYTES)
    _check(lib().idx_insert(_ptr(k), code, rows, stride, _ptr(slot_mapping), _ptr(cache), num_pages,
                            PAGE_SIZE, _stream(stream)), "idx_insert")
    return cache


def insert_quantize(k, slot_mapping, cache, q, q_values=None, q_scales=None, stream=None):
    """insert(k, slot_mapping, cache) and quantize(q) in one launch; returns (q_values, q_scales)."""
    torch = _torch()
    rows, stride, code = _rows_view(k, "k")
    q_rows, q_stride, q_code = _rows_view(q, "q")
    _dev(slot_mapping, "slot_mapping", torch.int64)
    _dev(cache, "cache", torch.uint8)
    if slot_mapping.numel() != rows or not slot_mapping.is_contiguous():
        raise MxidxError("slot_mapping must be a contiguous int64 [N]")
    if not cache.is_contiguous() or cache.numel() % (PAGE_SIZE * ROW_BYTES) != 0:
        raise MxidxError("cache must be a contiguous uint8 [num_pages, 64*68]")
    lead = tuple(q.shape[:-1])
    if q_values is None:
        q_values = torch.empty(lead + (CODE_BYTES,), dtype=torch.uint8, device=q.device)
    if q_scales is None:
        q_scales = torch.empty(lead + (SCALE_BYTES,), dtype=torch.uint8, device=q.device)
    _dev(q_values, "q_values", torch.uint8)
    _dev(q_scales, "q_scales", torch.uint8)
    if q_values.numel() != q_rows * CODE_BYTES or q_scales.numel() != q_rows * SCALE_BYTES or \
            not q_values.is_contiguous() or not q_scales.is_contiguous():
        raise MxidxError("q_values/q_scales must be contiguous [rows, 64] / [rows, 4]")
    num_pages = cache.numel() // (PAGE_SIZE * ROW_BYTES)
    _check(lib().idx_insert_quantize(_ptr(k), code, rows, stride, _ptr(slot_mapping), _ptr(cache),
                                     num_pages, PAGE_SIZE, _ptr(q), q_code, q_rows, q_stride,
                                     _ptr(q_values), _ptr(q_scales), _stream(stream)),
           "idx_insert_quantize")
    return q_values, q_scales


def insert_quantize_rope(k, slot_mapping, cache, q, cos, sin, rope_dim, mode="neox",
                         positions=None, q_values=None, q_scales=None, stream=None):
    """insert(k, slot_mapping, cache) and quantize_rope(q [T, H, 128], ...) in one
    launch; returns (q_values [T, H, 64], q_scales [T, H, 4])."""
    torch = _torch()
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        raise MxidxError("q must be [T, H, 128]")
    T, H = q.shape[0], q.shape[1]
    rows, stride, code = _rows_view(k, "k")
    q_rows, q_stride, q_code = _rows_view(q, "q")
    _check_rope_tables(cos, sin, rope_dim, positions, T)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    _dev(cache, "cache", torch.uint8)
    if slot_mapping.numel() != rows or not slot_mapping.is_contiguous():
        raise MxidxError("slot_mapping must be a contiguous int64 [N]")
    if not cache.is_contiguous() or cache.numel() % (PAGE_SIZE * ROW_BYTES) != 0:
        raise MxidxError("cache must be a contiguous uint8 [num_pages, 64*68]")
    if q_values is None:
        q_values = torch.empty((T, H, CODE_BYTES), dtype=torch.uint8, device=q.device)
    if q_scales is None:
        q_scales = torch.empty((T, H, SCALE_BYTES), dtype=torch.uint8, device=q.device)
    _dev(q_values, "q_values", torch.uint8)
    _dev(q_scales, "q_scales", torch.uint8)
    if q_values.numel() != q_rows * CODE_BYTES or q_scales.numel() != q_rows * SCALE_BYTES or \
            not q_values.is_contiguous() or not q_scales.is_contiguous():
        raise MxidxError("q_values/q_scales must be contiguous [T, H, 64] / [T, H, 4]")
    rope = _rope_block(cos, sin, rope_dim, mode, positions)
    num_pages = cache.numel() // (PAGE_SIZE * ROW_BYTES)
    _check(lib().idx_insert_quantize_rope(_ptr(k), code, rows, stride, _ptr(slot_mapping),
                                          _ptr(cache), num_pages, PAGE_SIZE, _ptr(q), q_code,
                                          q_rows, q_stride, H, ctypes.addressof(rope),
                                          _ptr(q_values), _ptr(q_scales), _stream(stream)),
           "idx_insert_quantize_rope")
    return q_values, q_scales


def gather(cache, block_table, seq_lens, cu_seq_offsets, max_seq_len, total_tokens,
           k_values=None, k_scales=None, stream=None):
    """Paged cache -> contiguous (k_values u8 [total, 64], k_scales u8 [total, 4])."""
    torch = _torch()
    _dev(cache, "cache", torch.uint8)
    _dev(block_table, "block_table", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(cu_seq_offsets, "cu_seq_offsets", torch.int64)
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise MxidxError("block_table must be [batch, pages] with unit inner stride")
    batch = block_table.shape[0]
    if seq_lens.numel() != batch or cu_seq_offsets.numel() != batch:
        raise MxidxError("seq_lens / cu_seq_offsets must have one entry per sequence")
    if block_table.shape[1] * PAGE_SIZE < max_seq_len or not cache.is_contiguous():
        raise MxidxError("block_table has fewer pages than max_seq_len needs")
    if k_values is None:
        k_values = torch.zeros((total_tokens, CODE_BYTES), dtype=torch.uint8, device=cache.device)
    if k_scales is None:
        k_scales = torch.zeros((total_tokens, SCALE_BYTES), dtype=torch.uint8, device=cache.device)
    for name, t, cols in (("k_values", k_values, CODE_BYTES), ("k_scales", k_scales, SCALE_BYTES)):
        _dev(t, name, torch.uint8)
        if not t.is_contiguous() or t.numel() < total_tokens * cols:
            raise MxidxError(f"{name} must be a contiguous uint8 [total_tokens, {cols}]")
    num_pages = cache.numel() // (PAGE_SIZE * ROW_BYTES)
    _check(lib().idx_gather(_ptr(cache), num_pages, PAGE_SIZE, _ptr(block_table), block_table.stride(0),
                            _ptr(seq_lens), _ptr(cu_seq_offsets), batch, int(max_seq_len),
                            int(total_tokens), _ptr(k_values), _ptr(k_scales), _stream(stream)),
           "idx_gather")
    return k_values, k_scales


def logits_prefill(q_values, q_scales, k_values, k_scales, weights, ks, ke, logits=None,
                   clean=True, stream=None):
    """Dense logits [T, S] (fp32) for rows t over columns [ks[t], ke[t])."""
    torch = _torch()
    T, H = q_values.shape[0], q_values.shape[1]
    S = k_values.shape[0]
    for name, t, dt in (("q_values", q_values, torch.uint8), ("q_scales", q_scales, torch.uint8),
                        ("k_values", k_values, torch.uint8), ("k_scales", k_scales, torch.uint8),
                        ("weights", weights, torch.float32), ("ke", ke, torch.int32)):
        _dev(t, name, dt)
        if not t.is_contiguous():
            raise MxidxError(f"{name} must be contiguous")
    if ks is not None:
        _dev(ks, "ks", torch.int32)
    if tuple(q_values.shape) != (T, H, CODE_BYTES) or tuple(q_scales.shape) != (T, H, SCALE_BYTES) \
            or tuple(k_values.shape) != (S, CODE_BYTES) or tuple(k_scales.shape) != (S, SCALE_BYTES) \
            or tuple(weights.shape) != (T, H):
        raise MxidxError("shape mismatch among q/k/weights")
    if ke.numel() != T or (ks is not None and (ks.numel() != T or not ks.is_contiguous())):
        raise MxidxError("ks / ke must hold one entry per query row")
    if logits is None:
        fill = float("-inf") if clean else 0.0
        logits = torch.full((T, S), fill, dtype=torch.float32, device=q_values.device)
    _dev(logits, "logits", torch.float32)
    if logits.dim() != 2 or logits.stride(1) != 1 or logits.shape[0] < T or logits.shape[1] < S:
        raise MxidxError("logits must be [>=T, >=S] with contiguous rows")
    _check(lib().idx_logits_prefill(_ptr(q_values), _ptr(q_scales), _ptr(k_values), _ptr(k_scales),
                                    _ptr(weights), _ptr(ks), _ptr(ke), T, H, S, _ptr(logits),
                                    logits.stride(0), 1 if clean else 0, _stream(stream)),
           "idx_logits_prefill")
    return logits


def logits_paged(q_values, q_scales, weights, cache, block_table, context_lens, next_n,
                 max_context_len, logits=None, clean=True, stream=None):
    """Decode logits [B*next_n, max_context_len] (fp32) read through the block table."""
    torch = _torch()
    R, H = q_values.shape[0], q_values.shape[1]
    B = context_lens.numel()
    for name, t, dt in (("q_values", q_values, torch.uint8), ("q_scales", q_scales, torch.uint8),
                        ("weights", weights, torch.float32), ("cache", cache, torch.uint8),
                        ("block_table", block_table, torch.int32),
                        ("context_lens", context_lens, torch.int32)):
        _dev(t, name, dt)
    if R != B * next_n:
        raise MxidxError("q rows must be batch * next_n")
    for name, t in (("q_values", q_values), ("q_scales", q_scales), ("weights", weights),
                    ("cache", cache), ("context_lens", context_lens)):
        if not t.is_contiguous():
            raise MxidxError(f"{name} must be contiguous")
    if tuple(q_values.shape) != (R, H, CODE_BYTES) or tuple(q_scales.shape) != (R, H, SCALE_BYTES) \
            or tuple(weights.shape) != (R, H):
        raise MxidxError("shape mismatch among q/weights")
    if block_table.dim() != 2 or block_table.stride(1) != 1 or block_table.shape[0] != B:
        raise MxidxError("block_table must be [batch, pages] with unit inner stride")
    if block_table.shape[1] * PAGE_SIZE < max_context_len:
        raise MxidxError("block_table has fewer pages than max_context_len needs")
    if logits is None:
        fill = float("-inf") if clean else 0.0
        logits = torch.full((R, max_context_len), fill, dtype=torch.float32, device=q_values.device)
    _dev(logits, "logits", torch.float32)
    if logits.dim() != 2 or logits.stride(1) != 1 or logits.shape[0] < R or \
            logits.shape[1] < max_context_len:
        raise MxidxError("logits must be [>=rows, >=max_context_len] with contiguous rows")
    num_pages = cache.numel() // (PAGE_SIZE * ROW_BYTES)
    _check(lib().idx_logits_paged(_ptr(q_values), _ptr(q_scales), _ptr(weights), _ptr(cache), num_pages,
                                  PAGE_SIZE, _ptr(block_table), block_table.stride(0),
                                  _ptr(context_lens), B, next_n, H, int(max_context_len),
                                  _ptr(logits), logits.stride(0), 1 if clean else 0, _stream(stream)),
           "idx_logits_paged")
    return logits


def _paged_insert_args(q, k_new, weights, cache, block_table, context_lens, next_n,
                       max_context_len, logits, clean):
    """Checks of the one-launch decode step; returns (dtype code, rows, heads,
    batch, logits, num_pages)."""
    torch = _torch()
    for name, t in (("q", q), ("k_new", k_new)):
        _dev(t, name)
        if t.dtype not in (torch.bfloat16, torch.float32):
            raise MxidxError(f"{name} must be bfloat16 or float32")
        if not t.is_contiguous():
            raise MxidxError(f"{name} must be contiguous")
    if k_new.dtype != q.dtype:
        raise MxidxError("q and k_new must have one dtype")
    code = IDX_BF16 if q.dtype == torch.bfloat16 else IDX_F32
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        raise MxidxError("q must be [rows, heads, 128]")
    R, H = q.shape[0], q.shape[1]
    B = context_lens.numel()
    if R != B * next_n:
        raise MxidxError("q rows must be batch * next_n")
    if tuple(k_new.shape) != (R, HEAD_DIM):
        raise MxidxError("k_new must be [batch * next_n, 128]")
    for name, t, dt in (("weights", weights, torch.float32), ("cache", cache, torch.uint8),
                        ("block_table", block_table, torch.int32),
                        ("context_lens", context_lens, torch.int32)):
        _dev(t, name, dt)
    for name, t in (("weights", weights), ("cache", cache), ("context_lens", context_lens)):
        if not t.is_contiguous():
            raise MxidxError(f"{name} must be contiguous")
    if tuple(weights.shape) != (R, H):
        raise MxidxError("weights must be [rows, heads]")
    if block_table.dim() != 2 or block_table.stride(1) != 1 or block_table.shape[0] != B:
        raise MxidxError("block_table must be [batch, pages] with unit inner stride")
    if block_table.shape[1] * PAGE_SIZE < max_context_len:
        raise MxidxError("block_table has fewer pages than max_context_len needs")
    if logits is None:
        fill = float("-inf") if clean else 0.0
        logits = torch.full((R, max_context_len), fill, dtype=torch.float32, device=q.device)
    _dev(logits, "logits", torch.float32)
    if logits.dim() != 2 or logits.stride(1) != 1 or logits.shape[0] < R or \
            logits.shape[1] < max_context_len:
        raise MxidxError("logits must be [>=rows, >=max_context_len] with contiguous rows")
    num_pages = cache.numel() // (PAGE_SIZE * ROW_BYTES)
    return code, R, H, B, logits, num_pages


def logits_paged_insert(q, k_new, weights, cache, block_table, context_lens, next_n,
                        max_context_len, logits=None, clean=True, stream=None):
    """One decode step in one launch: the new tokens' K (k_new [B*next_n, 128], the
    last next_n positions of each sequence) into their block-table slots, q
    [B*next_n, H, 128] encoded to MXFP4, and the decode logits [B*next_n,
    max_context_len] of the updated cache (as insert + quantize + logits_paged)."""
    code, R, H, B, logits, num_pages = _paged_insert_args(
        q, k_new, weights, cache, block_table, context_lens, next_n, max_context_len, logits,
        clean)
    _check(lib().idx_logits_paged_insert(_ptr(q), _ptr(k_new), code, _ptr(weights), _ptr(cache),
                                         num_pages, PAGE_SIZE, _ptr(block_table),
                                         block_table.stride(0), _ptr(context_lens), B, next_n, H,
                                         int(max_context_len), _ptr(logits), logits.stride(0),
                                         1 if clean else 0, _stream(stream)),
           "idx_logits_paged_insert")
    return logits


def logits_paged_insert_rope(q, k_new, weights, cache, block_table, context_lens, next_n,
                             max_context_len, cos, sin, rope_dim, mode="neox", positions=None,
                             logits=None, clean=True, stream=None):
    """logits_paged_insert with q rotated first (as quantize_rope; positions
    [B*next_n] int64, or None: each row at its token's position
    context_lens[b] - next_n + i).  Neox pairing takes rope_dim 64 or 128 here."""
    code, R, H, B, logits, num_pages = _paged_insert_args(
        q, k_new, weights, cache, block_table, context_lens, next_n, max_context_len, logits,
        clean)
    _check_rope_tables(cos, sin, rope_dim, positions, R)
    rope = _rope_block(cos, sin, rope_dim, mode, positions)
    _check(lib().idx_logits_paged_insert_rope(_ptr(q), _ptr(k_new), code, _ptr(weights),
                                              _ptr(cache), num_pages, PAGE_SIZE,
                                              _ptr(block_table), block_table.stride(0),
                                              _ptr(context_lens), B, next_n, H,
                                              int(max_context_len), _ptr(logits),
                                              logits.stride(0), 1 if clean else 0,
                                              ctypes.addressof(rope), _stream(stream)),
           "idx_logits_paged_insert_rope")
    return logits


def topk(logits, ks, ke, k, out=None, stream=None):
    """Per-row top-k column indices (int32 [rows, k], -1 padded)."""
    torch = _torch()
    _dev(logits, "logits", torch.float32)
    _dev(ke, "ke", torch.int32)
    if ks is not None:
        _dev(ks, "ks", torch.int32)
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise MxidxError("logits must be 2-D with contiguous rows")
    rows = logits.shape[0]
    if ke.numel() != rows or not ke.is_contiguous() or \
            (ks is not None and (ks.numel() != rows or not ks.is_contiguous())):
        raise MxidxError("ks / ke must hold one entry per row")
    if out is None:
        out = torch.empty((rows, k), dtype=torch.int32, device=logits.device)
    _dev(out, "out", torch.int32)
    if not out.is_contiguous() or tuple(out.shape) != (rows, k):
        raise MxidxError("out must be a contiguous int32 [rows, k]")
    _check(lib().idx_topk(_ptr(logits), rows, logits.stride(0), _ptr(ks), _ptr(ke), k, _ptr(out),
                          _stream(stream)), "idx_topk")
    return out


def topk_workspace_bytes(rows, row_stride):
    """Bytes of device workspace topk_ws needs for `rows` rows of stride `row_stride`
    (0 when it does not split rows)."""
    return int(lib().idx_topk_workspace_bytes(rows, row_stride))


def topk_workspace(rows, row_stride, device=None):
    """A uint8 workspace for topk_ws (uninitialized; reusable across calls in stream order)."""
    torch = _torch()
    n = topk_workspace_bytes(rows, row_stride)
    return torch.empty(max(n, 1), dtype=torch.uint8,
                       device=device if device is not None else torch.cuda.current_device())


def topk_ws(logits, ks, ke, k, workspace, out=None, stream=None):
    """topk with a device workspace (from topk_workspace): the same sets; few long rows
    are split over workgroups."""
    torch = _torch()
    _dev(logits, "logits", torch.float32)
    _dev(ke, "ke", torch.int32)
    _dev(workspace, "workspace", torch.uint8)
    if ks is not None:
        _dev(ks, "ks", torch.int32)
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise MxidxError("logits must be 2-D with contiguous rows")
    rows = logits.shape[0]
    if ke.numel() != rows or not ke.is_contiguous() or \
            (ks is not None and (ks.numel() != rows or not ks.is_contiguous())):
        raise MxidxError("ks / ke must hold one entry per row")
    if not workspace.is_contiguous():
        raise MxidxError("workspace must be contiguous")
    if out is None:
        out = torch.empty((rows, k), dtype=torch.int32, device=logits.device)
    _dev(out, "out", torch.int32)
    if not out.is_contiguous() or tuple(out.shape) != (rows, k):
        raise MxidxError("out must be a contiguous int32 [rows, k]")
    _check(lib().idx_topk_ws(_ptr(logits), rows, logits.stride(0), _ptr(ks), _ptr(ke), k, _ptr(out),
                             _ptr(workspace), workspace.numel(), _stream(stream)), "idx_topk_ws")
    return out


# ---------------------------------------------------------------------------
# FP8 (E4M3) indexer cache: 128 E4M3 values + an fp32 scale per row
# ---------------------------------------------------------------------------

def _fp8_cache_pages(cache):
    torch = _torch()
    _dev(cache, "cache", torch.uint8)
    if not cache.is_contiguous() or cache.numel() % (PAGE_SIZE * FP8_ROW_BYTES) != 0:
        raise MxidxError("cache must be a contiguous uint8 [num_pages, 64*132]")
    return cache.numel() // (PAGE_SIZE * FP8_ROW_BYTES)


def quantize_fp8(x, round_scale=False, weights=None, values=None, scales=None, weights_out=None,
                 stream=None):
    """FP8-encode rows of 128 values: returns (values u8 [..., 128], scales f32 [...]) and,
    with ``weights`` (one fp32 per row, e.g. [T, H] for q [T, H, 128]), also the folded
    weights w' = weights * scales as a third result."""
    torch = _torch()
    rows, stride, code = _rows_view(x, "x")
    lead = tuple(x.shape[:-1])
    if values is None:
        values = torch.empty(lead + (HEAD_DIM,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(lead, dtype=torch.float32, device=x.device)
    _dev(values, "values", torch.uint8)
    _dev(scales, "scales", torch.float32)
    if values.numel() != rows * HEAD_DIM or scales.numel() != rows or \
            not values.is_contiguous() or not scales.is_contiguous():
        raise MxidxError("values/scales must be contiguous [rows, 128] / [rows]")
    if weights is not None:
        _dev(weights, "weights", torch.float32)
        if weights.numel() != rows or not weights.is_contiguous():
            raise MxidxError("weights must be a contiguous fp32 tensor with one entry per row")
        if weights_out is None:
            weights_out = torch.empty_like(weights)
        _dev(weights_out, "weights_out", torch.float32)
        if weights_out.numel() != rows or not weights_out.is_contiguous():
            raise MxidxError("weights_out must be a contiguous fp32 tensor with one entry per row")
    fmt = FP8_SCALE_POW2 if round_scale else FP8_SCALE_F32
    _check(lib().idx_quantize_fp8(_ptr(x), code, rows, stride, fmt, _ptr(values), _ptr(scales),
                                  _ptr(weights), _ptr(weights_out), _stream(stream)),
           "idx_quantize_fp8")
    return (values, scales) if weights is None else (values, scales, weights_out)


def insert_fp8(k, slot_mapping, cache, round_scale=False, stream=None):
    """FP8-encode K rows [N, 128] into ``cache`` [num_pages, 64*132] (in place)."""
    torch = _torch()
    rows, stride, code = _rows_view(k, "k")
    _dev(slot_mapping, "slot_mapping", torch.int64)
    if slot_mapping.numel() != rows or not slot_mapping.is_contiguous():
        raise MxidxError("slot_mapping must be a contiguous int64 [N]")
    num_pages = _fp8_cache_pages(cache)
    fmt = FP8_SCALE_POW2 if round_scale else FP8_SCALE_F32
    _check(lib().idx_insert_fp8(_ptr(k), code, rows, stride, fmt, _ptr(slot_mapping), _ptr(cache),
                                num_pages, PAGE_SIZE, _stream(stream)), "idx_insert_fp8")
    return cache


def gather_fp8(cache, block_table, seq_lens, cu_seq_offsets, max_seq_len, total_tokens,
               k_values=None, k_scales=None, stream=None):
    """FP8 paged cache -> contiguous (k_values u8 [total, 128], k_scales f32 [total])."""
    torch = _torch()
    num_pages = _fp8_cache_pages(cache)
    _dev(block_table, "block_table", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(cu_seq_offsets, "cu_seq_offsets", torch.int64)
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise MxidxError("block_table must be [batch, pages] with unit inner stride")
    batch = block_table.shape[0]
    if seq_lens.numel() != batch or cu_seq_offsets.numel() != batch:
        raise MxidxError("seq_lens / cu_seq_offsets must have one entry per sequence")
    if block_table.shape[1] * PAGE_SIZE < max_seq_len:
        raise MxidxError("block_table has fewer pages than max_seq_len needs")
    if k_values is None:
        k_values = torch.zeros((total_tokens, HEAD_DIM), dtype=torch.uint8, device=cache.device)
    if k_scales is None:
        k_scales = torch.zeros((total_tokens,), dtype=torch.float32, device=cache.device)
    _dev(k_values, "k_values", torch.uint8)
    _dev(k_scales, "k_scales", torch.float32)
    if not k_values.is_contiguous() or k_values.numel() < total_tokens * HEAD_DIM or \
            not k_scales.is_contiguous() or k_scales.numel() < total_tokens:
        raise MxidxError("k_values / k_scales must be contiguous [total, 128] uint8 / [total] fp32")
    _check(lib().idx_gather_fp8(_ptr(cache), num_pages, PAGE_SIZE, _ptr(block_table),
                                block_table.stride(0), _ptr(seq_lens), _ptr(cu_seq_offsets), batch,
                                int(max_seq_len), int(total_tokens), _ptr(k_values), _ptr(k_scales),
                                _stream(stream)), "idx_gather_fp8")
    return k_values, k_scales


def logits_prefill_fp8(q_values, weights, k_values, k_scales, ks, ke, logits=None, clean=True,
                       stream=None):
    """Dense FP8 logits [T, S]: q_values u8 [T, H, 128], weights f32 [T, H] (the folded w'),
    k_values u8 [S, 128], k_scales f32 [S]."""
    torch = _torch()
    T, H = q_values.shape[0], q_values.shape[1]
    S = k_values.shape[0]
    for name, t, dt in (("q_values", q_values, torch.uint8), ("weights", weights, torch.float32),
                        ("k_values", k_values, torch.uint8), ("k_scales", k_scales, torch.float32),
                        ("ke", ke, torch.int32)):
        _dev(t, name, dt)
        if not t.is_contiguous():
            raise MxidxError(f"{name} must be contiguous")
    if ks is not None:
        _dev(ks, "ks", torch.int32)
    if tuple(q_values.shape) != (T, H, HEAD_DIM) or tuple(weights.shape) != (T, H) or \
            tuple(k_values.shape) != (S, HEAD_DIM) or tuple(k_scales.shape) != (S,):
        raise MxidxError("shape mismatch among q/k/weights")
    if ke.numel() != T or (ks is not None and (ks.numel() != T or not ks.is_contiguous())):
        raise MxidxError("ks / ke must hold one entry per query row")
    if logits is None:
        fill = float("-inf") if clean else 0.0
        logits = torch.full((T, S), fill, dtype=torch.float32, device=q_values.device)
    _dev(logits, "logits", torch.float32)
    if logits.dim() != 2 or logits.stride(1) != 1 or logits.shape[0] < T or logits.shape[1] < S:
        raise MxidxError("logits must be [>=T, >=S] with contiguous rows")
    _check(lib().idx_logits_prefill_fp8(_ptr(q_values), _ptr(weights), _ptr(k_values),
                                        _ptr(k_scales), _ptr(ks), _ptr(ke), T, H, S, _ptr(logits),
                                        logits.stride(0), 1 if clean else 0, _stream(stream)),
           "idx_logits_prefill_fp8")
    return logits


def logits_paged_fp8(q_values, weights, cache, block_table, context_lens, next_n,
                     max_context_len, logits=None, clean=True, stream=None):
    """Paged FP8 decode logits [B*next_n, max_context_len]: q_values u8 [B*next_n, H, 128],
    weights f32 [B*next_n, H] (the folded w')."""
    torch = _torch()
    R, H = q_values.shape[0], q_values.shape[1]
    B = context_lens.numel()
    num_pages = _fp8_cache_pages(cache)
    for name, t, dt in (("q_values", q_values, torch.uint8), ("weights", weights, torch.float32),
                        ("block_table", block_table, torch.int32),
                        ("context_lens", context_lens, torch.int32)):
        _dev(t, name, dt)
    if R != B * next_n:
        raise MxidxError("q rows must be batch * next_n")
    for name, t in (("q_values", q_values), ("weights", weights), ("context_lens", context_lens)):
        if not t.is_contiguous():
            raise MxidxError(f"{name} must be contiguous")
    if tuple(q_values.shape) != (R, H, HEAD_DIM) or tuple(weights.shape) != (R, H):
        raise MxidxError("shape mismatch among q/weights")
    if block_table.dim() != 2 or block_table.stride(1) != 1 or block_table.shape[0] != B:
        raise MxidxError("block_table must be [batch, pages] with unit inner stride")
    if block_table.shape[1] * PAGE_SIZE < max_context_len:
        raise MxidxError("block_table has fewer pages than max_context_len needs")
    if logits is None:
        fill = float("-inf") if clean else 0.0
        logits = torch.full((R, max_context_len), fill, dtype=torch.float32, device=q_values.device)
    _dev(logits, "logits", torch.float32)
    if logits.dim() != 2 or logits.stride(1) != 1 or logits.shape[0] < R or \
            logits.shape[1] < max_context_len:
        raise MxidxError("logits must be [>=rows, >=max_context_len] with contiguous rows")
    _check(lib().idx_logits_paged_fp8(_ptr(q_values), _ptr(weights), _ptr(cache), num_pages,
                                      PAGE_SIZE, _ptr(block_table), block_table.stride(0),
                                      _ptr(context_lens), B, next_n, H, int(max_context_len),
                                      _ptr(logits), logits.stride(0), 1 if clean else 0,
                                      _stream(stream)), "idx_logits_paged_fp8")
    return logits


def logits_paged_insert_fp8(q, k_new, weights, cache, block_table, context_lens, next_n,
                            max_context_len, round_scale=False, logits=None, clean=True,
                            stream=None):
    """The FP8 decode step in one launch: the new tokens' K (k_new [B*next_n, 128])
    into their block-table slots of the FP8 cache, q [B*next_n, H, 128] encoded to
    E4M3 with its scales folded into the weights (weights [B*next_n, H], not
    folded), and the decode logits (as insert_fp8 + quantize_fp8 + logits_paged_fp8)."""
    code, R, H, B, logits, _ = _paged_insert_args(
        q, k_new, weights, cache, block_table, context_lens, next_n, max_context_len, logits,
        clean)
    num_pages = _fp8_cache_pages(cache)
    fmt = FP8_SCALE_POW2 if round_scale else FP8_SCALE_F32
    _check(lib().idx_logits_paged_insert_fp8(_ptr(q), _ptr(k_new), code, _ptr(weights), fmt,
                                             _ptr(cache), num_pages, PAGE_SIZE,
                                             _ptr(block_table), block_table.stride(0),
                                             _ptr(context_lens), B, next_n, H,
                                             int(max_context_len), _ptr(logits),
                                             logits.stride(0), 1 if clean else 0,
                                             _stream(stream)), "idx_logits_paged_insert_fp8")
    return logits


def kpool_insert(k, gate_score, ape, slot_mapping, cache, kpool, fmt="mxfp4", round_scale=False,
                 return_compressed=False, stream=None):
    """Pool kpool consecutive tokens of k [n, 128] (softmax over gate_score [n, 128] +
    ape [kpool, 128] per dimension) and write the pooled rows of the pool-end
    positions (slot >= 0, position >= kpool - 1) into ``cache`` (MXFP4
    [pages, 64*68] or, with fmt="fp8", [pages, 64*132]).  With
    return_compressed, also returns the fp32 pooled rows [n, 128] (rows of
    unwritten positions are zero)."""
    torch = _torch()
    n, stride, code = _rows_view(k, "k")
    _dev(gate_score, "gate_score", torch.float32)
    _dev(ape, "ape", torch.float32)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    _dev(cache, "cache", torch.uint8)
    if gate_score.shape != (n, HEAD_DIM) or not gate_score.is_contiguous():
        raise MxidxError("gate_score must be a contiguous fp32 [n, 128]")
    if ape.shape != (kpool, HEAD_DIM) or not ape.is_contiguous():
        raise MxidxError("ape must be a contiguous fp32 [kpool, 128]")
    if slot_mapping.numel() != n or not slot_mapping.is_contiguous():
        raise MxidxError("slot_mapping must be a contiguous int64 [n]")
    row = {"mxfp4": ROW_BYTES, "fp8": FP8_ROW_BYTES}[fmt]
    if not cache.is_contiguous() or cache.numel() % (PAGE_SIZE * row) != 0:
        raise MxidxError(f"cache must be a contiguous uint8 [num_pages, 64*{row}]")
    comp = torch.zeros((n, HEAD_DIM), dtype=torch.float32, device=k.device) if return_compressed else None
    _check(lib().idx_kpool_insert(_ptr(k), code, n, stride, _ptr(gate_score), _ptr(ape),
                                  _ptr(slot_mapping), kpool, 0 if fmt == "mxfp4" else 1,
                                  FP8_SCALE_POW2 if round_scale else FP8_SCALE_F32, _ptr(cache),
                                  cache.numel() // (PAGE_SIZE * row), PAGE_SIZE, _ptr(comp),
                                  _stream(stream)), "idx_kpool_insert")
    return (cache, comp) if return_compressed else cache


def topk_noalloc(logits, ks, ke, k, out=None, stream=None):
    """topk_ws with the library's static device scratch instead of a caller's
    workspace (no device allocation by the library; `out` is allocated here only
    when it is not given).  Raises when the call needs more than
    TOPK_NOALLOC_MAX_WORKSPACE bytes of workspace."""
    torch = _torch()
    _dev(logits, "logits", torch.float32)
    _dev(ke, "ke", torch.int32)
    if ks is not None:
        _dev(ks, "ks", torch.int32)
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise MxidxError("logits must be 2-D with contiguous rows")
    rows = logits.shape[0]
    if ke.numel() != rows or not ke.is_contiguous() or \
            (ks is not None and (ks.numel() != rows or not ks.is_contiguous())):
        raise MxidxError("ks / ke must hold one entry per row")
    if out is None:
        out = torch.empty((rows, k), dtype=torch.int32, device=logits.device)
    _dev(out, "out", torch.int32)
    if not out.is_contiguous() or tuple(out.shape) != (rows, k):
        raise MxidxError("out must be a contiguous int32 [rows, k]")
    _check(lib().idx_topk_noalloc(_ptr(logits), rows, logits.stride(0), _ptr(ks), _ptr(ke), k,
                                  _ptr(out), _stream(stream)), "idx_topk_noalloc")
    return out


def topk_merge(values, indices, interleave, k, out=None, stream=None):
    """Merge per-rank top-k lists (values f32 / indices i32 [world, rows, k_in], local
    positions, -1 empty) into global top-k positions [rows, k] (-1 padded)."""
    torch = _torch()
    _dev(values, "values", torch.float32)
    _dev(indices, "indices", torch.int32)
    if values.dim() != 3 or values.shape != indices.shape:
        raise MxidxError("values and indices must both be [world, rows, k_in]")
    if not values.is_contiguous() or not indices.is_contiguous():
        raise MxidxError("values and indices must be contiguous")
    world, rows, k_in = values.shape
    if out is None:
        out = torch.empty((rows, k), dtype=torch.int32, device=values.device)
    _dev(out, "out", torch.int32)
    if out.shape != (rows, k) or not out.is_contiguous():
        raise MxidxError("out must be a contiguous int32 [rows, k]")
    _check(lib().idx_topk_merge(_ptr(values), _ptr(indices), world, rows, k_in, interleave, k,
                                _ptr(out), _stream(stream)), "idx_topk_merge")
    return out


# ---------------------------------------------------------------------------
# a serving step around the indexer
# ---------------------------------------------------------------------------

_NORMS = {"none": 0, "rms": 1, "layer": 2}
_MODES = {"neox": ROPE_NEOX, "interleaved": ROPE_INTERLEAVED}
_COLUMNS = {"sequence": 0, "gathered": 1}


def _code(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise MxidxError(f"{name} must be one of {sorted(table)}, got {value!r}") from None


def _on(device, t, name, dtype, shape=None):
    """The address of t: a tensor of that type on that device, contiguous with that shape where
    one is given."""
    if t.get_device() == device.index and t.dtype is dtype and \
            (shape is None or (t.shape == shape and t.is_contiguous())):
        return t.data_ptr()
    if t.device != device:
        raise MxidxError(f"{name} must be a device tensor on {device}, got {t.device}")
    if t.dtype is not dtype:
        raise MxidxError(f"{name} must be {dtype}, got {t.dtype}")
    raise MxidxError(f"{name} must be contiguous of shape {shape}, got {tuple(t.shape)}")


_PACKED = {}


def _packed(name):
    """(number, packer of the arguments' 8-byte words, their count) of a call."""
    words = "".join("d" if t in (_float, _double) else "q" for t in EXPORTS[name][1])
    _PACKED[name] = lib().idx_entry(name.encode()), struct.Struct("=" + words).pack, len(words)
    return _PACKED[name]


def _call(name, device, stream, *args):
    """One call of the library with `device` current, on `stream` (None: that device's
    current stream).  Null pointers are 0; the arguments go over packed (idx_call): one by one their
    conversion takes as long as the launch."""
    torch = _torch()
    index = device.index
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device != device:
        raise MxidxError(f"{name}: the stream belongs to {stream.device}, the tensors to {device}")
    else:
        raw = stream.cuda_stream
    entry, pack, count = _PACKED.get(name) or _packed(name)
    try:
        words = pack(*args, raw)
    except struct.error as e:
        raise MxidxError(f"{name}: {e}") from None
    call = _LIB.idx_call
    if torch._C._cuda_getDevice() == index:
        status = call(entry, words, count)
    else:
        with torch.cuda.device(device):
            status = call(entry, words, count)
    if status != 0:
        _check(status, name)


def _empty(stream, shape, dtype, device, fill=None):
    """A new tensor, filled with a number where one is given, whose memory belongs to the call's stream."""
    torch = _torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return _empty(None, shape, dtype, device, fill)
    if fill is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return torch.full(shape, fill, dtype=dtype, device=device)


def _device_of(t, name):
    if not t.is_cuda:
        raise MxidxError(f"{name} must be a device tensor")
    return t.device


def _rope_args(device, cos, sin, rope_dim, mode, positions, tokens):
    """The checked idx_rope block of a call on `device` (host memory; the tensors must outlive it)."""
    torch = _torch()
    rope_dim = int(rope_dim)
    table = (cos.shape[0], rope_dim // 2)
    cp = _on(device, cos, "cos", torch.float32, table)
    sp = _on(device, sin, "sin", torch.float32, table)
    pp = 0 if positions is None else _on(device, positions, "positions", torch.int64, (tokens,))
    return _Rope(cp, sp, table[0], pp, rope_dim, _code(_MODES, mode, "mode"))


StepMap = collections.namedtuple("StepMap", ["slot_mapping", "positions", "row_seq", "ks", "ke",
                                             "cu_seq_offsets", "free_next"])


def step_map(seq_lens, query_lens, block_table, num_rows, free_pages=None, free_start=None,
             free_next=None, columns="sequence", slot_mapping=None, positions=None, row_seq=None,
             ks=None, ke=None, cu_seq_offsets=None, stream=None):
    """A step's bookkeeping from its request lengths, in one launch: returns StepMap.

    seq_lens / query_lens i32 [B]: each request's tokens and how many of them are new; the step's
    rows are the new tokens in order, padded to ``num_rows``.  With ``free_pages`` (i32) and
    ``free_start`` (i64 [1]) the pages that the step enters are taken from that list and
    written into ``block_table`` [B, pages]; ``free_next`` (i64 [1]) says where the list
    goes on.  ``columns``: "sequence" (paged logits) or "gathered" (rows of gather / dense
    logits).  Padding rows get slot -1, position 0, sequence -1 and an empty window."""
    torch = _torch()
    device = _device_of(seq_lens, "seq_lens")
    i32, i64 = torch.int32, torch.int64
    B, rows = seq_lens.numel(), int(num_rows)
    if rows < 0:
        raise MxidxError("num_rows must not be negative")
    sp = _on(device, seq_lens, "seq_lens", i32, (B,))
    qp = _on(device, query_lens, "query_lens", i32, (B,))
    bp = _on(device, block_table, "block_table", i32)
    shape, strides = block_table.shape, block_table.stride()
    if len(shape) != 2 or shape[0] != B or (shape[1] > 1 and strides[1] != 1 and B):
        raise MxidxError("block_table must be [B, pages] with unit inner stride")
    pages = shape[1]
    stride = strides[0] if B > 1 else max(pages, 1)
    fp = ip = 0
    free = 0
    if free_pages is not None:
        if free_start is None:
            raise MxidxError("free_pages needs free_start")
        free = free_pages.numel()
        ip = _on(device, free_start, "free_start", i64, (1,))
        # an empty list has no address of its own, and is still a list
        fp = _on(device, free_pages, "free_pages", i32, (free,)) or ip
    elif free_start is not None:
        raise MxidxError("free_start needs free_pages")

    if slot_mapping is None:
        slot_mapping = _empty(stream, rows, i64, device)
    if positions is None:
        positions = _empty(stream, rows, i64, device)
    if row_seq is None:
        row_seq = _empty(stream, rows, i32, device)
    if ks is None:
        ks = _empty(stream, rows, i32, device)
    if ke is None:
        ke = _empty(stream, rows, i32, device)
    if cu_seq_offsets is None:
        cu_seq_offsets = _empty(stream, B + 1, i64, device)
    if free_next is None:
        free_next = _empty(stream, 1, i64, device)
    n = (rows,)
    _call("idx_step_map", device, stream, sp, qp, B, bp, stride, pages, fp, free, ip,
          _on(device, free_next, "free_next", i64, (1,)), PAGE_SIZE,
          _code(_COLUMNS, columns, "columns"), rows, _on(device, slot_mapping, "slot_mapping", i64, n),
          _on(device, positions, "positions", i64, n), _on(device, row_seq, "row_seq", i32, n),
          _on(device, ks, "ks", i32, n), _on(device, ke, "ke", i32, n),
          _on(device, cu_seq_offsets, "cu_seq_offsets", i64, (B + 1,)))
    return StepMap(slot_mapping, positions, row_seq, ks, ke, cu_seq_offsets, free_next)


def _heads_block(device, stream, x, out, norm, weight, bias, eps, name, tokens, dtype):
    """(idx_heads block, out) of x [T, H, 128] or [T, 128]."""
    shape, strides = x.shape, x.stride()
    xp = _on(device, x, name, dtype)
    if len(shape) not in (2, 3) or shape[-1] != HEAD_DIM or shape[0] != tokens:
        raise MxidxError(f"{name} must be [{tokens}, H, {HEAD_DIM}] or [{tokens}, {HEAD_DIM}]")
    if out is None:
        out = _empty(stream, shape, dtype, device)
    op = _on(device, out, f"{name}_out", dtype)
    if out.shape != shape:
        raise MxidxError(f"{name}_out must have {name}'s shape")
    out_strides = out.stride()
    heads = shape[1] if len(shape) == 3 else 1
    if tokens and heads:
        if strides[-1] != 1 or out_strides[-1] != 1:
            raise MxidxError(f"{name} and {name}_out must have a contiguous last dim")
        if op == xp and out_strides != strides:
            raise MxidxError(f"{name}_out may be {name} itself only with the same strides")
    wp = 0 if weight is None else _on(device, weight, f"{name}_weight", _torch().float32, (HEAD_DIM,))
    bp = 0 if bias is None else _on(device, bias, f"{name}_bias", _torch().float32, (HEAD_DIM,))
    return _Heads(xp, op, strides[0], strides[1] if len(shape) == 3 else HEAD_DIM, out_strides[0],
                  out_strides[1] if len(shape) == 3 else HEAD_DIM, heads,
                  _code(_NORMS, norm, f"{name}_norm"), wp, bp, eps), out


def norm_rope(q, k, cos, sin, rope_dim, mode="neox", positions=None, q_norm="none", q_weight=None,
              q_bias=None, k_norm="layer", k_weight=None, k_bias=None, eps=1e-6, q_out=None,
              k_out=None, stream=None):
    """Per-head norm ("none", "rms", "layer"; fp32 weight / bias [128] or None) and RoPE on the
    first ``rope_dim`` dims of the indexer's rows, in one launch: q [T, H, 128] and k
    [T, 128] or [T, Hk, 128], bf16 or fp32, either of them None; cos / sin / positions /
    mode as for quantize_rope.  Returns (q_out, k_out), of the inputs' type; an output may
    be its input."""
    first = q if q is not None else k
    if first is None:
        raise MxidxError("norm_rope needs q or k")
    torch = _torch()
    device = _device_of(first, "q" if q is not None else "k")
    dtype = first.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise MxidxError("q and k must be bfloat16 or float32")
    T = first.shape[0]
    rope = _rope_args(device, cos, sin, rope_dim, mode, positions, T)
    qb = kb = None
    if q is not None:
        qb, q_out = _heads_block(device, stream, q, q_out, q_norm, q_weight, q_bias, eps, "q", T, dtype)
    if k is not None:
        kb, k_out = _heads_block(device, stream, k, k_out, k_norm, k_weight, k_bias, eps, "k", T, dtype)
    _call("idx_norm_rope", device, stream, 0 if qb is None else ctypes.addressof(qb),
          0 if kb is None else ctypes.addressof(kb), IDX_BF16 if dtype == torch.bfloat16 else IDX_F32,
          T, ctypes.addressof(rope))
    return (None if q is None else q_out), (None if k is None else k_out)


def _latent_cache(device, cache):
    """(address, num_pages, latent) of a latent cache."""
    torch = _torch()
    cp = _on(device, cache, "cache", torch.bfloat16)
    shape = cache.shape
    if len(shape) != 3 or shape[1] != PAGE_SIZE or not cache.is_contiguous() or \
            shape[2] - LATENT_ROPE not in LATENT_DIMS:
        raise MxidxError("cache must be a contiguous bfloat16 [num_pages, 64, latent + 64], latent "
                         f"one of {LATENT_DIMS}")
    return cp, shape[0], shape[2] - LATENT_ROPE


def _latent_insert(call, cache_of, kv, slot_mapping, cache, cos, sin, mode, positions, norm, weight,
                   eps, q_pe, q_out, stream):
    """The checked call of idx_latent_insert or idx_latent_insert_mxfp4."""
    torch = _torch()
    device = _device_of(kv, "kv")
    dtype = kv.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise MxidxError("kv must be bfloat16 or float32")
    cp, num_pages, latent = cache_of(device, cache)
    shape, kv_strides = kv.shape, kv.stride()
    if len(shape) != 2 or shape[1] != latent + LATENT_ROPE or (shape[0] and kv_strides[1] != 1):
        raise MxidxError(f"kv must be [T, {latent + LATENT_ROPE}] with a contiguous last dim")
    T = shape[0]
    mp = _on(device, slot_mapping, "slot_mapping", torch.int64, (T,))
    wp = 0 if weight is None else _on(device, weight, "weight", torch.float32, (latent,))
    rope = _rope_args(device, cos, sin, LATENT_ROPE, mode, positions, T)
    qp = op = 0
    H = qs = qh = os_ = oh = 0
    if q_pe is not None:
        qp = _on(device, q_pe, "q_pe", dtype)
        shape = q_pe.shape
        if len(shape) != 3 or shape[0] != T or shape[2] != LATENT_ROPE:
            raise MxidxError(f"q_pe must be [{T}, H, {LATENT_ROPE}]")
        H = shape[1]
        if q_out is None:
            q_out = _empty(stream, shape, torch.bfloat16, device)
        op = _on(device, q_out, "q_out", torch.bfloat16)
        if q_out.shape != shape:
            raise MxidxError("q_out must have q_pe's shape")
        (qs, qh, qi), (os_, oh, oi) = q_pe.stride(), q_out.stride()
        if T and H and (qi != 1 or oi != 1):
            raise MxidxError("q_pe and q_out must have a contiguous last dim")
    elif q_out is not None:
        raise MxidxError("q_out needs q_pe")
    _call(call, device, stream, kv.data_ptr(),
          IDX_BF16 if dtype == torch.bfloat16 else IDX_F32, T, kv_strides[0], latent,
          _code({"none": 0, "rms": 1}, norm, "norm"), wp, eps, ctypes.addressof(rope), mp, cp,
          num_pages, PAGE_SIZE, qp, H, qs, qh, op, os_, oh)
    return cache if q_pe is None else (cache, q_out)


def latent_insert(kv, slot_mapping, cache, cos, sin, mode="neox", positions=None, norm="rms",
                  weight=None, eps=1e-6, q_pe=None, q_out=None, stream=None):
    """Latent rows kv [T, latent + 64] (bf16 / fp32) into the latent cache [num_pages, 64,
    latent + 64] bf16: the latent part RMS-normed (``norm`` "rms", fp32 ``weight`` [latent] or
    None; or "none"), the last 64 values rotated (cos / sin fp32 [table_rows, 32]), slots < 0
    skipped.  ``q_pe`` [T, H, 64]: the query's positional part, rotated into ``q_out``
    [T, H, 64] bf16 (``q[..., latent:]`` of attn_paged's query, say; q_pe itself if that is
    bf16) in the same launch.  Returns cache, or (cache, q_out) with q_pe."""
    return _latent_insert("idx_latent_insert", _latent_cache, kv, slot_mapping, cache, cos, sin, mode,
                          positions, norm, weight, eps, q_pe, q_out, stream)


def latent_mxfp4_row_bytes(latent):
    """Bytes of a token in the MXFP4 latent cache: codes, scales and 64 bf16 values."""
    return latent // 2 + latent // 32 + 2 * LATENT_ROPE


_LATENT_OF_PAGE = {PAGE_SIZE * latent_mxfp4_row_bytes(n): n for n in LATENT_DIMS}


def _latent_mxfp4_cache(device, cache):
    """(address, num_pages, latent) of an MXFP4 latent cache."""
    cp = _on(device, cache, "cache", _torch().uint8)
    shape = cache.shape
    latent = _LATENT_OF_PAGE.get(shape[1]) if len(shape) == 2 else None
    if latent is None or not cache.is_contiguous():
        raise MxidxError("cache must be a contiguous uint8 [num_pages, 64 * latent_mxfp4_row_bytes(latent)], "
                         f"latent one of {LATENT_DIMS}")
    return cp, shape[0], latent


def latent_insert_mxfp4(kv, slot_mapping, cache, cos, sin, mode="neox", positions=None, norm="rms",
                        weight=None, eps=1e-6, q_pe=None, q_out=None, stream=None):
    """latent_insert into the MXFP4 latent cache (uint8 [num_pages, 64 * latent_mxfp4_row_bytes(latent)]):
    the latent part normed in 64 bits and written as MXFP4 codes and scales, the last 64 values
    rotated and kept in bf16.  Arguments, query rows and result as latent_insert's."""
    return _latent_insert("idx_latent_insert_mxfp4", _latent_mxfp4_cache, kv, slot_mapping, cache, cos, sin,
                          mode, positions, norm, weight, eps, q_pe, q_out, stream)


def latent_gather_mxfp4(cache, block_table, seq_lens, cu_seq_offsets, max_seq_len, total_tokens, out=None,
                        stream=None):
    """MXFP4 latent cache -> contiguous bf16 rows [total_tokens, latent + 64], exact: token j of sequence b
    (block_table i32 [B, pages], seq_lens i32 [B]) to row cu_seq_offsets[b] + j (i64, at least B of them:
    step_map's B + 1 will do).  Rows that no token maps to are zeros in a new ``out`` and stay as
    they were in a given one."""
    torch = _torch()
    device = _device_of(cache, "cache")
    cp, num_pages, latent = _latent_mxfp4_cache(device, cache)
    bp = _on(device, block_table, "block_table", torch.int32)
    shape, strides = block_table.shape, block_table.stride()
    if len(shape) != 2 or (shape[1] > 1 and strides[1] != 1 and shape[0]):
        raise MxidxError("block_table must be [B, pages] with unit inner stride")
    B, pages = shape
    if max_seq_len > pages * PAGE_SIZE:
        raise MxidxError("block_table has fewer pages than max_seq_len needs")
    stride = strides[0] if B > 1 else max(pages, 1)
    sp = _on(device, seq_lens, "seq_lens", torch.int32, (B,))
    op = _on(device, cu_seq_offsets, "cu_seq_offsets", torch.int64)
    shape = cu_seq_offsets.shape
    if len(shape) != 1 or shape[0] < B or not cu_seq_offsets.is_contiguous():
        raise MxidxError(f"cu_seq_offsets must be a contiguous int64 of {B} offsets or more")
    width = latent + LATENT_ROPE
    if total_tokens < 0:
        raise MxidxError("total_tokens must not be negative")
    if out is None:
        out = _empty(stream, (total_tokens, width), torch.bfloat16, device, fill=0)
    rp = _on(device, out, "out", torch.bfloat16)
    shape, strides = out.shape, out.stride()
    if len(shape) != 2 or shape[0] < total_tokens or shape[1] != width or (strides[1] != 1 and total_tokens):
        raise MxidxError(f"out must be [{total_tokens}, {width}] with a contiguous last dim")
    _call("idx_latent_gather_mxfp4", device, stream, cp, num_pages, PAGE_SIZE, latent, bp, stride, sp, op,
          B, max_seq_len, total_tokens, rp, strides[0])
    return out


def attn_workspace_bytes(rows, heads, latent, entries, mxfp4=False):
    """Workspace bytes of attn_paged, or of attn_paged_mxfp4; entries: k with indices, else max_tokens
    (0: no workspace).  Fewer rows, heads or entries may need more."""
    if mxfp4:
        return int(lib().idx_attn_workspace_bytes_mxfp4(rows, heads, latent, entries))
    return int(lib().idx_attn_workspace_bytes(rows, heads, latent, entries))


def attn_workspace_max_bytes(rows, heads, latent, entries):
    """Workspace bytes that are enough for attn_paged calls with up to so many rows, heads and entries."""
    return int(lib().idx_attn_workspace_max_bytes(rows, heads, latent, entries))


def attn_workspace(rows, heads, latent, entries, device="cuda"):
    """A workspace for attn_paged calls with up to so many rows, heads and entries: reusable, not by
    calls that may run at the same time."""
    torch = _torch()
    return torch.empty(max(attn_workspace_max_bytes(rows, heads, latent, entries), 1),
                       dtype=torch.uint8, device=device)


def _attn_paged(call, cache_of, q, cache, block_table, ke, scale, indices, ks, row_seq, max_tokens, out, lse,
                workspace, stream):
    """The checked call of idx_attn_paged or idx_attn_paged_mxfp4."""
    torch = _torch()
    device = _device_of(q, "q")
    cp, num_pages, latent = cache_of(device, cache)
    bf16, i32 = torch.bfloat16, torch.int32
    qp = _on(device, q, "q", bf16)
    shape, q_strides = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != latent + LATENT_ROPE or (q_strides[2] != 1 and q.numel()):
        raise MxidxError(f"q must be [rows, H, {latent + LATENT_ROPE}] with a contiguous last dim")
    rows, H = shape[0], shape[1]
    bp = _on(device, block_table, "block_table", i32)
    shape, strides = block_table.shape, block_table.stride()
    if len(shape) != 2 or (shape[1] > 1 and strides[1] != 1 and shape[0]):
        raise MxidxError("block_table must be [B, pages] with unit inner stride")
    B, pages = shape
    stride = strides[0] if B > 1 else max(pages, 1)
    if max_tokens is None:
        max_tokens = pages * PAGE_SIZE
    elif max_tokens > pages * PAGE_SIZE:
        raise MxidxError("block_table has fewer pages than max_tokens needs")
    ep = _on(device, ke, "ke", i32, (rows,))
    kp = 0 if ks is None else _on(device, ks, "ks", i32, (rows,))
    rp = 0 if row_seq is None else _on(device, row_seq, "row_seq", i32, (rows,))
    ip, istride, k = 0, 0, 0
    if indices is not None:
        ip = _on(device, indices, "indices", i32)
        shape, strides = indices.shape, indices.stride()
        if len(shape) != 2 or shape[0] != rows or (shape[1] > 1 and strides[1] != 1 and rows):
            raise MxidxError("indices must be [rows, k] with unit inner stride")
        k, istride = shape[1], strides[0]
        if k > 0x7fffffff:
            raise MxidxError("indices has too many columns")
        ip = ip or ep      # a list of no columns has no address of its own, and is still a list
    if out is None:
        out = _empty(stream, (rows, H, latent), bf16, device)
    op = _on(device, out, "out", bf16)
    strides = out.stride()
    if out.shape != (rows, H, latent) or (strides[2] != 1 and rows and H):
        raise MxidxError(f"out must be [{rows}, {H}, {latent}] with a contiguous last dim")
    if lse is None:
        lse = _empty(stream, (rows, H), torch.float32, device)
    lp = _on(device, lse, "lse", torch.float32, (rows, H))
    wp, wb = 0, 0
    if workspace is None:
        need = attn_workspace_bytes(rows, H, latent, k if indices is not None else max_tokens,
                                    call == "idx_attn_paged_mxfp4")
        if need:
            workspace = _empty(stream, need, torch.uint8, device)
    if workspace is not None:
        wp, wb = _on(device, workspace, "workspace", torch.uint8), workspace.numel()
        if not workspace.is_contiguous():      # an expanded view has less memory than numel
            raise MxidxError("workspace must be contiguous")
    _call(call, device, stream, qp, q_strides[0], q_strides[1], rows, H, latent, cp,
          num_pages, PAGE_SIZE, bp, stride, B, rp, kp, ep, ip, istride, k, max_tokens, scale, op,
          strides[0], strides[1], lp, wp, wb)
    return out, lse


def attn_paged(q, cache, block_table, ke, scale, indices=None, ks=None, row_seq=None,
               max_tokens=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of query rows q [rows, H, latent + 64] (bf16) over the latent cache: returns
    (out bf16 [rows, H, latent], lse fp32 [rows, H]).

    Row r sees its sequence's tokens 0 .. ke[r] - ks[r] - 1 (ks None: 0), all of them or those
    of ``indices`` (int32 [rows, k] columns in [ks, ke), topk's output; -1 skipped).
    ``row_seq`` i32 [rows]: the row's sequence (None: rows / B rows each, in order); rows of no
    sequence stay as they are.  ``max_tokens`` bounds ke - ks (None: what block_table holds).
    ``workspace``: attn_workspace's, allocated here when it is not given."""
    return _attn_paged("idx_attn_paged", _latent_cache, q, cache, block_table, ke, scale, indices, ks, row_seq,
                       max_tokens, out, lse, workspace, stream)


def attn_paged_mxfp4(q, cache, block_table, ke, scale, indices=None, ks=None, row_seq=None,
                     max_tokens=None, out=None, lse=None, workspace=None, stream=None):
    """attn_paged over the MXFP4 latent cache (uint8 [num_pages, 64 * latent_mxfp4_row_bytes(latent)]):
    the same arguments, workspace (attn_workspace's) and results."""
    return _attn_paged("idx_attn_paged_mxfp4", _latent_mxfp4_cache, q, cache, block_table, ke, scale, indices, ks,
                       row_seq, max_tokens, out, lse, workspace, stream)


def attn_prompt_workspace_bytes(rows, heads, kv_heads, dk, dv, seqs, max_seq_len):
    """Workspace bytes of attn_prompt (0: none); PROMPT_MAX_WORKSPACE are enough for every call."""
    return int(lib().idx_attn_prompt_workspace_bytes(rows, heads, kv_heads, dk, dv, seqs, max_seq_len))


def attn_prompt_workspace(device="cuda"):
    """A workspace for every attn_prompt call: reusable, not by calls that may run at the same time."""
    return _torch().empty(PROMPT_MAX_WORKSPACE, dtype=_torch().uint8, device=device)


def attn_prompt(q, k, v, seq_lens, query_lens, scale, causal=True, max_seq_len=None, out=None, lse=None,
                workspace=None, stream=None):
    """Attention of packed requests over contiguous keys and values: q [T, Hq, dk], k [S, Hk, dk],
    v [S, Hk, dv] (bf16, (dk, dv) one of PROMPT_DIMS, Hq a multiple of Hk, up to 256): returns (out bf16
    [T, Hq, dv], lse fp32 [T, Hq]).

    seq_lens / query_lens i32 [B], B up to 1024, as step_map's: request b's seq_lens[b] tokens follow the requests'
    before it in k and v, the last query_lens[b] of them are its rows in q.  ``causal``: a row
    sees the tokens up to its own (else all of its request's).  Rows behind the last request's
    are zeros (lse -inf) in a new out and stay as they were in a given one.  ``max_seq_len``
    bounds seq_lens (None: S).  ``workspace``: attn_prompt_workspace's, allocated here when it is
    not given."""
    torch = _torch()
    device = _device_of(q, "q")
    bf16 = torch.bfloat16
    qp, kp, vp = _on(device, q, "q", bf16), _on(device, k, "k", bf16), _on(device, v, "v", bf16)
    qs, ks, vs = q.shape, k.shape, v.shape
    if len(qs) != 3 or len(ks) != 3 or len(vs) != 3 or ks[2] != qs[2] or vs[0] != ks[0] or vs[1] != ks[1]:
        raise MxidxError("q, k and v must be [T, Hq, dk], [S, Hk, dk] and [S, Hk, dv]")
    (T, Hq, dk), (S, Hk, dv) = qs, vs
    (q0, q1, q2), (k0, k1, k2), (v0, v1, v2) = q.stride(), k.stride(), v.stride()
    if (T and q2 != 1) or (S and (k2 != 1 or v2 != 1)):
        raise MxidxError("q, k and v must have a contiguous last dim")
    B = seq_lens.numel()
    sp = _on(device, seq_lens, "seq_lens", torch.int32, (B,))
    np_ = _on(device, query_lens, "query_lens", torch.int32, (B,))
    if max_seq_len is None:
        max_seq_len = S
    if out is None:
        out = _empty(stream, (T, Hq, dv), bf16, device, fill=0)
    op = _on(device, out, "out", bf16)
    o0, o1, o2 = out.stride()
    if out.shape != (T, Hq, dv) or (o2 != 1 and T):
        raise MxidxError(f"out must be [{T}, {Hq}, {dv}] with a contiguous last dim")
    if lse is None:
        lse = _empty(stream, (T, Hq), torch.float32, device, fill=float("-inf"))
    lp = _on(device, lse, "lse", torch.float32, (T, Hq))
    wp, wb = 0, 0
    if workspace is None:
        need = attn_prompt_workspace_bytes(T, Hq, Hk, dk, dv, B, max_seq_len)
        if need:
            workspace = _empty(stream, need, torch.uint8, device)
    if workspace is not None:
        wp, wb = _on(device, workspace, "workspace", torch.uint8), workspace.numel()
        if not workspace.is_contiguous():      # an expanded view has less memory than numel
            raise MxidxError("workspace must be contiguous")
    _call("idx_attn_prompt", device, stream, qp, q0, q1, T, Hq, kp, k0, k1, vp, v0, v1, S, Hk, dk, dv, sp, np_, B,
          max_seq_len, 1 if causal else 0, scale, op, o0, o1, lp, wp, wb)
    return out, lse
