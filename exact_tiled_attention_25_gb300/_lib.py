"""ctypes view of libattn_gb300.so (the C ABI declared in include/attn_gb300.h).

Loading never falls back to anything: if the library is missing or fails to
load, every entry point raises.
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB_PATH, NATIVE_PATH

c_int = ctypes.c_int
c_float = ctypes.c_float
c_size_t = ctypes.c_size_t
c_void_p = ctypes.c_void_p
c_char_p = ctypes.c_char_p
c_longlong = ctypes.c_longlong
c_double = ctypes.c_double
c_strides = ctypes.POINTER(c_longlong)   # host array of element strides, or None

# name -> (restype, argtypes); mirrors include/attn_gb300.h
SIGNATURES = {
    "attn_fwd": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                         c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_void_p]),
    "attn_fwd_schedule": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_int,
                                  c_void_p]),
    "attn_fwd_gqa": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_int, c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_void_p]),
    "attn_fwd_varlen": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_float, c_int,
                                c_void_p]),
    "attn_bwd_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int]),
    "attn_bwd_gqa": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                             c_int, c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_void_p]),
    "attn_bwd_varlen_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "attn_bwd_varlen": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p,
                                c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_float, c_int,
                                c_void_p]),
    "attn_bwd": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                         c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                         c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_void_p]),
    "attn_bwd_noalloc": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p,
                                 c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_void_p]),
    "attn_fp8_quantize": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_int, c_int, c_int, c_int, c_int, c_void_p]),
    "attn_fp8_quantize_gqa": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_int, c_int, c_int, c_int, c_int, c_int, c_void_p]),
    "attn_fwd_fp8_gqa": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int, c_int,
                                 c_float, c_void_p]),
    "attn_fp8_quantize_bf16": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_int, c_int, c_int, c_int, c_int, c_int, c_void_p]),
    "attn_fp8_quantize_varlen": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int,
                                         c_int, c_void_p]),
    "attn_fwd_fp8_varlen": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                    c_int, c_int, c_int, c_float, c_void_p]),
    "attn_fp8_quantize_rope": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                       c_void_p]),
    "attn_fp8_quantize_ex": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int, c_int,
                                     c_int, c_void_p]),
    "attn_decode_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int, c_int]),
    "attn_decode_paged": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_size_t, c_int, c_int, c_int, c_int, c_int,
                                  c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_void_p]),
    "attn_decode_paged_fp8": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                      c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                      c_int, c_int, c_float, c_int, c_void_p]),
    "attn_fwd_fp8_schedule": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int, c_float,
                                      c_int, c_void_p]),
    "attn_selftest_exp2": (c_int, [c_void_p, c_void_p, c_void_p, ctypes.c_longlong, c_void_p]),
    "attn_fwd_fp8": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int, c_float,
                             c_void_p]),
    "attn_cross_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int, c_int]),
    "attn_cross_bwd_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "attn_cross_fwd": (c_int, [c_void_p] * 7 + [c_size_t] + [c_int] * 6 + [c_float, c_int, c_void_p]),
    "attn_cross_bwd": (c_int, [c_void_p] * 11 + [c_size_t] + [c_int] * 6 + [c_float, c_int, c_void_p]),
    "attn_rope_table": (c_int, [c_void_p, c_void_p, c_longlong, c_int, c_double, c_double, c_longlong,
                                c_double, c_double, c_double, c_longlong, c_void_p]),
    "attn_rope": (c_int, [c_void_p] * 7 + [c_int] * 7 + [c_strides] * 4 + [c_int, c_int, c_int, c_void_p]),
    "attn_block_tables": (c_int, [c_void_p] * 9 + [c_int] * 5 + [c_void_p]),
    "attn_cache_append": (c_int, [c_void_p] * 10 + [c_int] * 8 + [c_strides] * 3 + [c_int, c_int, c_void_p]),
    "attn_cache_append_fp8": (c_int, [c_void_p] * 14 + [c_int] * 10 + [c_strides] * 3 +
                              [c_int, c_int, c_void_p]),
    "attn_cache_append_fp4": (c_int, [c_void_p] * 13 + [c_int] * 8 + [c_strides] * 3 + [c_int, c_int, c_void_p]),
    "attn_decode_fp4_workspace_size": (c_size_t, [c_int] * 6),
    "attn_decode_paged_fp4": (c_int, [c_void_p] * 11 + [c_size_t] + [c_int] * 10 + [c_float, c_int, c_void_p]),
    "attn_cache_read": (c_int, [c_void_p] * 8 + [c_int] * 8 + [c_void_p]),
    "attn_cache_read_fp8": (c_int, [c_void_p] * 11 + [c_int] * 8 + [c_void_p]),
    "attn_cache_read_fp4": (c_int, [c_void_p] * 11 + [c_int] * 8 + [c_void_p]),
    "attn_merge": (c_int, [c_void_p] * 6 + [c_int] * 6 + [c_void_p]),
    "attn_selftest_wait_timeout": (c_int, [ctypes.c_uint, c_void_p]),
    "attn_get_device_status": (c_int, [c_void_p]),
    "attn_status_string": (c_char_p, [c_int]),
    "attn_last_error": (c_char_p, []),
}

_LIB = None
_NATIVE = None


def load(path: str | None = None):
    """Load the library once and declare every entry point's signature."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is not built; run exact_tiled_attention_25_gb300.build.build() "
            "(nvcc for sm_103a is required)")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _LIB = lib
    return lib


def native(on_error):
    """The compiled part of the binding, tied to the library; on_error(code, name)
    raises for a status other than 0."""
    global _NATIVE
    if _NATIVE is None:
        load()
        import torch  # noqa: F401  (its libraries have to be loaded first)
        if not os.path.exists(NATIVE_PATH):
            raise RuntimeError(f"{NATIVE_PATH} is not built; run exact_tiled_attention_25_gb300.build.build()")
        from . import _native
        _native.bind(LIB_PATH, on_error)
        _NATIVE = _native
    return _NATIVE
