"""ctypes binding of the serving operators of libi4s (include/i4s_serve.h),
same names as the C ABI.  Argument marshalling only, like ``_binding``; a
structure is passed as it is where a function takes its address.
"""

from __future__ import annotations

import ctypes
from typing import Optional

from . import _binding as B

I4S_KV_FORMAT_VERSION = 1
I4S_KV_MAX_REQUESTS = 4096
I4S_MAX_TOP_K = 32
I4S_MAX_TREE = 64

I4S_F16 = 0
I4S_BF16 = 1
I4S_F32 = 2

I4S_KV_BAD_LENGTH = 1
I4S_KV_ROW_FULL = 2
I4S_KV_NO_PAGES = 4
I4S_KV_NO_SLOTS = 8
I4S_KV_BAD_COUNT = 16


class i4s_kv_cache(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("k_vals", ctypes.c_void_p),
        ("v_vals", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
    ]


class i4s_kv_sizes(ctypes.Structure):
    _fields_ = [("vals", ctypes.c_uint64), ("scales", ctypes.c_uint64)]


class i4s_attention_args(ctypes.Structure):
    _fields_ = [
        ("cache", ctypes.c_void_p),
        ("q", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("q_heads", ctypes.c_int32),
        ("num_tokens", ctypes.c_int32),
        ("num_seqs", ctypes.c_int32),
        ("table", ctypes.c_void_p),
        ("table_width", ctypes.c_int32),
        ("lens", ctypes.c_void_p),
        ("q_start", ctypes.c_void_p),
        ("max_q", ctypes.c_int32),
        ("max_len", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("tree_mask", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_uint64),
    ]


_i32, _i64, _u64, _ptr = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
_cache_p = ctypes.POINTER(i4s_kv_cache)
_args_p = ctypes.POINTER(i4s_attention_args)

# every symbol include/i4s_serve.h declares, with its ctypes signature
SIGNATURES = {
    "i4s_kv_cache_sizes": (ctypes.c_int, [_i32] * 5 + [ctypes.POINTER(i4s_kv_sizes)]),
    "i4s_kv_extend": (ctypes.c_int, [_ptr, _i32, _i32, _i32, _ptr, _ptr, _ptr, _i32, _ptr, _i32] + [_ptr] * 7),
    "i4s_kv_append": (ctypes.c_int, [_cache_p, _ptr, _ptr, _i32, _i64, _i64, _i64, _i64, _ptr, _i32, _ptr]),
    "i4s_kv_read": (ctypes.c_int, [_cache_p, _ptr, _i32, _i32, _ptr, _ptr, _ptr]),
    "i4s_attention_workspace_size": (ctypes.c_int, [_args_p, ctypes.POINTER(_u64)]),
    "i4s_attention": (ctypes.c_int, [_args_p, _ptr]),
    "i4s_token_logprobs_workspace_size": (ctypes.c_int, [_i32] * 4 + [ctypes.POINTER(_u64)]),
    "i4s_token_logprobs": (ctypes.c_int, [_ptr, _i32, _i32, _i32, _i64, _ptr, _i32] + [_ptr] * 5 + [_u64, _ptr]),
}

_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """libi4s.so with the signatures of both headers attached."""
    global _lib
    if _lib is None:
        lib = B.load()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def __getattr__(name):
    # the library's functions under their C names, found when they are first used
    if name in SIGNATURES:
        globals()[name] = fn = getattr(load(), name)
        return fn
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
