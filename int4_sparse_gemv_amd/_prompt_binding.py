"""ctypes binding of the prompt's operators of libi4s (include/i4s_prompt.h),
same names as the C ABI.  Argument marshalling only, like ``_binding``; a
structure is passed as it is where a function takes its address.
"""

from __future__ import annotations

import ctypes
from typing import Optional

from . import _binding as B
from ._serve_binding import I4S_BF16, I4S_F16, I4S_F32  # noqa: F401  (the element types)

I4S_MX_FORMAT_VERSION = 1


class i4s_mx(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("vals", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
    ]


class i4s_mx_buffers(ctypes.Structure):
    _fields_ = [("vals", ctypes.c_uint64), ("scales", ctypes.c_uint64)]


class i4s_mx_product_args(ctypes.Structure):
    _fields_ = [
        ("w", ctypes.c_void_p),
        ("x", ctypes.c_void_p),
        ("x_values", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64),
        ("x_dtype", ctypes.c_int32),
        ("tokens", ctypes.c_int32),
        ("y", ctypes.c_void_p),
        ("y_stride", ctypes.c_int64),
        ("y_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_uint64),
    ]


class i4s_prompt_args(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("q_heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("num_tokens", ctypes.c_int32),
        ("num_keys", ctypes.c_int32),
        ("num_seqs", ctypes.c_int32),
        ("max_q", ctypes.c_int32),
        ("max_k", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
        ("q_start", ctypes.c_void_p),
        ("k_start", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_uint64),
    ]


_i32, _i64, _ptr = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_u64_p = ctypes.POINTER(ctypes.c_uint64)
_mx_p = ctypes.POINTER(i4s_mx)
_product_p = ctypes.POINTER(i4s_mx_product_args)
_prompt_p = ctypes.POINTER(i4s_prompt_args)

# every symbol include/i4s_prompt.h declares, with its ctypes signature
SIGNATURES = {
    "i4s_mx_sizes": (ctypes.c_int, [_i32, _i32, ctypes.POINTER(i4s_mx_buffers)]),
    "i4s_mx_quantize": (ctypes.c_int, [_ptr, _i32, _i64, _mx_p, _ptr]),
    "i4s_mx_read": (ctypes.c_int, [_mx_p, _i32, _ptr, _ptr]),
    "i4s_mx_product_workspace_size": (ctypes.c_int, [_product_p, _u64_p]),
    "i4s_mx_product": (ctypes.c_int, [_product_p, _ptr]),
    "i4s_prompt_attention_workspace_size": (ctypes.c_int, [_prompt_p, _u64_p]),
    "i4s_prompt_attention": (ctypes.c_int, [_prompt_p, _ptr]),
}

_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """libi4s.so with the signatures of this header and of i4s.h attached."""
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
