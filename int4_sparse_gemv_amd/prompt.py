"""What a prompt's step needs: products of any number of tokens in microscaled
4-bit floating point, and attention over whole prompts.

``mx_quantize`` brings weights (once) and activations into the microscaled
format (``MXTensor``: e2m1 values, a power-of-two scale for 32 columns),
``mx_read`` reads it back; ``mx_product`` multiplies tokens with a weight;
``prompt_attention`` attends from packed sequences of query tokens to their
own 16-bit keys and values, before ``kv_append`` writes those into the 4-bit
cache.  All call the HIP kernels of ``libi4s.so`` through
``include/i4s_prompt.h``, which states formats, rules and errors; they run on
the current stream of their tensors' device, allocate outputs and workspaces
with torch, never synchronise, and can be captured into a graph.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _binding as B
from . import _prompt_binding as P
from .serving import _DTYPES, _HALVES, _call, _check, _fit, _strides

__all__ = ["MXTensor", "mx_quantize", "mx_read", "mx_product", "prompt_attention"]


class MXTensor:
    """A matrix in the microscaled format: two caller-owned tensors and the C descriptor.

    ``vals``: uint8 [ceil(rows / 16), 2 * ceil(cols / 256), 1024]; ``scales``:
    uint8 [ceil(rows / 16), ceil(cols / 512), 256] (the layout inside is the
    format's).  What the tensors hold may change (``mx_quantize(x, out=...)``);
    which tensors they are, and the sizes, may not: the descriptor has their
    addresses.
    """

    def __init__(self, rows: int, cols: int, vals, scales):
        _fit(rows, cols)
        sz = P.i4s_mx_buffers()
        B.check(P.i4s_mx_sizes(rows, cols, sz), "i4s_mx_sizes")
        tiles = (rows + 15) // 16
        for name, t, shape in (("vals", vals, (tiles, 2 * ((cols + 255) // 256), 1024)),
                               ("scales", scales, (tiles, (cols + 511) // 512, 256))):
            if (t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_cuda or not t.is_contiguous()
                    or t.device != vals.device):
                raise ValueError(f"{name} must be a contiguous uint8 {list(shape)} tensor on one GPU")
        self._hold(rows, cols, vals, scales, vals.get_device())

    def _hold(self, rows, cols, vals, scales, index):
        descriptor = P.i4s_mx(rows, cols, vals.data_ptr(), scales.data_ptr())
        self.__dict__.update(rows=rows, cols=cols, vals=vals, scales=scales, index=index, shape=(rows, cols),
                             descriptor=descriptor, address=ctypes.addressof(descriptor))
        return self

    def __setattr__(self, name, value):
        raise AttributeError(f"an MXTensor's {name} is set when it is made; make another one")

    @property
    def device(self):
        return self.vals.device

    def nbytes(self) -> int:
        return self.vals.numel() + self.scales.numel()


def _rows_of(x, name):
    """(dtype number, row stride) of 16-bit [rows, cols] values with adjacent columns."""
    dtype = _HALVES.get(x.dtype)
    if dtype is None or x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a float16 or bfloat16 [rows, cols] tensor on a GPU")
    stride, step = x.stride()
    if step != 1 and x.shape[1] > 1:
        raise ValueError(f"the columns of {name} must lie next to each other")
    return dtype, (stride if x.shape[0] > 1 else x.shape[1])


def mx_quantize(x, out: Optional[MXTensor] = None) -> MXTensor:
    """Quantize x ([rows, cols], fp16 or bf16, cols a multiple of 32, rows may
    be strided) into the microscaled format; ``out`` takes the place of a new
    tensor."""
    dtype, stride = _rows_of(x, "x")
    rows, cols = x.shape
    _fit(rows, cols)
    if out is None:
        # the constructor's checks would find what is made here; the call checks rows and cols
        tiles = (rows + 15) // 16
        vals = x.new_empty((tiles, 2 * ((cols + 255) // 256), 1024), dtype=torch.uint8)
        out = MXTensor.__new__(MXTensor)._hold(rows, cols, vals, vals.new_empty((tiles, (cols + 511) // 512, 256)), x.get_device())
    elif out.shape != (rows, cols) or out.index != x.get_device():
        raise ValueError(f"out must be [{rows}, {cols}] on {x.device}, not {list(out.shape)} on {out.device}")
    st = _call(P.i4s_mx_quantize, out.index, x.data_ptr(), dtype, stride, out.descriptor)
    if st:
        B.check(st, "i4s_mx_quantize")
    return out


def mx_read(m: MXTensor, dtype=torch.float16):
    """The values that ``m`` holds, [rows, cols] of ``dtype``."""
    number = _DTYPES.get(dtype)
    if number is None:
        raise ValueError("dtype must be float16, bfloat16 or float32")
    out = m.vals.new_empty(m.shape, dtype=dtype)
    st = _call(P.i4s_mx_read, m.index, m.descriptor, number, out.data_ptr())
    if st:
        B.check(st, "i4s_mx_read")
    return out


@functools.lru_cache(maxsize=4096)
def _product_workspace(tokens: int, rows: int, cols: int, given: bool) -> int:
    """Bytes that a product of these sizes needs."""
    w = P.i4s_mx(rows, cols)
    x = P.i4s_mx(tokens, cols)
    a = P.i4s_mx_product_args(ctypes.addressof(w), ctypes.addressof(x) if given else None, None, 0, 0, tokens)
    n = ctypes.c_uint64()
    B.check(P.i4s_mx_product_workspace_size(a, n), "i4s_mx_product_workspace_size")
    return n.value


def mx_product(x, w: MXTensor, dtype=None, out=None):
    """y = x w^T: [tokens, rows of w] for tokens ``x``, an ``MXTensor`` or fp16
    or bf16 [tokens, cols of w] (quantized within the call, with the same
    result; tokens may be strided).  Sums are held in fp32 and rounded once to
    ``dtype`` (float16, bfloat16 or float32; x's, or ``out``'s, or float16).
    ``out`` may have strided tokens."""
    index, rows = w.index, w.rows
    given = isinstance(x, MXTensor)
    if given:
        tokens, cols, where = x.rows, x.cols, x.index
        address, values, x_stride, x_dtype = x.address, None, 0, 0
    else:
        x_dtype, x_stride = _rows_of(x, "x")
        (tokens, cols), where = x.shape, x.get_device()
        _fit(tokens)
        address, values = None, x.data_ptr()
        if dtype is None and out is None:
            dtype = x.dtype
    if cols != w.cols or where != index:
        raise ValueError(f"x has {cols} columns on GPU {where}, w {w.cols} on GPU {index}")
    if dtype is None:
        dtype = torch.float16 if out is None else out.dtype
    number = _DTYPES.get(dtype)
    if number is None:
        raise ValueError("dtype must be float16, bfloat16 or float32")
    y_stride = rows
    if out is None:
        out = w.vals.new_empty((tokens, rows), dtype=dtype)
    else:
        if (out.dtype is not dtype or out.shape != (tokens, rows) or out.get_device() != index
                or (rows > 1 and out.stride(1) != 1)):
            raise ValueError(f"out must be {dtype} {[tokens, rows]} on GPU {index} with adjacent columns, "
                             f"not {out.dtype} {list(out.shape)} on {out.device}")
        if tokens > 1:
            y_stride = out.stride(0)
    nbytes = _product_workspace(tokens, rows, cols, given)
    # a workspace of this call alone: calls on other streams and captured graphs have their own
    ws = w.vals.new_empty(nbytes) if nbytes else None
    st = _call(P.i4s_mx_product, index, P.i4s_mx_product_args(
        w.address, address, values, x_stride, x_dtype, tokens, out.data_ptr(), y_stride, number, 0,
        None if ws is None else ws.data_ptr(), nbytes))
    if st:
        B.check(st, "i4s_mx_product")
    return out


@functools.lru_cache(maxsize=4096)
def _attention_workspace(dtype, dim, heads, kv_heads, tokens, keys, n, max_q, max_k) -> int:
    """Bytes that a call of these sizes needs."""
    _fit(tokens, heads, keys, kv_heads, n, max_q, max_k)
    a = P.i4s_prompt_args(dtype=dtype, head_dim=dim, q_heads=heads, kv_heads=kv_heads, num_tokens=tokens, num_keys=keys,
                          num_seqs=n, max_q=max_q, max_k=max_k, scale=1.0)
    nbytes = ctypes.c_uint64()
    B.check(P.i4s_prompt_attention_workspace_size(a, nbytes), "i4s_prompt_attention_workspace_size")
    return nbytes.value


def prompt_attention(q, k, v, q_start=None, k_start=None, max_q: Optional[int] = None, max_k: int = 0, causal: bool = True,
                     scale: Optional[float] = None, out=None, lse=None):
    """Attention of packed sequences: q [tokens, q_heads, head_dim], k and v
    [keys, kv_heads, head_dim], all fp16 or all bf16, tokens and heads may be
    strided (slices of a fused q/k/v product are).

    ``q_start`` and ``k_start`` (int32 [sequences + 1]) bound each sequence's
    query tokens and keys; ``k_start`` defaults to ``q_start``, and without
    either there is one sequence of all tokens and all keys.  With ``causal``
    the last query token of a sequence sees all its keys and each token before
    it one less: a prompt, or the next chunk of one whose earlier keys are in k
    and v too.  ``max_q`` is the largest number of query tokens of a sequence
    and sizes the launch; its default, all of the tokens, is right but slow
    where sequences are many.  Rows of ``out`` that no sequence has, and tokens
    past a sequence's ``max_q``, are left as they were: whatever the memory
    held where ``out`` is not given.  ``max_k`` is the largest number of keys,
    if known.  ``scale`` defaults to head_dim ** -0.5.  ``lse`` (float32
    [tokens, q_heads]) receives the logarithm of the sum of exponentials.
    Returns [tokens, q_heads, head_dim] like q.
    """
    shape, kind, index = q.shape, q.dtype, q.get_device()
    dtype = _HALVES.get(kind)
    if dtype is None or len(shape) != 3 or index < 0:
        raise ValueError("q must be a float16 or bfloat16 [tokens, q_heads, head_dim] tensor on a GPU")
    tokens, heads, dim = shape
    held = k.shape
    if (len(held) != 3 or held != v.shape or held[2] != dim or k.dtype is not kind or v.dtype is not kind
            or k.get_device() != index or v.get_device() != index):
        raise ValueError(f"k and v must be {kind} [keys, kv_heads, {dim}] tensors on {q.device}")
    keys, kv_heads, _ = held
    if q_start is None:
        if k_start is not None:
            raise ValueError("k_start needs q_start")
        n, q_at, k_at = 1, None, None
    else:
        n = q_start.numel() - 1
        if n < 0:
            raise ValueError("q_start must be int32 [sequences + 1]")
        if k_start is None:
            k_start = q_start
        _check(q_start, torch.int32, (n + 1,), index, "q_start")
        _check(k_start, torch.int32, (n + 1,), index, "k_start")
        q_at, k_at = q_start.data_ptr(), k_start.data_ptr()
    if max_q is None:
        max_q = max(tokens, 1)
    if out is None:
        out = q.new_empty(shape)
    else:
        _check(out, kind, shape, index, "out")
    if lse is not None:
        _check(lse, torch.float32, (tokens, heads), index, "lse")
    nbytes = _attention_workspace(dtype, dim, heads, kv_heads, tokens, keys, n, max_q, max_k)
    # a workspace of this call alone: calls on other streams and captured graphs have their own
    ws = q.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    st = _call(P.i4s_prompt_attention, index, P.i4s_prompt_args(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), *_strides(q, "q"), *_strides(k, "k"), *_strides(v, "v"), dtype, dim, heads,
        kv_heads, tokens, keys, n, max_q, max_k, 1 if causal else 0, dim ** -0.5 if scale is None else scale, 0,
        q_at, k_at, out.data_ptr(), None if lse is None else lse.data_ptr(),
        None if ws is None else ws.data_ptr(), nbytes))
    if st:
        B.check(st, "i4s_prompt_attention")
    return out
