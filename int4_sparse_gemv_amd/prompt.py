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
    format's).
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
        self.rows, self.cols, self.vals, self.scales = rows, cols, vals, scales
        self.device = vals.device
        self.index = self.device.index
        self.descriptor = P.i4s_mx(rows, cols, vals.data_ptr(), scales.data_ptr())
        self.address = ctypes.addressof(self.descriptor)

    @property
    def shape(self):
        return self.rows, self.cols

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
        sz = P.i4s_mx_buffers()
        B.check(P.i4s_mx_sizes(rows, cols, sz), "i4s_mx_sizes")
        tiles = (rows + 15) // 16
        out = MXTensor(rows, cols, x.new_empty((tiles, 2 * ((cols + 255) // 256), 1024), dtype=torch.uint8),
                       x.new_empty((tiles, (cols + 511) // 512, 256), dtype=torch.uint8))
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


def mx_product(x, w: MXTensor, dtype=None, out=None):
    """y = x w^T: [tokens, rows of w] for tokens ``x``, an ``MXTensor`` or fp16
    or bf16 [tokens, cols of w] (quantized within the call, with the same
    result; tokens may be strided).  Sums are held in fp32 and rounded once to
    ``dtype`` (float16, bfloat16 or float32; x's, or ``out``'s, or float16).
    ``out`` may have strided tokens."""
    index = w.index
    a = P.i4s_mx_product_args()
    if isinstance(x, MXTensor):
        tokens, cols, where = x.rows, x.cols, x.index
        a.x = x.address
    else:
        a.x_dtype, a.x_stride = _rows_of(x, "x")
        (tokens, cols), where = x.shape, x.get_device()
        _fit(tokens)
        a.x_values = x.data_ptr()
        if dtype is None and out is None:
            dtype = x.dtype
    if cols != w.cols or where != index:
        raise ValueError(f"x has {cols} columns on GPU {where}, w {w.cols} on GPU {index}")
    if dtype is None:
        dtype = torch.float16 if out is None else out.dtype
    number = _DTYPES.get(dtype)
    if number is None:
        raise ValueError("dtype must be float16, bfloat16 or float32")
    shape = (tokens, w.rows)
    if out is None:
        out = w.vals.new_empty(shape, dtype=dtype)
        a.y_stride = w.rows
    else:
        if out.dtype is not dtype or out.shape != shape or out.get_device() != index or (w.rows > 1 and out.stride(1) != 1):
            raise ValueError(f"out must be {dtype} {list(shape)} on GPU {index} with adjacent columns, "
                             f"not {out.dtype} {list(out.shape)} on {out.device}")
        a.y_stride = out.stride(0) if tokens > 1 else w.rows
    a.w, a.tokens, a.y, a.y_dtype = w.address, tokens, out.data_ptr(), number
    nbytes = ctypes.c_uint64()
    st = P.i4s_mx_product_workspace_size(a, nbytes)
    if st:
        B.check(st, "i4s_mx_product_workspace_size")
    if nbytes.value:
        # of this call alone: calls on other streams and captured graphs have their own
        ws = w.vals.new_empty(nbytes.value)
        a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes.value
    st = _call(P.i4s_mx_product, index, a)
    if st:
        B.check(st, "i4s_mx_product")
    return out


def _whole(n, device):
    """[0, n]: where the one sequence begins and ends."""
    if n == 0:
        return torch.zeros(2, dtype=torch.int32, device=device)
    return torch.arange(0, n + 1, n, dtype=torch.int32, device=device)


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
    shape, dtype, index = q.shape, _HALVES.get(q.dtype), q.get_device()
    if dtype is None or len(shape) != 3 or index < 0:
        raise ValueError("q must be a float16 or bfloat16 [tokens, q_heads, head_dim] tensor on a GPU")
    tokens, heads, dim = shape
    if (k.dim() != 3 or k.shape != v.shape or k.shape[2] != dim or k.dtype is not q.dtype or v.dtype is not q.dtype
            or k.get_device() != index or v.get_device() != index):
        raise ValueError(f"k and v must be {q.dtype} [keys, kv_heads, {dim}] tensors on {q.device}")
    keys, kv_heads = k.shape[0], k.shape[1]
    qs, ks, vs = _strides(q, "q"), _strides(k, "k"), _strides(v, "v")
    if q_start is None:
        if k_start is not None:
            raise ValueError("k_start needs q_start")
        q_start = _whole(tokens, q.device)
        k_start = q_start if keys == tokens else _whole(keys, q.device)
    if k_start is None:
        k_start = q_start
    n = q_start.numel() - 1
    if n < 0:
        raise ValueError("q_start must be int32 [sequences + 1]")
    _check(q_start, torch.int32, (n + 1,), index, "q_start")
    _check(k_start, torch.int32, (n + 1,), index, "k_start")
    if max_q is None:
        max_q = max(tokens, 1)
    _fit(tokens, heads, keys, kv_heads, n, max_q, max_k)
    if out is None:
        out = q.new_empty(shape)
    else:
        _check(out, q.dtype, shape, index, "out")
    if lse is not None:
        _check(lse, torch.float32, (tokens, heads), index, "lse")
    a = P.i4s_prompt_args(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], dtype, dim, heads, kv_heads,
        tokens, keys, n, max_q, max_k, int(bool(causal)), dim ** -0.5 if scale is None else scale, 0, q_start.data_ptr(),
        k_start.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), None, 0)
    nbytes = ctypes.c_uint64()
    st = P.i4s_prompt_attention_workspace_size(a, nbytes)
    if st:
        B.check(st, "i4s_prompt_attention_workspace_size")
    if nbytes.value:
        # of this call alone: calls on other streams and captured graphs have their own
        ws = q.new_empty(nbytes.value, dtype=torch.uint8)
        a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes.value
    st = _call(P.i4s_prompt_attention, index, a)
    if st:
        B.check(st, "i4s_prompt_attention")
    return out
