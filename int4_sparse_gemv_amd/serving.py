"""What a decode or verification step needs between the packed products.

``kv_cache`` makes a paged KV cache held in 4 bits; ``kv_extend`` gives new
tokens their pages and slots from the requests' lengths, on the GPU;
``kv_append`` quantizes their keys and values into the cache and ``kv_read``
reads tokens back; ``kv_attention`` attends over the cache for one or several
query tokens per sequence (in order, or a tree of candidates);
``token_logprobs`` scores given tokens.  All call the HIP kernels of
``libi4s.so`` through ``include/i4s_serve.h``, which states formats, rules and
errors; they run on the current stream of their tensors' device, allocate
outputs and workspaces with torch, never synchronise, and can be captured
into a graph.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import _binding as B
from . import _serve_binding as S

__all__ = ["KVCache", "KVStep", "TokenLogprobs", "kv_cache", "kv_extend", "kv_append", "kv_read", "kv_attention",
           "token_logprobs"]

_DTYPES = {torch.float16: S.I4S_F16, torch.bfloat16: S.I4S_BF16, torch.float32: S.I4S_F32}
_HALVES = {torch.float16: S.I4S_F16, torch.bfloat16: S.I4S_BF16}

# The checks of a call are part of its time (a launch takes 3 us, a call 5 to
# 8): identity of types, devices as numbers, messages only when they are needed.


def _call(fn, index, *args):
    """fn(*args, stream) on the current stream of device `index`, with that device current."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return fn(*args, torch.cuda.current_stream(index).cuda_stream)
    return fn(*args, torch._C._cuda_getCurrentRawStream(index))


def _check(t, dtype, shape, index, name) -> None:
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on GPU {index}, "
                         f"not {t.dtype} {list(t.shape)} on {t.device}")


def _fit(*numbers) -> None:
    """ctypes would pass the lower half of a number that 32 bits do not hold."""
    if max(numbers) > 2147483647 or min(numbers) < -2147483648:
        raise ValueError(f"{[n for n in numbers if not -2**31 <= n < 2**31]}: 32 bits do not hold this number")


def _strides(t, name):
    """(token, head) strides of [tokens, heads, channels]; an axis of one counts as 0."""
    token, head, channel = t.stride()
    if channel != 1:
        raise ValueError(f"the channels of {name} must lie next to each other")
    shape = t.shape
    return (token if shape[0] > 1 else 0), (head if shape[1] > 1 else 0)


class KVCache:
    """A 4-bit paged cache: four caller-owned tensors and the C descriptor.

    ``k_vals``, ``v_vals``: uint8 [pages, kv_heads, page_size * head_dim / 2];
    ``k_scales``, ``v_scales``: float16 [pages, kv_heads, page_size * head_dim
    / group_size] (the layout inside is the format's).
    """

    def __init__(self, page_size: int, kv_heads: int, head_dim: int, group_size: int, k_vals, v_vals, k_scales, v_scales):
        pages = k_vals.shape[0]
        _fit(pages, page_size, kv_heads, head_dim, group_size)
        sz = S.i4s_kv_sizes()
        B.check(S.i4s_kv_cache_sizes(pages, page_size, kv_heads, head_dim, group_size, sz), "i4s_kv_cache_sizes")
        values = page_size * head_dim
        for name, t, dtype, last in (("k_vals", k_vals, torch.uint8, values // 2), ("v_vals", v_vals, torch.uint8, values // 2),
                                     ("k_scales", k_scales, torch.float16, values // group_size),
                                     ("v_scales", v_scales, torch.float16, values // group_size)):
            if (t.dtype != dtype or tuple(t.shape) != (pages, kv_heads, last) or not t.is_cuda or not t.is_contiguous()
                    or t.device != k_vals.device):
                raise ValueError(f"{name} must be a contiguous {dtype} [{pages}, {kv_heads}, {last}] tensor on one GPU")
        self.page_size, self.kv_heads, self.head_dim, self.group_size = page_size, kv_heads, head_dim, group_size
        self.num_pages = pages
        self.k_vals, self.v_vals, self.k_scales, self.v_scales = k_vals, v_vals, k_scales, v_scales
        self.device = k_vals.device
        self.index = self.device.index
        d = S.i4s_kv_cache()
        d.num_pages, d.page_size, d.kv_heads, d.head_dim, d.group_size = pages, page_size, kv_heads, head_dim, group_size
        d.k_vals, d.v_vals = k_vals.data_ptr(), v_vals.data_ptr()
        d.k_scales, d.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
        self.descriptor = d

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k_vals, self.v_vals, self.k_scales, self.v_scales))


def kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, group_size: int = 64, device="cuda") -> KVCache:
    """Allocate a cache (its values start as zeros)."""
    _fit(num_pages, page_size, kv_heads, head_dim, group_size)
    sz = S.i4s_kv_sizes()
    B.check(S.i4s_kv_cache_sizes(num_pages, page_size, kv_heads, head_dim, group_size, sz), "i4s_kv_cache_sizes")
    values = page_size * head_dim
    vals = [torch.full((num_pages, kv_heads, values // 2), 0x88, dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros(num_pages, kv_heads, values // group_size, dtype=torch.float16, device=device) for _ in range(2)]
    return KVCache(page_size, kv_heads, head_dim, group_size, *vals, *scales)


class KVStep(NamedTuple):
    """What ``kv_extend`` gives: int32 tensors on the GPU (``free_count`` and
    ``flags`` have one element; flags are the I4S_KV_* bits, 0 when all fits)."""
    lens: object
    q_start: object
    slots: object
    positions: object
    free_count: object
    flags: object


def kv_extend(table, lens, new_lens, free_pages, free_count, page_size: int, capacity: int) -> KVStep:
    """Pages and slots of ``new_lens[i]`` new tokens for each request i that
    holds ``lens[i]`` tokens.

    ``table`` (int32 [requests, width]) gets the numbers of the new pages,
    taken from the end of ``free_pages[:free_count]``; ``capacity`` bounds the
    new tokens (slots past them are -1).  If anything does not fit, nothing
    changes and ``flags`` says why.  The result's ``lens`` and ``free_count``
    are the next call's; a finished request's pages are given back by writing
    them to ``free_pages`` at ``free_count`` and raising that.
    """
    index = table.get_device()
    if table.dim() != 2 or index < 0:
        raise ValueError("table must be int32 [requests, width] on a GPU")
    n, width = shape = table.shape
    _check(table, torch.int32, shape, index, "table")
    _check(lens, torch.int32, (n,), index, "lens")
    _check(new_lens, torch.int32, (n,), index, "new_lens")
    entries = free_pages.numel()
    _check(free_pages, torch.int32, (entries,), index, "free_pages")
    _check(free_count, torch.int32, (1,), index, "free_count")
    _fit(n, width, page_size, entries, capacity)
    # one allocation: lens, q_start, count, flags, slots, positions
    buf = table.new_empty(2 * n + 3 + 2 * capacity)
    at = buf.data_ptr()
    start, count, slots = at + 4 * n, at + 8 * n + 4, at + 8 * n + 12
    st = _call(S.i4s_kv_extend, index, table.data_ptr(), n, width, page_size, lens.data_ptr(), new_lens.data_ptr(),
               free_pages.data_ptr(), entries, free_count.data_ptr(), capacity, at, start, slots, slots + 4 * capacity, count,
               count + 4)
    if st:
        B.check(st, "i4s_kv_extend")
    new, start, count, flags, slots, positions = buf.split_with_sizes((n, n + 1, 1, 1, capacity, capacity))
    return KVStep(new, start, slots, positions, count, flags)


def kv_append(cache: KVCache, k, v, slots) -> None:
    """Quantize k, v ([tokens, kv_heads, head_dim], fp16 or bf16) into ``slots``
    (int32 [tokens]; -1 skips a token).  Tokens and heads may be strided."""
    shape, dtype, index = k.shape, _HALVES.get(k.dtype), cache.index
    if (dtype is None or len(shape) != 3 or shape[1] != cache.kv_heads or shape[2] != cache.head_dim or v.shape != shape
            or v.dtype is not k.dtype):
        raise ValueError(f"k and v must be float16 or bfloat16 [tokens, {cache.kv_heads}, {cache.head_dim}]")
    if k.get_device() != index or v.get_device() != index:
        raise ValueError(f"k and v must be on {cache.device}")
    tokens = shape[0]
    _fit(0, tokens)
    _check(slots, torch.int32, (tokens,), index, "slots")
    ks, vs = _strides(k, "k"), _strides(v, "v")
    st = _call(S.i4s_kv_append, index, cache.descriptor, k.data_ptr(), v.data_ptr(), dtype, ks[0], ks[1], vs[0],
               vs[1], slots.data_ptr(), tokens)
    if st:
        B.check(st, "i4s_kv_append")


def kv_read(cache: KVCache, slots, dtype=torch.float16):
    """(k, v) of the tokens at ``slots``, [tokens, kv_heads, head_dim] of
    ``dtype``; a slot outside the cache gives zeros."""
    number, shape, index = _DTYPES.get(dtype), slots.shape, cache.index
    if number is None:
        raise ValueError("dtype must be float16, bfloat16 or float32")
    if len(shape) != 1:
        raise ValueError("slots must be int32 [tokens]")
    tokens = shape[0]
    _fit(0, tokens)
    _check(slots, torch.int32, shape, index, "slots")
    k = slots.new_empty((tokens, cache.kv_heads, cache.head_dim), dtype=dtype)
    v = torch.empty_like(k)
    st = _call(S.i4s_kv_read, index, cache.descriptor, slots.data_ptr(), tokens, number, k.data_ptr(), v.data_ptr())
    if st:
        B.check(st, "i4s_kv_read")
    return k, v


def kv_attention(cache: KVCache, q, table, lens, q_start=None, max_q: Optional[int] = None, max_len: int = 0,
                 scale: Optional[float] = None, tree_mask=None, out=None, lse=None):
    """Attention of the query tokens ``q`` ([tokens, q_heads, head_dim], fp16
    or bf16, tokens and heads may be strided) over the cache.

    ``table`` int32 [sequences, width] and ``lens`` int32 [sequences] say what
    each sequence holds, its query tokens included (append them first).
    ``q_start`` int32 [sequences + 1] bounds the query tokens of each, at most
    ``max_q``; without it every sequence has one.  ``max_q`` sizes the launch;
    its default, all of the tokens (with ``tree_mask`` the 64 that a mask can
    name), is right but slow where sequences have few of many.  Rows of ``out``
    that no sequence has, and tokens past a sequence's ``max_q``, are left as
    they were: whatever the memory held where ``out`` is not given.
    ``max_len`` is the largest length, if known.  ``scale`` defaults to
    head_dim ** -0.5.  Token t sees the keys up to its own; with ``tree_mask``
    (int64 [tokens]) it sees the keys before the sequence's query tokens and
    those query tokens whose bit is set.  ``lse`` (float32 [tokens, q_heads])
    receives the logarithm of the sum of exponentials.  Returns [tokens,
    q_heads, head_dim] like q.
    """
    shape, dtype, index = q.shape, _HALVES.get(q.dtype), cache.index
    if dtype is None or len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError(f"q must be float16 or bfloat16 [tokens, q_heads, {cache.head_dim}]")
    if q.get_device() != index:
        raise ValueError(f"q is on {q.device}, the cache on {cache.device}")
    tokens, heads, dim = shape
    if table.dim() != 2:
        raise ValueError("table must be int32 [sequences, width]")
    n, width = rows = table.shape
    _check(table, torch.int32, rows, index, "table")
    _check(lens, torch.int32, (n,), index, "lens")
    token_stride, head_stride = _strides(q, "q")
    if q_start is not None:
        _check(q_start, torch.int32, (n + 1,), index, "q_start")
        if max_q is None:
            max_q = max(tokens, 1)
            if tree_mask is not None and tokens <= S.I4S_MAX_TREE * n:
                max_q = min(max_q, S.I4S_MAX_TREE)
    elif max_q is None:
        max_q = 1
    _fit(tokens, heads, n, width, max_q, max_len)
    if tree_mask is not None:
        _check(tree_mask, torch.int64, (tokens,), index, "tree_mask")
    if out is None:
        out = q.new_empty(shape)
    else:
        _check(out, q.dtype, shape, index, "out")
    if lse is not None:
        _check(lse, torch.float32, (tokens, heads), index, "lse")
    a = S.i4s_attention_args(
        ctypes.addressof(cache.descriptor), q.data_ptr(), token_stride, head_stride, dtype, heads, tokens, n, table.data_ptr(),
        width, lens.data_ptr(), None if q_start is None else q_start.data_ptr(), max_q, max_len,
        dim ** -0.5 if scale is None else scale, None if tree_mask is None else tree_mask.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), None, 0)
    nbytes = ctypes.c_uint64()
    st = S.i4s_attention_workspace_size(a, nbytes)
    if st:
        B.check(st, "i4s_attention_workspace_size")
    if nbytes.value:
        # of this call alone: calls on other streams and captured graphs have their own
        ws = q.new_empty(nbytes.value, dtype=torch.uint8)
        a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes.value
    st = _call(S.i4s_attention, index, a)
    if st:
        B.check(st, "i4s_attention")
    return out


class TokenLogprobs(NamedTuple):
    logprobs: object      # float32 [rows]
    entropy: object       # float32 [rows], nats
    top_ids: object       # int32 [rows, top_k]
    top_logprobs: object  # float32 [rows, top_k]


@functools.lru_cache(maxsize=4096)
def _logprobs_workspace(dtype: int, rows: int, vocab: int, top_k: int) -> int:
    _fit(rows, vocab, top_k)
    n = ctypes.c_uint64()
    B.check(S.i4s_token_logprobs_workspace_size(dtype, rows, vocab, top_k, n), "i4s_token_logprobs_workspace_size")
    return n.value


def token_logprobs(logits, tokens, top_k: int = 0) -> TokenLogprobs:
    """Log probabilities of ``tokens`` (int64 [rows]) under ``logits`` ([rows,
    vocab], fp16, bf16 or fp32, rows may be strided), the entropy of every row
    and its ``top_k`` largest alternatives (equal ones: lower index first)."""
    dtype, index = _DTYPES.get(logits.dtype), logits.get_device()
    if dtype is None or logits.dim() != 2 or index < 0:
        raise ValueError("logits must be a float16, bfloat16 or float32 [rows, vocab] tensor on a GPU")
    rows, vocab = logits.shape
    _check(tokens, torch.int64, (rows,), index, "tokens")
    stride, step = logits.stride()
    if step != 1 and vocab > 1:
        raise ValueError("the values of a row must lie next to each other")
    if rows < 2:
        stride = vocab
    nbytes = _logprobs_workspace(dtype, rows, vocab, top_k)
    ws = logits.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    logprobs = logits.new_empty(rows, dtype=torch.float32)
    entropy = torch.empty_like(logprobs)
    top_ids = tokens.new_empty((rows, top_k), dtype=torch.int32)
    top = logprobs.new_empty((rows, top_k))
    st = _call(S.i4s_token_logprobs, index, logits.data_ptr(), dtype, rows, vocab, stride, tokens.data_ptr(), top_k,
               logprobs.data_ptr(), entropy.data_ptr(), top_ids.data_ptr(), top.data_ptr(),
               None if ws is None else ws.data_ptr(), nbytes)
    if st:
        B.check(st, "i4s_token_logprobs")
    return TokenLogprobs(logprobs, entropy, top_ids, top)
