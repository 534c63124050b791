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


def _call(fn, device, *args):
    """fn(*args, stream) on the device's current stream, with the device current."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return fn(*args, torch.cuda.current_stream(device).cuda_stream)
    return fn(*args, torch._C._cuda_getCurrentRawStream(device.index))


def _int32(t, shape, device, name) -> None:
    if t.dtype != torch.int32 or tuple(t.shape) != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on {device}")


def _strides(t, name):
    """(token, head) strides of [tokens, heads, channels]; an axis of one counts as 0."""
    token, head, channel = t.stride()
    if channel != 1:
        raise ValueError(f"the channels of {name} must lie next to each other")
    return (token if t.shape[0] > 1 else 0), (head if t.shape[1] > 1 else 0)


class KVCache:
    """A 4-bit paged cache: four caller-owned tensors and the C descriptor.

    ``k_vals``, ``v_vals``: uint8 [pages, kv_heads, page_size * head_dim / 2];
    ``k_scales``, ``v_scales``: float16 [pages, kv_heads, page_size * head_dim
    / group_size] (the layout inside is the format's).
    """

    def __init__(self, page_size: int, kv_heads: int, head_dim: int, group_size: int, k_vals, v_vals, k_scales, v_scales):
        pages = k_vals.shape[0]
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
        d = S.i4s_kv_cache()
        d.num_pages, d.page_size, d.kv_heads, d.head_dim, d.group_size = pages, page_size, kv_heads, head_dim, group_size
        d.k_vals, d.v_vals = k_vals.data_ptr(), v_vals.data_ptr()
        d.k_scales, d.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
        self.descriptor = d

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k_vals, self.v_vals, self.k_scales, self.v_scales))


def kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, group_size: int = 64, device="cuda") -> KVCache:
    """Allocate a cache (its values start as zeros)."""
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
    if table.dim() != 2:
        raise ValueError("table must be int32 [requests, width]")
    n, width = table.shape
    device = table.device
    _int32(table, (n, width), device, "table")
    _int32(lens, (n,), device, "lens")
    _int32(new_lens, (n,), device, "new_lens")
    _int32(free_pages, (free_pages.numel(),), device, "free_pages")
    _int32(free_count, (1,), device, "free_count")
    if not table.is_cuda:
        raise ValueError("table must be on a GPU")
    # one allocation: lens, q_start, count, flags, slots, positions
    buf = torch.empty(2 * n + 3 + 2 * capacity, dtype=torch.int32, device=device)
    at = buf.data_ptr()
    o_start, o_count, o_slots = n, 2 * n + 1, 2 * n + 3
    st = _call(S.load().i4s_kv_extend, device, table.data_ptr(), n, width, page_size, lens.data_ptr(), new_lens.data_ptr(),
               free_pages.data_ptr(), free_pages.numel(), free_count.data_ptr(), capacity, at, at + 4 * o_start,
               at + 4 * o_slots, at + 4 * (o_slots + capacity), at + 4 * o_count, at + 4 * (o_count + 1))
    if st:
        B.check(st, "i4s_kv_extend")
    new, start, count, flags, slots, positions = buf.split_with_sizes((n, n + 1, 1, 1, capacity, capacity))
    return KVStep(new, start, slots, positions, count, flags)


def kv_append(cache: KVCache, k, v, slots) -> None:
    """Quantize k, v ([tokens, kv_heads, head_dim], fp16 or bf16) into ``slots``
    (int32 [tokens]; -1 skips a token).  Tokens and heads may be strided."""
    shape = k.shape
    if (len(shape) != 3 or shape != v.shape or shape[1] != cache.kv_heads or shape[2] != cache.head_dim
            or k.dtype != v.dtype or k.dtype not in (torch.float16, torch.bfloat16)):
        raise ValueError(f"k and v must be float16 or bfloat16 [tokens, {cache.kv_heads}, {cache.head_dim}]")
    device = cache.device
    if k.device != device or v.device != device:
        raise ValueError(f"k and v must be on {device}")
    tokens = shape[0]
    _int32(slots, (tokens,), device, "slots")
    ks, vs = _strides(k, "k"), _strides(v, "v")
    st = _call(S.load().i4s_kv_append, device, cache.descriptor, k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], ks[0], ks[1],
               vs[0], vs[1], slots.data_ptr(), tokens)
    if st:
        B.check(st, "i4s_kv_append")


def kv_read(cache: KVCache, slots, dtype=torch.float16):
    """(k, v) of the tokens at ``slots``, [tokens, kv_heads, head_dim] of
    ``dtype``; a slot outside the cache gives zeros."""
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float16, bfloat16 or float32")
    if slots.dim() != 1:
        raise ValueError("slots must be int32 [tokens]")
    device, tokens = cache.device, slots.shape[0]
    _int32(slots, (tokens,), device, "slots")
    k, v = torch.empty((2, tokens, cache.kv_heads, cache.head_dim), dtype=dtype, device=device).unbind()
    st = _call(S.load().i4s_kv_read, device, cache.descriptor, slots.data_ptr(), tokens, _DTYPES[dtype], k.data_ptr(),
               v.data_ptr())
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
    ``max_q`` (default: all of them); without it every sequence has one.
    ``max_len`` is the largest length, if known.  ``scale`` defaults to
    head_dim ** -0.5.  Token t sees the keys up to its own; with ``tree_mask``
    (int64 [tokens]) it sees the keys before the sequence's query tokens and
    those query tokens whose bit is set.  ``lse`` (float32 [tokens, q_heads])
    receives the logarithm of the sum of exponentials.  Returns [tokens,
    q_heads, head_dim] like q.
    """
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"q must be float16 or bfloat16 [tokens, q_heads, {cache.head_dim}]")
    device = cache.device
    if q.device != device:
        raise ValueError(f"q is on {q.device}, the cache on {device}")
    tokens, heads, dim = q.shape
    if table.dim() != 2:
        raise ValueError("table must be int32 [sequences, width]")
    n, width = table.shape
    _int32(table, (n, width), device, "table")
    _int32(lens, (n,), device, "lens")
    qs = _strides(q, "q")
    a = S.i4s_attention_args()
    if q_start is not None:
        _int32(q_start, (n + 1,), device, "q_start")
        a.q_start = q_start.data_ptr()
        a.max_q = max_q if max_q is not None else max(tokens, 1)
    else:
        a.max_q = max_q if max_q is not None else 1
    if tree_mask is not None:
        if tree_mask.dtype != torch.int64 or tuple(tree_mask.shape) != (tokens,) or tree_mask.device != device or not tree_mask.is_contiguous():
            raise ValueError(f"tree_mask must be a contiguous int64 [{tokens}] tensor on {device}")
        a.tree_mask = tree_mask.data_ptr()
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=q.dtype, device=device)
    elif out.dtype != q.dtype or out.shape != q.shape or out.device != device or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {q.dtype} {list(q.shape)} tensor on {device}")
    if lse is not None:
        if lse.dtype != torch.float32 or tuple(lse.shape) != (tokens, heads) or lse.device != device or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 [{tokens}, {heads}] tensor on {device}")
        a.lse = lse.data_ptr()
    a.cache = ctypes.addressof(cache.descriptor)
    a.q, a.q_token_stride, a.q_head_stride = q.data_ptr(), qs[0], qs[1]
    a.dtype, a.q_heads, a.num_tokens, a.num_seqs = _DTYPES[q.dtype], heads, tokens, n
    a.table, a.table_width, a.lens = table.data_ptr(), width, lens.data_ptr()
    a.max_len, a.scale, a.out = max_len, dim ** -0.5 if scale is None else scale, out.data_ptr()
    lib = S.load()
    nbytes = ctypes.c_uint64()
    st = lib.i4s_attention_workspace_size(a, nbytes)
    if st:
        B.check(st, "i4s_attention_workspace_size")
    if nbytes.value:
        # of this call alone: calls on other streams and captured graphs have their own
        ws = torch.empty(nbytes.value, dtype=torch.uint8, device=device)
        a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes.value
    st = _call(lib.i4s_attention, device, a)
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
    n = ctypes.c_uint64()
    B.check(S.i4s_token_logprobs_workspace_size(dtype, rows, vocab, top_k, n), "i4s_token_logprobs_workspace_size")
    return n.value


def token_logprobs(logits, tokens, top_k: int = 0) -> TokenLogprobs:
    """Log probabilities of ``tokens`` (int64 [rows]) under ``logits`` ([rows,
    vocab], fp16, bf16 or fp32, rows may be strided), the entropy of every row
    and its ``top_k`` largest alternatives (equal ones: lower index first)."""
    if logits.dim() != 2 or logits.dtype not in _DTYPES or not logits.is_cuda:
        raise ValueError("logits must be a float16, bfloat16 or float32 [rows, vocab] tensor on a GPU")
    rows, vocab = logits.shape
    device = logits.device
    if tokens.dtype != torch.int64 or tuple(tokens.shape) != (rows,) or tokens.device != device or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a contiguous int64 [{rows}] tensor on {device}")
    if logits.stride(1) != 1 and vocab > 1:
        raise ValueError("the values of a row must lie next to each other")
    stride = logits.stride(0) if rows > 1 else vocab
    dtype = _DTYPES[logits.dtype]
    nbytes = _logprobs_workspace(dtype, rows, vocab, top_k)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    out = torch.empty((2, rows), dtype=torch.float32, device=device)
    top_ids = torch.empty((rows, top_k), dtype=torch.int32, device=device)
    top = torch.empty((rows, top_k), dtype=torch.float32, device=device)
    at = out.data_ptr()
    st = _call(S.load().i4s_token_logprobs, device, logits.data_ptr(), dtype, rows, vocab, stride, tokens.data_ptr(), top_k,
               at, at + 4 * rows, top_ids.data_ptr(), top.data_ptr(), ws.data_ptr() if ws is not None else None, nbytes)
    if st:
        B.check(st, "i4s_token_logprobs")
    return TokenLogprobs(out[0], out[1], top_ids, top)
