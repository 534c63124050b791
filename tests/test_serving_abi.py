"""CPU tests of include/i4s_serve.h: declarations, struct layouts, sizes and
the refusals of every entry point, before any device call."""

import ctypes
import os
import re
import subprocess

import pytest

from int4_sparse_gemv_amd import _binding as B
from int4_sparse_gemv_amd import _serve_binding as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "i4s_serve.h")
BAD, SMALL = B.I4S_ERR_INVALID_ARGUMENT, B.I4S_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from int4_sparse_gemv_amd import build
        build.build()
    return S.load()


def test_header_binding_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(i4s_[a-z_]+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True).stdout
    exported = set(re.findall(r"\bT (i4s_[a-z_]+)$", out, flags=re.M))
    assert declared == set(S.SIGNATURES) and declared <= exported
    for name in ("I4S_KV_FORMAT_VERSION", "I4S_KV_MAX_REQUESTS", "I4S_MAX_TOP_K", "I4S_MAX_TREE", "I4S_KV_BAD_LENGTH",
                 "I4S_KV_ROW_FULL", "I4S_KV_NO_PAGES", "I4S_KV_NO_SLOTS", "I4S_KV_BAD_COUNT"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(S, name)


def test_struct_layouts(tmp_path):
    src = tmp_path / "layout.c"
    fields = [f for f, _ in S.i4s_attention_args._fields_]
    src.write_text('#include <stdio.h>\n#include "i4s_serve.h"\nint main(void) {\n'
                   '  printf("%zu %zu %zu %zu", sizeof(i4s_kv_cache), offsetof(i4s_kv_cache, k_vals), '
                   'offsetof(i4s_kv_cache, v_scales), sizeof(i4s_kv_sizes));\n  printf(" %zu", sizeof(i4s_attention_args));\n'
                   + "".join(f'  printf(" %zu", offsetof(i4s_attention_args, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    C, A = S.i4s_kv_cache, S.i4s_attention_args
    assert got == [ctypes.sizeof(C), C.k_vals.offset, C.v_scales.offset, ctypes.sizeof(S.i4s_kv_sizes), ctypes.sizeof(A),
                   *[getattr(A, f).offset for f in fields]]


@pytest.mark.parametrize("args,vals,scales", [((1, 16, 1, 64, 32), 512, 64), ((1000, 128, 40, 128, 64), 327680000, 20480000),
                                              ((8388607, 256, 8, 128, 128), 8388607 * 256 * 512, 8388607 * 256 * 16)])
def test_cache_sizes(lib, args, vals, scales):
    sz = S.i4s_kv_sizes()
    assert S.i4s_kv_cache_sizes(*args, sz) == 0 and (sz.vals, sz.scales) == (vals, scales)


@pytest.mark.parametrize("args", [(0, 16, 1, 64, 32), (1, 15, 1, 64, 32), (1, 8, 1, 64, 32), (1, 48, 1, 64, 32),
                                  (1, 512, 1, 64, 32), (1, 16, 0, 64, 32), (1, 16, 1025, 64, 32), (1, 16, 1, 96, 32),
                                  (1, 16, 1, 64, 128), (1, 16, 1, 128, 16), (8388608, 256, 1, 64, 32), (-1, 16, 1, 64, 32)])
def test_cache_sizes_refuses(lib, args):
    sz = S.i4s_kv_sizes()
    assert S.i4s_kv_cache_sizes(*args, sz) == BAD and B.i4s_last_error()
    assert lib.i4s_kv_cache_sizes(1, 16, 1, 64, 32, None) == BAD


GIB = 1 << 30


def cache(**kw):
    c = S.i4s_kv_cache()
    c.num_pages, c.page_size, c.kv_heads, c.head_dim, c.group_size = 10, 16, 2, 64, 32
    c.k_vals, c.v_vals, c.k_scales, c.v_scales = GIB, 2 * GIB, 3 * GIB, 4 * GIB
    for k, v in kw.items():
        setattr(c, k, v)
    return c


EXTEND = dict(table=GIB, n=3, width=4, page=16, lens=2 * GIB, new=3 * GIB, free=4 * GIB, entries=5, count=5 * GIB, capacity=9,
              lens_out=6 * GIB, q_start=7 * GIB, slots=8 * GIB, positions=9 * GIB, count_out=10 * GIB, flags=11 * GIB)


@pytest.mark.parametrize("change", [dict(table=None), dict(table=GIB + 2), dict(n=-1), dict(n=4097), dict(width=0), dict(page=20),
                                    dict(lens=None), dict(new=1), dict(free=None), dict(entries=-1), dict(count=None),
                                    dict(capacity=-1), dict(lens_out=2 * GIB), dict(q_start=None), dict(slots=GIB),
                                    dict(positions=8 * GIB + 32), dict(count_out=5 * GIB), dict(flags=None), dict(flags=10 * GIB),
                                    dict(table=4 * GIB + 16)])
def test_extend_refuses(lib, change):
    a = dict(EXTEND, **change)
    assert S.i4s_kv_extend(*a.values(), None) == BAD and B.i4s_last_error()


APPEND = dict(k=5 * GIB, v=6 * GIB, dtype=0, kt=128, kh=64, vt=128, vh=64, slots=7 * GIB, tokens=4)


@pytest.mark.parametrize("change", [dict(k=None), dict(v=6 * GIB + 8), dict(dtype=2), dict(dtype=-1), dict(kt=12), dict(vh=-8),
                                    dict(kt=1 << 41), dict(slots=None), dict(slots=7 * GIB + 1), dict(tokens=-1), dict(tokens=2**31 - 1),
                                    dict(k=GIB + 64), dict(v=4 * GIB), dict(slots=3 * GIB)])
def test_append_refuses(lib, change):
    a = dict(APPEND, **change)
    assert S.i4s_kv_append(cache(), *a.values(), None) == BAD and B.i4s_last_error()


@pytest.mark.parametrize("change", [dict(k_vals=None), dict(v_vals=2 * GIB + 8), dict(k_scales=3 * GIB + 2), dict(v_scales=None),
                                    dict(reserved=1), dict(num_pages=0), dict(head_dim=32), dict(group_size=48),
                                    dict(v_vals=GIB + 16)])
def test_every_call_refuses_a_bad_cache(lib, change):
    c = cache(**change)
    overlapping = change.get("v_vals") == GIB + 16  # only a call that writes the cache minds
    assert S.i4s_kv_append(c, *APPEND.values(), None) == BAD
    if not overlapping:
        assert S.i4s_kv_read(c, 7 * GIB, 4, 0, 8 * GIB, 9 * GIB, None) == BAD
        assert S.i4s_attention(attention(c), None) == BAD
    assert lib.i4s_kv_append(None, *APPEND.values(), None) == BAD
    assert lib.i4s_kv_read(None, 7 * GIB, 4, 0, 8 * GIB, 9 * GIB, None) == BAD


@pytest.mark.parametrize("args", [(None, 4, 0, 8 * GIB, 9 * GIB), (7 * GIB, -1, 0, 8 * GIB, 9 * GIB), (7 * GIB, 4, 3, 8 * GIB, 9 * GIB),
                                  (7 * GIB, 4, 0, None, 9 * GIB), (7 * GIB, 4, 0, 8 * GIB, 9 * GIB + 8), (7 * GIB, 4, 0, GIB, 9 * GIB),
                                  (7 * GIB, 4, 2, 8 * GIB, 8 * GIB + 16), (7 * GIB, 4, 0, 8 * GIB, 7 * GIB)])
def test_read_refuses(lib, args):
    assert S.i4s_kv_read(cache(), *args, None) == BAD and B.i4s_last_error()


def attention(c, **kw):
    a = S.i4s_attention_args()
    a._keep = c
    a.cache = ctypes.addressof(c)
    a.q, a.q_token_stride, a.q_head_stride = 5 * GIB, 256, 64
    a.dtype, a.q_heads, a.num_tokens, a.num_seqs = 0, 4, 6, 2
    a.table, a.table_width, a.lens, a.q_start = 6 * GIB, 100, 7 * GIB, 8 * GIB
    a.max_q, a.max_len, a.scale, a.out = 5, 0, 0.125, 9 * GIB
    a.lse, a.tree_mask = 10 * GIB, 11 * GIB
    a.workspace, a.workspace_bytes = 12 * GIB, GIB
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(cache=None), dict(q=None), dict(q=5 * GIB + 8), dict(q_token_stride=7), dict(q_head_stride=-8), dict(dtype=2), dict(q_heads=3),
    dict(q_heads=0), dict(num_tokens=-1), dict(num_seqs=-1), dict(num_seqs=65536), dict(table=None), dict(table_width=0),
    dict(table_width=(1 << 26) + 1), dict(lens=None), dict(lens=7 * GIB + 2), dict(q_start=None), dict(max_q=0), dict(max_q=65),
    dict(max_len=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None),
    dict(out=9 * GIB + 4), dict(out=5 * GIB), dict(lse=9 * GIB), dict(lse=10 * GIB + 2), dict(tree_mask=11 * GIB + 4),
    dict(workspace=None), dict(workspace=12 * GIB + 8), dict(workspace=GIB), dict(out=12 * GIB), dict(lse=7 * GIB)])
def test_attention_refuses(lib, change):
    a = attention(cache(), **change)
    assert S.i4s_attention(a, None) == BAD and B.i4s_last_error()


def test_attention_workspace(lib):
    n = ctypes.c_uint64()
    a = attention(cache())
    assert S.i4s_attention_workspace_size(a, n) == 0 and n.value > 0 and n.value % 16 == 0
    # partial outputs, offsets and sums of every piece
    assert n.value % (6 * 4 * (64 + 4) * 4) == 0
    a.workspace_bytes = n.value - 1
    assert S.i4s_attention(a, None) == SMALL
    a.num_tokens = a.num_seqs = 0
    assert S.i4s_attention_workspace_size(a, n) == 0 and n.value == 0
    assert S.i4s_attention(a, None) == 0  # nothing to do
    # many rows, or few keys: nothing is split
    for kw in (dict(num_seqs=4096, num_tokens=4096, tree_mask=None), dict(max_len=16)):
        assert S.i4s_attention_workspace_size(attention(cache(), **kw), n) == 0 and n.value == 0
    assert lib.i4s_attention_workspace_size(ctypes.byref(a), None) == BAD
    assert lib.i4s_attention_workspace_size(None, ctypes.byref(n)) == BAD
    assert lib.i4s_attention(None, None) == BAD
    for q, heads in ((1 << 20, 65536), (1 << 20, 8), (1 << 7, 65536)):
        big = attention(cache(), num_seqs=65535, max_q=q, tree_mask=None, q_heads=heads)
        assert S.i4s_attention_workspace_size(big, n) == BAD


LOGPROBS = dict(logits=GIB, dtype=0, rows=3, vocab=90000, stride=90000, tokens=2 * GIB, top_k=5, lp=3 * GIB, ent=4 * GIB,
                ids=5 * GIB, top=6 * GIB, ws=7 * GIB, ws_bytes=1 << 20)


@pytest.mark.parametrize("change", [dict(logits=None), dict(logits=GIB + 1), dict(dtype=3), dict(rows=-1), dict(rows=1 << 23), dict(vocab=0),
                                    dict(vocab=(1 << 30) + 1), dict(stride=89999), dict(tokens=None), dict(tokens=2 * GIB + 4),
                                    dict(top_k=-1), dict(top_k=33), dict(vocab=4), dict(lp=None), dict(ent=4 * GIB + 1),
                                    dict(ids=None), dict(top=None), dict(ids=6 * GIB), dict(lp=4 * GIB), dict(ws=None),
                                    dict(ws=7 * GIB + 8), dict(ws=GIB), dict(ent=GIB + 100), dict(top=2 * GIB)])
def test_logprobs_refuses(lib, change):
    a = dict(LOGPROBS, **change)
    assert S.i4s_token_logprobs(*a.values(), None) == BAD and B.i4s_last_error()


def test_logprobs_workspace(lib):
    n = ctypes.c_uint64()
    assert S.i4s_token_logprobs_workspace_size(0, 3, 90000, 5, n) == 0 and n.value > 0
    a = dict(LOGPROBS, ws_bytes=n.value - 1)
    assert S.i4s_token_logprobs(*a.values(), None) == SMALL
    assert S.i4s_token_logprobs(*dict(LOGPROBS, rows=0).values(), None) == 0
    for rows, vocab in ((5000, 200000), (1, 500), (0, 90000)):
        assert S.i4s_token_logprobs_workspace_size(2, rows, vocab, 5, n) == 0 and n.value == 0
    assert S.i4s_token_logprobs_workspace_size(0, 3, 90000, 33, n) == BAD
    assert lib.i4s_token_logprobs_workspace_size(0, 3, 90000, 5, None) == BAD
