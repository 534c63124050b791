"""CPU tests of include/i4s_prompt.h: declarations, struct layouts, sizes and
the refusals of every entry point, before any device call."""

import ctypes
import os
import re
import subprocess

import pytest

from int4_sparse_gemv_amd import _binding as B
from int4_sparse_gemv_amd import _prompt_binding as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "i4s_prompt.h")
BAD, SMALL = B.I4S_ERR_INVALID_ARGUMENT, B.I4S_ERR_WORKSPACE_TOO_SMALL
GIB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from int4_sparse_gemv_amd import build
        build.build()
    return P.load()


def test_header_binding_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(i4s_[a-z_]+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True).stdout
    exported = set(re.findall(r"\bT (i4s_[a-z_]+)$", out, flags=re.M))
    assert declared == set(P.SIGNATURES) and declared <= exported
    assert int(re.search(r"#define I4S_MX_FORMAT_VERSION (\d+)", text).group(1)) == P.I4S_MX_FORMAT_VERSION
    for name in P.SIGNATURES:
        assert getattr(P, name) is getattr(lib, name), name
    with pytest.raises(AttributeError):
        P.i4s_run


def test_struct_layouts(tmp_path):
    src = tmp_path / "layout.c"
    structs = [P.i4s_mx, P.i4s_mx_buffers, P.i4s_mx_product_args, P.i4s_prompt_args]
    src.write_text('#include <stdio.h>\n#include "i4s_prompt.h"\nint main(void) {\n' + "".join(
        f'  printf("%zu ", sizeof({s.__name__}));\n' + "".join(
            f'  printf("%zu ", offsetof({s.__name__}, {f}));\n' for f, _ in s._fields_) for s in structs) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [n for s in structs for n in (ctypes.sizeof(s), *(getattr(s, f).offset for f, _ in s._fields_))]


# ---------------------------------------------------------------------------
# the microscaled format


@pytest.mark.parametrize("rows,cols,vals,scales", [(0, 32, 0, 0), (1, 32, 2048, 256), (16, 256, 2048, 256), (17, 288, 8192, 512),
                                                   (50257, 4096, 3142 * 32 * 1024, 3142 * 8 * 256),
                                                   ((1 << 18) - 16, 1 << 20, 16383 * 8192 * 1024, 16383 * 2048 * 256)])
def test_mx_sizes(lib, rows, cols, vals, scales):
    sz = P.i4s_mx_buffers()
    assert P.i4s_mx_sizes(rows, cols, sz) == 0 and (sz.vals, sz.scales) == (vals, scales)


@pytest.mark.parametrize("rows,cols", [(-1, 32), ((1 << 24) + 1, 32), (1, 0), (1, 31), (1, 48), (1, -32), (1, (1 << 20) + 32),
                                       (1 << 18, 1 << 20)])
def test_mx_sizes_refuses(lib, rows, cols):
    assert P.i4s_mx_sizes(rows, cols, P.i4s_mx_buffers()) == BAD and B.i4s_last_error()
    assert P.i4s_mx_sizes(1, 32, None) == BAD


def mx(rows=20, cols=64, vals=GIB, scales=2 * GIB):
    return P.i4s_mx(rows, cols, vals, scales)


QUANTIZE = dict(x=3 * GIB, dtype=0, stride=64, out=mx())


@pytest.mark.parametrize("change", [dict(x=None), dict(x=3 * GIB + 8), dict(dtype=2), dict(dtype=-1), dict(stride=56),
                                    dict(stride=68), dict(stride=(1 << 40) + 8), dict(stride=-64), dict(out=None),
                                    dict(out=mx(rows=-1)), dict(out=mx(cols=40)), dict(out=mx(vals=None)), dict(out=mx(vals=GIB + 8)),
                                    dict(out=mx(scales=None)), dict(out=mx(scales=2 * GIB + 4)), dict(x=GIB), dict(x=2 * GIB - 128),
                                    dict(out=mx(vals=2 * GIB)), dict(x=GIB - 2 * 64 * 20 + 16)])
def test_quantize_refuses(lib, change):
    a = dict(QUANTIZE, **change)
    assert P.i4s_mx_quantize(*a.values(), None) == BAD and B.i4s_last_error()


@pytest.mark.parametrize("change", [dict(m=None), dict(m=mx(vals=None)), dict(m=mx(scales=8)), dict(m=mx(cols=0)), dict(dtype=3),
                                    dict(dtype=-1), dict(out=None), dict(out=3 * GIB + 4), dict(out=GIB), dict(out=2 * GIB)])
def test_read_refuses(lib, change):
    a = dict(dict(m=mx(), dtype=1, out=3 * GIB), **change)
    assert P.i4s_mx_read(*a.values(), None) == BAD and B.i4s_last_error()


def test_nothing_to_do_needs_no_device(lib):
    none = mx(0, 64, None, None)
    assert P.i4s_mx_quantize(None, 0, 64, none, None) == 0 and P.i4s_mx_read(none, 0, None, None) == 0
    assert P.i4s_mx_product(product(tokens=0), None) == 0 and P.i4s_mx_product(product(w=none, y_stride=0), None) == 0
    for change in (dict(num_tokens=0), dict(num_seqs=0)):
        assert P.i4s_prompt_attention(attention(**change), None) == 0


# ---------------------------------------------------------------------------
# products


def product(w=mx(), x=None, **kw):
    a = P.i4s_mx_product_args()
    a._keep = (w, x)
    a.w = None if w is None else ctypes.addressof(w)
    a.x = None if x is None else ctypes.addressof(x)
    a.x_values, a.x_stride, a.x_dtype, a.tokens = 3 * GIB, 64, 0, 50
    a.y, a.y_stride, a.y_dtype = 4 * GIB, 20, 0
    a.workspace, a.workspace_bytes = 5 * GIB, GIB
    for k, v in kw.items():
        setattr(a, k, v)
    return a


GIVEN = dict(x=mx(50, 64, 6 * GIB, 7 * GIB))


@pytest.mark.parametrize("change", [
    dict(w=None), dict(w=mx(rows=-1)), dict(w=mx(cols=33)), dict(w=mx(vals=None)), dict(w=mx(scales=2 * GIB + 8)),
    dict(x=mx(49, 64, 6 * GIB, 7 * GIB)), dict(x=mx(50, 96, 6 * GIB, 7 * GIB)), dict(x=mx(50, 64, None, 7 * GIB)),
    dict(x=mx(50, 64, 6 * GIB, 7 * GIB + 1)), dict(x_values=None), dict(x_values=3 * GIB + 2), dict(x_stride=56),
    dict(x_stride=65), dict(x_stride=(1 << 40) + 8), dict(x_dtype=2), dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(y=None),
    dict(y=4 * GIB + 1), dict(y_dtype=2, y=4 * GIB + 2), dict(y_dtype=3), dict(y_stride=19), dict(y_stride=(1 << 40) + 1),
    dict(reserved=1), dict(workspace=None), dict(workspace=5 * GIB + 8), dict(y=GIB), dict(y=2 * GIB), dict(y=3 * GIB),
    dict(y=5 * GIB), dict(workspace=3 * GIB), dict(workspace=GIB), dict(GIVEN, y=6 * GIB), dict(GIVEN, y=7 * GIB),
    dict(w=mx(1 << 24, 32), tokens=1 << 24, y_stride=1 << 24)])
def test_product_refuses(lib, change):
    assert P.i4s_mx_product(product(**change), None) == BAD and B.i4s_last_error()


def test_product_workspace(lib):
    n = ctypes.c_uint64()
    size = lambda **kw: (P.i4s_mx_product_workspace_size(product(**kw), n), n.value)[1]  # noqa: E731
    assert size() == 4 * 2048 + 4 * 256 and size(**GIVEN) == 0 and size(tokens=16) == 0 and size(tokens=0) == 0
    assert size(w=mx(20, 8192), tokens=8) == 64 * 1024 + 16 * 256 and size(w=mx(20, 8192), tokens=7) == 0
    assert P.i4s_mx_product(product(workspace_bytes=4 * 2048 + 4 * 256 - 1), None) == SMALL
    assert P.i4s_mx_product_workspace_size(product(), None) == BAD
    assert P.i4s_mx_product_workspace_size(None, n) == BAD and P.i4s_mx_product(None, None) == BAD
    assert P.i4s_mx_product_workspace_size(product(w=mx(cols=16)), n) == BAD


def test_product_workspace_looks_only_whether_x_is_given(lib):
    """The tokens in the format need no workspace, whatever their descriptor holds at this time."""
    n = ctypes.c_uint64(7)
    for x in (P.i4s_mx(), mx(49, 96, None, None)):
        assert P.i4s_mx_product_workspace_size(product(x=x), n) == 0 and n.value == 0
        assert P.i4s_mx_product(product(x=x), None) == BAD  # the call looks at it
    a = product()
    a.x = 8  # nothing lies there
    assert P.i4s_mx_product_workspace_size(a, n) == 0 and n.value == 0


@pytest.mark.parametrize("tokens,rows,cols,ok", [(1 << 24, 63 * 128, 32, True), (1 << 24, 63 * 128 + 1, 32, False),
                                                 (63 * 128, 1 << 24, 32, True), (63 * 128 + 1, 1 << 24, 32, False),
                                                 (16 * 16383, 16, 1 << 20, True), (16 * 16384, 16, 1 << 20, False),
                                                 (16 * ((1 << 20) - 1), 16, 32 * 512, True), (16 << 20, 16, 32 * 512, False)])
@pytest.mark.parametrize("given", [False, True])
def test_product_limits(lib, tokens, rows, cols, ok, given):
    """The bounds of sizes together, as the header states them."""
    text = " ".join(re.sub(r"\n \* ?", " ", open(HEADER).read()).split())
    assert "ceil(tokens/128) * ceil(rows/128) is at most 2^23 - 1" in text
    assert "ceil(rows/16) * ceil(cols/512) <= 2^25 - 4" in text
    n = ctypes.c_uint64()
    a = product(w=mx(rows, cols), x=mx(tokens, cols, 6 * GIB, 7 * GIB) if given else None, tokens=tokens)
    assert P.i4s_mx_product_workspace_size(a, n) == (0 if ok else BAD)


# ---------------------------------------------------------------------------
# attention of whole prompts


def attention(**kw):
    a = P.i4s_prompt_args()
    a.q, a.k, a.v = GIB, 2 * GIB, 3 * GIB
    a.q_token_stride, a.q_head_stride = 256, 64
    a.k_token_stride = a.v_token_stride = 128
    a.k_head_stride = a.v_head_stride = 64
    a.dtype, a.head_dim, a.q_heads, a.kv_heads = 0, 64, 4, 2
    a.num_tokens, a.num_keys, a.num_seqs, a.max_q, a.max_k, a.causal, a.scale = 10, 5000, 3, 4, 0, 1, 0.125
    a.q_start, a.k_start, a.out, a.lse = 4 * GIB, 5 * GIB, 6 * GIB, 7 * GIB
    a.workspace, a.workspace_bytes = 8 * GIB, GIB
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=GIB + 8), dict(k=None), dict(k=2 * GIB + 2), dict(v=None), dict(v=3 * GIB + 8), dict(q_token_stride=4),
    dict(q_head_stride=-8), dict(k_token_stride=(1 << 23) + 8), dict(k_head_stride=60), dict(v_token_stride=-128),
    dict(v_head_stride=(1 << 40) + 8), dict(dtype=2), dict(dtype=-1), dict(head_dim=32), dict(head_dim=96), dict(head_dim=512),
    dict(q_heads=0), dict(q_heads=3), dict(q_heads=65538), dict(kv_heads=0), dict(kv_heads=1025, q_heads=1025), dict(num_tokens=-1),
    dict(num_tokens=(1 << 30) + 1), dict(num_keys=-1), dict(num_keys=(1 << 30) + 1), dict(num_seqs=-1), dict(num_seqs=65536),
    dict(max_q=0), dict(max_q=(1 << 24) + 1), dict(max_k=-1), dict(causal=2), dict(causal=-1), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(reserved=1), dict(q_start=None), dict(q_start=4 * GIB + 2),
    dict(k_start=None), dict(k_start=5 * GIB + 1), dict(q_start=None, k_start=None), dict(out=None), dict(out=6 * GIB + 8), dict(lse=7 * GIB + 2), dict(out=GIB),
    dict(out=2 * GIB), dict(out=3 * GIB), dict(out=4 * GIB), dict(lse=6 * GIB), dict(lse=5 * GIB), dict(workspace=None),
    dict(workspace=8 * GIB + 4), dict(workspace=6 * GIB), dict(workspace=GIB), dict(num_seqs=65535, max_q=1 << 13)])
def test_attention_refuses(lib, change):
    assert P.i4s_prompt_attention(attention(**change), None) == BAD and B.i4s_last_error()


def test_attention_workspace(lib):
    n = ctypes.c_uint64()
    assert P.i4s_prompt_attention_workspace_size(attention(), n) == 0
    pieces, rest = divmod(n.value, 10 * 4 * (64 + 2) * 4)
    assert pieces > 1 and not rest
    assert P.i4s_prompt_attention(attention(workspace_bytes=n.value - 1), None) == SMALL
    for change in (dict(num_keys=500), dict(num_tokens=0), dict(num_seqs=0), dict(max_k=512)):
        assert P.i4s_prompt_attention_workspace_size(attention(**change), n) == 0 and n.value == 0
    assert P.i4s_prompt_attention_workspace_size(attention(), None) == BAD
    assert P.i4s_prompt_attention_workspace_size(None, n) == BAD and P.i4s_prompt_attention(None, None) == BAD
    assert P.i4s_prompt_attention_workspace_size(attention(head_dim=80), n) == BAD
