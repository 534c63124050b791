"""The prompt's operators on the GPU against their float64 definitions
(``oracle/prompt_oracle.py``): the microscaled format, products in it,
attention over whole prompts, and a step that runs them together.

Tolerances come from the arithmetic.  The microscaled format is exact: codes
and scale bytes are equal.  A value rounded to a type is off by at most half a
step, ``eps / 2`` of itself, or half of the smallest subnormal.  A product of
two held values is exact, and an fp32 sum of K of them in any order is off by
at most K roundings, each 2^-24 of what the sum of magnitudes is; the matrix
instruction adds 128 at a time, aligned, with at least fp32's 24 bits: K / 32 + 8
steps of 2^-23 of the sum of magnitudes are allowed.

Scores of attention are such sums of D products: off by at most (D + 4) 2^-24
scale sum |q| |k|, and a score off by d moves a probability by a factor exp(2d)
at most.  Probabilities are rounded to the type (half a step of each; below
fp16's normal range by 2^-25, where a row's largest probability is 2^7 at
least: 2^-32 of it), sums over n keys by n 2^-24, and so is the running
rescaling, once a step of 32 keys: (n + 8) 2^-23 covers both.
"""

import numpy as np
import pytest

from oracle import prompt_oracle as O
from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def i4s():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int4_sparse_gemv_amd as I
    return I


def say(*a):
    print(*a, flush=True)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half of the smallest subnormal."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def draw(rng, rows, cols, dtype, spread=2.0):
    x = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal(cols)))
    return x.to(dtype).cuda()


# ---------------------------------------------------------------------------
# the microscaled format


def check_format(i4s, x):
    m = i4s.mx_quantize(x)
    rows, cols = x.shape
    code, scale = O.mx_quantize(f64(x))
    got = O.mx_unpack(m.vals.cpu().numpy().reshape(-1), m.scales.cpu().numpy().reshape(-1), rows, cols)
    np.testing.assert_array_equal(got[1], scale)
    np.testing.assert_array_equal(got[0], code)
    want = O.mx_values(code, scale)
    for dtype in (F32, BF16, F16):
        y = i4s.mx_read(m, dtype)
        rounded = torch.from_numpy(want).to(dtype)  # exact in fp32 and bf16; to fp16 the one rounding
        assert torch.equal(y.cpu().nan_to_num(7.0), rounded.nan_to_num(7.0))
        assert torch.equal(y.cpu().isnan(), rounded.isnan())
    # what lies past the columns is 0
    full = O.mx_unpack(m.vals.cpu().numpy().reshape(-1), m.scales.cpu().numpy().reshape(-1), rows, -(-cols // 256) * 256)
    assert not full[0][:, cols:].any() and not full[1][:, cols // 32:].any()
    return m


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (16, 128), (17, 256), (15, 544), (33, 512), (64, 1056),
                                       (257, 4096), (5, 11008)])
def test_quantize(i4s, rows, cols, dtype):
    say("quantize", rows, cols, dtype)
    rng = np.random.default_rng(rows + cols)
    check_format(i4s, draw(rng, rows, cols, dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_value_beside_every_scale(i4s, dtype):
    """All finite values of the type, alone in their block and beside each of 16 powers of two."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    bits = bits[torch.isfinite(bits)]
    bits = bits[:bits.numel() // 16 * 16]
    top = torch.tensor([2.0 ** k for k in range(-14, 16, 2)] + [0.0]).to(dtype)
    x = torch.zeros(16, bits.numel() // 16, 32, dtype=dtype)
    for r in range(16):
        v = bits.view(-1, 16)
        x[r, :, 0:32:2] = v
        x[r, :, 1] = top[r] if r < 15 else 0
    alone = torch.zeros(bits.numel(), 32, dtype=dtype)
    alone[:, 9] = bits
    check_format(i4s, x.reshape(16 * 8, -1)[:, :x[0].numel() // 8 // 32 * 32].cuda())
    check_format(i4s, alone.view(-1, 64).cuda())


def test_ties_signs_and_zeros(i4s):
    row = [6, 5, -5, 3.5, -3.5, 2.5, -2.5, 1.75, -1.75, 1.25, -1.25, 0.75, -0.75, 0.25, -0.25, 0.0, -0.0, 7.9, -7.9, 4.5,
           0.2, -0.2, 0.26, 0.74, 0.76, 1.24, 1.26, 1.74, 1.76, 2.4, 2.6, 3.4]
    x = torch.tensor([row, [0.0] * 32, [-0.0] * 32, [2.0 ** -24] * 32], dtype=F16).cuda()
    m = check_format(i4s, x)
    y = i4s.mx_read(m, F32).cpu()
    assert torch.equal(torch.signbit(y[:3]), torch.signbit(x[:3].cpu()))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_block_that_is_not_finite(i4s, dtype, bad):
    rng = np.random.default_rng(5)
    x = draw(rng, 18, 256, dtype)
    x[3, 40] = bad
    x[17, 255] = bad
    m = check_format(i4s, x)
    w = i4s.mx_quantize(draw(rng, 24, 256, dtype))
    for tokens in (m, x):
        y = i4s.mx_product(tokens, w, dtype=F32)
        gone = y.isnan().all(1)
        assert gone.nonzero().flatten().tolist() == [3, 17] and not y[~gone].isnan().any()
    y = i4s.mx_product(w, m, dtype=F32)
    assert y.isnan().all(0).nonzero().flatten().tolist() == [3, 17] and int(y.isnan().sum()) == 2 * 24


def test_strided_rows_and_a_given_tensor(i4s):
    rng = np.random.default_rng(6)
    wide = draw(rng, 37, 1024, BF16)
    m = check_format(i4s, wide[:, 320:320 + 416])
    x = draw(rng, 37, 416, BF16)
    again = i4s.mx_quantize(x, out=m)
    assert again is m
    code, scale = O.mx_quantize(f64(x))
    np.testing.assert_array_equal(f64(i4s.mx_read(m, F32)), O.mx_values(code, scale))
    # rows past the last are not written
    vals, scales = torch.full_like(m.vals, 0xA5), torch.full_like(m.scales, 0xA5)
    part = i4s.MXTensor(37, 416, vals, scales)
    i4s.mx_quantize(x, out=part)
    byte, _, at = O.mx_places(48, 416)
    assert (vals.cpu().numpy().reshape(-1)[byte[37:]] == 0xA5).all()
    assert (scales.cpu().numpy().reshape(-1)[at[37:]] == 0xA5).all()


def test_no_rows(i4s):
    m = i4s.mx_quantize(torch.empty(0, 64, dtype=F16, device="cuda"))
    assert i4s.mx_read(m).shape == (0, 64)
    w = i4s.mx_quantize(torch.ones(20, 64, dtype=F16, device="cuda"))
    assert i4s.mx_product(m, w).shape == (0, 20) and i4s.mx_product(w, m).shape == (20, 0)
    assert i4s.mx_product(torch.empty(0, 64, dtype=BF16, device="cuda"), w).dtype == BF16


# ---------------------------------------------------------------------------
# products


def check_product(i4s, x, w, y, dtype):
    """y against the product of what the two tensors hold."""
    xv, wv = f64(i4s.mx_read(x, F32)), f64(i4s.mx_read(w, F32))
    want, size = O.product(xv, wv)
    tol = (x.cols / 32 + 8) * 2.0 ** -23 * size + least(F32)
    if dtype != F32:
        tol = tol * 1.01 + half_step(dtype) * np.abs(want) + least(dtype)
    far = np.abs(f64(y) - want)
    assert y.dtype == dtype and (far <= tol).all(), (float((far / tol).max()), np.argwhere(far > tol)[:5])


SIZES = [(1, 16, 32), (1, 4096, 4096), (2, 33, 96), (5, 1000, 512), (15, 77, 1056), (16, 256, 4096), (17, 100, 288),
         (31, 513, 768), (33, 48, 1024), (50, 300, 2080), (64, 129, 512), (65, 127, 256), (65, 1, 64), (100, 257, 544),
         (128, 128, 128), (129, 400, 1312), (257, 640, 992), (300, 31, 4096), (511, 513, 800), (3, 8300, 512), (15, 16400, 224),
         (16, 9000, 4096),
         (16, 500, 8224), (11, 129, 8192), (9, 4100, 5120)]


@pytest.mark.parametrize("tokens,rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_product(i4s, tokens, rows, cols, dtype):
    say("product", tokens, rows, cols, dtype)
    rng = np.random.default_rng(tokens + rows + cols)
    x = draw(rng, tokens, cols, dtype, 0.7)
    w = i4s.mx_quantize(draw(rng, rows, cols, dtype, 0.3) * 0.05)
    xq = i4s.mx_quantize(x)
    for out in (dtype, F32):
        y = i4s.mx_product(xq, w, dtype=out)
        check_product(i4s, xq, w, y, out)
        assert torch.equal(i4s.mx_product(x, w, dtype=out), y)  # quantized within the call: the same bits
    assert torch.equal(i4s.mx_product(xq, w, dtype=F32), y)     # and again


@pytest.mark.parametrize("tokens,rows,cols", [(4096, 4096, 1024), (2049, 8200, 544), (1100, 1501, 288), (1023, 1399, 1312),
                                              (3897, 3801, 288), (3900, 3900, 96), (511, 4033, 1312), (383, 5003, 288), (100, 16300, 96)])
def test_product_many(i4s, tokens, rows, cols):
    """The largest blocks, whole and ragged."""
    say("product", tokens, rows, cols)
    rng = np.random.default_rng(tokens)
    x = i4s.mx_quantize(draw(rng, tokens, cols, BF16, 0.7))
    w = i4s.mx_quantize(draw(rng, rows, cols, BF16, 0.3))
    for out in (F32, BF16, F16):
        check_product(i4s, x, w, i4s.mx_product(x, w, dtype=out), out)


@pytest.mark.parametrize("tokens", [1, 16, 20, 70])
def test_product_strides(i4s, tokens):
    """Strided tokens, strided outputs, odd rows: what lies between is left as it was."""
    rng = np.random.default_rng(tokens)
    wide = draw(rng, tokens, 1000, F16, 0.7)
    x, w = wide[:, 200:200 + 640], i4s.mx_quantize(draw(rng, 83, 640, F16, 0.3))
    xq = i4s.mx_quantize(x)
    buf = torch.full((tokens + 1, 131), 7.0, dtype=F32, device="cuda")
    y = i4s.mx_product(x, w, out=buf[:tokens, 9:9 + 83])
    check_product(i4s, xq, w, y, F32)
    keep = buf.clone()
    keep[:tokens, 9:92] = 7.0
    assert (keep == 7.0).all()


@pytest.mark.parametrize("tokens,rows,wide", [(1100, 1501, 1511), (3897, 3801, 3805), (401, 4001, 4005), (1200, 4401, 4405)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_product_many_at_odd_places(i4s, tokens, rows, wide, dtype):
    """Outputs of the largest blocks at odd offsets and strides: the same values, and what lies between stays."""
    rng = np.random.default_rng(rows)
    x, w = (i4s.mx_quantize(draw(rng, n, 160, F16, 0.3)) for n in (tokens, rows))
    buf = torch.full((tokens, wide), 7.0, dtype=dtype, device="cuda")
    y = i4s.mx_product(x, w, out=buf[:, 3:3 + rows])
    assert torch.equal(y, i4s.mx_product(x, w, dtype=dtype))
    assert (buf[:, :3] == 7.0).all() and (buf[:, 3 + rows:] == 7.0).all()


@pytest.mark.parametrize("tokens,rows", [(3, 40), (40, 300), (400, 4000), (1100, 1501), (1200, 4400), (3900, 3900)])
def test_product_with_a_block_that_is_not_finite(i4s, tokens, rows):
    """Its token, or its weight row, gets NaN; nothing else changes."""
    rng = np.random.default_rng(tokens)
    x, w = draw(rng, tokens, 96, F16, 0.3), draw(rng, rows, 96, F16, 0.3)
    x[0, 5], x[tokens - 1, 95], w[rows - 2, 40] = float("nan"), float("inf"), float("-inf")
    xc, wc = x.clone(), w.clone()
    xc[0, 5], xc[tokens - 1, 95], wc[rows - 2, 40] = 0, 0, 0
    y = i4s.mx_product(x, i4s.mx_quantize(w), dtype=F32)
    want = i4s.mx_product(xc, i4s.mx_quantize(wc), dtype=F32)
    want[0], want[tokens - 1], want[:, rows - 2] = float("nan"), float("nan"), float("nan")
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(3.0), want.nan_to_num(3.0))


def test_product_long_offsets(i4s):
    """A weight past 4 GB, and tokens and outputs whose strides pass it."""
    say("long offsets")
    rows, cols = 1 << 17, 65568
    sizes = ((rows // 16, 2 * -(-cols // 256), 1024), (rows // 16, -(-cols // 512), 256))
    w = i4s.MXTensor(rows, cols, torch.randint(256, sizes[0], dtype=torch.uint8, device="cuda"),
                     torch.full(sizes[1], 120, dtype=torch.uint8, device="cuda"))
    assert w.vals.numel() > 1 << 32
    w.vals[:, -1], w.scales[:, -1] = 0, 0  # past the columns
    w.vals[:, 512, 256:], w.scales[:, 128] = 0, 0
    w.scales[:, 128, 0:64:4] = 120  # the last block of 32
    rng = np.random.default_rng(1)
    for tokens in (3, 80, 300):
        x, out = (torch.empty(tokens, 1 << 24, dtype=F16, device="cuda")[:, 64:64 + n] for n in (cols, rows))
        x.copy_(draw(rng, tokens, cols, F16, 0.2))
        i4s.mx_product(x, w, out=out)
        # the last tiles by themselves
        tail = i4s.MXTensor(48, cols, w.vals[-3:].clone(), w.scales[-3:].clone())
        check_product(i4s, i4s.mx_quantize(x), tail, out[:, -48:], F16)
        del x, out


# ---------------------------------------------------------------------------
# attention of whole prompts


def packed(rng, lengths, heads, share, dim, dtype, fused=False, pad=0):
    nq, nk = [a for a, _ in lengths], [b for _, b in lengths]
    starts = [torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32).cuda() for x in (nq, nk)]
    def make(n, h):
        return torch.from_numpy(rng.standard_normal((n + pad, h, dim))).to(dtype).cuda()
    if fused:
        big = make(sum(nq), heads * (share + 2))
        q, k, v = big.split((heads * share, heads, heads), 1)
    else:
        q, k, v = make(sum(nq), heads * share), make(sum(nk), heads), make(sum(nk), heads)
    return q, k, v, starts


def check_attention(q, k, v, starts, out, lse, causal, scale, dtype):
    at = [s.tolist() for s in starts]
    qn, kn, vn = f64(q), f64(k), f64(v)
    dim, u = q.shape[2], half_step(dtype)
    for i in range(len(at[0]) - 1):
        a, b, c, d = at[0][i], at[0][i + 1], at[1][i], at[1][i + 1]
        want, want_lse, spread = O.attention(qn[a:b], kn[c:d], vn[c:d], causal, scale)
        if b == a:
            continue
        share = q.shape[1] // k.shape[1]
        size = np.abs(kn[c:d]).max(0) if d > c else np.zeros(k.shape[1:])   # [kv_heads, D]
        reach = scale * (np.abs(qn[a:b]) * np.repeat(size, share, 0)).sum(-1)
        delta = (dim + 4) * 2.0 ** -24 * reach
        biggest = np.repeat(np.abs(vn[c:d]).max(0), share, 0) if d > c else 0.0
        n = max(d - c, 1)
        rel = np.expm1(2 * delta)[..., None] + u + (n + 8) * 2.0 ** -23
        tol = spread * rel * 1.01 + u * np.abs(want) + least(dtype)
        if dtype == F16:
            tol = tol + 2.0 ** -32 * n * biggest
        far = np.abs(f64(out[a:b]) - want)
        assert (far <= tol).all(), (i, float((far / tol).max()), np.argwhere(far > tol)[:4])
        if lse is not None:
            got = f64(lse[a:b])
            tol = delta + (n + 8) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(np.isfinite(want_lse), want_lse, 0)) + 2e-6
            same = np.isneginf(want_lse) == np.isneginf(got)
            with np.errstate(invalid="ignore"):
                assert same.all() and (np.isneginf(got) | (np.abs(got - want_lse) <= tol)).all()


BATCHES = {
    "one": [(1, 1)], "few": [(3, 3)], "tile": [(64, 64)], "past": [(65, 65)], "odd": [(61, 61), (1, 1), (0, 0), (130, 130)],
    "chunk": [(33, 97), (5, 200), (64, 64)], "token": [(1, 700)], "tokens": [(1, 65), (1, 1), (2, 300)],
    "none": [(40, 7), (3, 0), (70, 64)], "long": [(300, 300)],
}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("heads,share,dim", [(1, 1, 128), (2, 4, 64), (2, 5, 128), (1, 7, 256), (8, 1, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention(i4s, batch, heads, share, dim, dtype):
    say("attention", batch, heads, share, dim, dtype)
    rng = np.random.default_rng(len(batch) + heads + dim)
    lengths = BATCHES[batch]
    q, k, v, starts = packed(rng, lengths, heads, share, dim, dtype)
    for causal in (True, False):
        lse = torch.full(q.shape[:2], 5.0, device="cuda")
        out = i4s.prompt_attention(q, k, v, *starts, max_q=max(a for a, _ in lengths), max_k=max(max(b for _, b in lengths), 1),
                                   causal=causal, lse=lse)
        check_attention(q, k, v, starts, out, lse, causal, dim ** -0.5, dtype)
        again = i4s.prompt_attention(q, k, v, *starts, causal=causal)  # sizes from the tensors: another launch
        check_attention(q, k, v, starts, again, None, causal, dim ** -0.5, dtype)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("share,length", [(1, 5000), (4, 3001), (8, 2048)])
def test_attention_of_one_token_over_many_keys(i4s, dim, share, length):
    rng = np.random.default_rng(dim + length)
    q, k, v, starts = packed(rng, [(1, length), (1, 10), (1, length // 2)], 2, share, dim, BF16)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = i4s.prompt_attention(q, k, v, *starts, max_q=1, max_k=length, lse=lse)
    check_attention(q, k, v, starts, out, lse, True, dim ** -0.5, BF16)


def test_attention_strides_and_rows_outside(i4s):
    """Slices of a fused product, padding behind the last sequence, tokens past max_q."""
    rng = np.random.default_rng(3)
    lengths = [(40, 40), (70, 70), (9, 9)]
    q, k, v, starts = packed(rng, lengths, 2, 3, 128, F16, fused=True, pad=13)
    starts[0] = starts[0].clone()
    out = torch.full(q.shape, 3.0, dtype=F16, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    assert i4s.prompt_attention(q, k, v, starts[0], max_q=70, out=out, lse=lse) is out
    check_attention(q, k, v, starts, out, lse, True, 128 ** -0.5, F16)
    assert (out[119:] == 3.0).all() and (lse[119:] == 3.0).all()
    short = torch.full(q.shape, 3.0, dtype=F16, device="cuda")
    i4s.prompt_attention(q, k, v, starts[0], max_q=41, out=short)
    assert torch.equal(short[:40], out[:40]) and torch.equal(short[40:81], out[40:81]) and (short[81:110] == 3.0).all()
    one = i4s.prompt_attention(q[:40], k[:40], v[:40])
    assert torch.equal(one, out[:40])


def test_attention_broadcast_heads_and_tokens(i4s):
    """Strides of zero: one head, or one token, for all."""
    rng = np.random.default_rng(4)
    q, k, v, starts = packed(rng, [(50, 50)], 1, 4, 64, BF16)
    wide_k, wide_v = k.expand(50, 4, 64), v[:1].expand(50, 4, 64)
    out = i4s.prompt_attention(q, wide_k, wide_v, *starts)
    check_attention(q, wide_k, wide_v, starts, out, None, True, 64 ** -0.5, BF16)


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, F16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_a_token_does_not_see_does_not_matter(i4s, dim, dtype, bad):
    rng = np.random.default_rng(dim)
    lengths = [(100, 100), (50, 80), (30, 30)]
    q, k, v, starts = packed(rng, lengths, 2, 2, dim, dtype)
    clean = i4s.prompt_attention(q, k, v, *starts, max_q=100, max_k=100)
    for where in (k, v):
        keep = where.clone()
        where[70, 1, 5] = bad     # sequence 0: tokens from 70 on, heads of KV head 1
        where[179, :, 7] = bad    # the last key of sequence 1: its last token
        where[180, 0, :] = bad    # the first of sequence 2: all of its tokens, heads of KV head 0
        out = i4s.prompt_attention(q, k, v, *starts, max_q=100, max_k=100)
        hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        hit[70:100, 2:] = True
        hit[149] = True
        hit[150:, :2] = True
        assert torch.equal(out[~hit], clean[~hit])
        if where is v:
            part = torch.zeros_like(out, dtype=torch.bool)
            part[70:100, 2:, 5] = part[149, :, 7] = part[150:, :2, :] = True
            assert torch.equal(out[~part], clean[~part])
            got = out[part].float()
            assert got.isnan().all() if bad != bad else (got == bad).all()
        elif bad != bad:
            assert out[hit].isnan().all()
        where.copy_(keep)


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 30.0, 1e30])
def test_attention_scales_and_far_scores(i4s, scale):
    rng = np.random.default_rng(9)
    q, k, v, starts = packed(rng, [(90, 90), (3, 200)], 1, 2, 128, BF16)
    q, k = (q * 0 + torch.randint(-1, 2, q.shape, device="cuda")).to(BF16), (torch.randint(-2, 3, k.shape, device="cuda")).to(BF16)
    k = k + 1000.0 * (scale == 1e-3)  # whole-number scores: exact
    out = i4s.prompt_attention(q, k, v, *starts, scale=scale)
    assert out.isfinite().all()
    at = [s.tolist() for s in starts]
    for i in range(2):
        a, b, c, d = at[0][i], at[0][i + 1], at[1][i], at[1][i + 1]
        want, _, spread = O.attention(f64(q[a:b]), f64(k[c:d]), f64(v[c:d]), True, float(np.float32(scale)))
        # the exponent is a whole-number difference times scale log2(e) in fp32: 2 roundings, where it matters below 2^7
        tol = spread * (half_step(BF16) + 200 * 2.0 ** -23 + 2.0 ** -15) * 1.01 + half_step(BF16) * np.abs(want)
        assert (np.abs(f64(out[a:b]) - want) <= tol).all()


def test_starts_outside_the_tensors(i4s):
    """Moved into range; a sequence that ends before it begins is empty; a row that two claim has values of either."""
    rng = np.random.default_rng(2)
    q, k, v, _ = packed(rng, [(60, 60)], 2, 1, 64, F16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    out = torch.full(q.shape, 3.0, dtype=F16, device="cuda")
    i4s.prompt_attention(q, k, v, i32(-5, 20, 10, 100), max_q=60, out=out)
    a, b = i4s.prompt_attention(q[:20], k[:20], v[:20]), i4s.prompt_attention(q[10:], k[10:], v[10:])
    assert torch.equal(out[:10], a[:10]) and torch.equal(out[20:], b[10:])
    assert ((out[10:20] == a[10:]) | (out[10:20] == b[:10])).all()
    none = i4s.prompt_attention(q, k, v, i32(0, 60), i32(2 ** 31 - 1, -2 ** 31))
    assert (none == 0).all()


def test_attention_without_tokens_or_keys(i4s):
    z = lambda n, h: torch.zeros(n, h, 64, dtype=F16, device="cuda")  # noqa: E731
    assert i4s.prompt_attention(z(0, 2), z(5, 1), z(5, 1)).shape == (0, 2, 64)
    lse = torch.zeros(3, 2, device="cuda")
    out = i4s.prompt_attention(z(3, 2) + 1, z(0, 1), z(0, 1), lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16)])
def test_attention_of_many_pairs(i4s, dim, dtype):
    """More pairs of sequence and KV head than run together, rows of very different lengths among them."""
    say("pairs", dim, dtype)
    rng = np.random.default_rng(dim)
    lengths = [(610, 610)] + [(n, n) for n in (1, 40, 33, 128, 129, 7, 64, 65, 2)] + [(30, 300)]
    q, k, v, starts = packed(rng, lengths, 8, 4, dim, dtype)
    out = i4s.prompt_attention(q, k, v, *starts, max_q=610, max_k=610)
    check_attention(q, k, v, starts, out, None, True, dim ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_of_large_blocks(i4s, dtype):
    """Enough long rows for the largest blocks, and short, empty and odd sequences beside them; then values that are not
    finite where tokens do not see them."""
    say("large blocks", dtype)
    rng = np.random.default_rng(16)
    lengths = [(300, 6200), (3, 0), (40, 7), (33, 900), (1, 1), (256, 256), (257, 300)] + [(n, n) for n in range(38)]
    q, k, v, starts = packed(rng, lengths, 2, 4, 128, dtype)
    outs = []
    for causal in (True, False):
        lse = torch.empty(q.shape[:2], device="cuda")
        outs.append(i4s.prompt_attention(q, k, v, *starts, max_q=300, max_k=6200, causal=causal, lse=lse))
        check_attention(q, k, v, starts, outs[-1], lse, causal, 128 ** -0.5, dtype)
    again = i4s.prompt_attention(q, k, v, *starts, max_q=300, max_k=6200)
    assert torch.equal(again, outs[0])
    k[6190, 1], v[6100, 0], v[6199, 1, 60:] = float("nan"), float("inf"), float("nan")
    out = i4s.prompt_attention(q, k, v, *starts, max_q=300, max_k=6200)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit[290:300, 4:], hit[200:300, :4] = True, True
    assert torch.equal(out[~hit], outs[0][~hit])
    assert out[290:300, 4:].isnan().all() and (out[200:300, :4] == float("inf")).all()
    k[6190, 1] = 0
    plain = i4s.prompt_attention(q, k, v, *starts, max_q=300, max_k=6200)
    assert plain[299, 4:, 60:].isnan().all() and plain[299, 4:, :60].isfinite().all() and plain[:299, 4:].isfinite().all()


@pytest.mark.parametrize("max_k", [0, 1, 1000, 3001])
@pytest.mark.parametrize("tokens", [1, 20, 100])
def test_attention_split_over_blocks(i4s, tokens, max_k):
    """Long keys in pieces, and a largest length that is not given, or too small: the same within the tolerance."""
    rng = np.random.default_rng(tokens)
    q, k, v, starts = packed(rng, [(tokens, 3001), (tokens, tokens), (2, 0)], 1, 2, 128, F16)
    for causal in (True, False):
        lse = torch.empty(q.shape[:2], device="cuda")
        out = i4s.prompt_attention(q, k, v, *starts, max_q=max(tokens, 2), max_k=max_k, causal=causal, lse=lse)
        check_attention(q, k, v, starts, out, lse, causal, 128 ** -0.5, F16)


def test_attention_long_offsets(i4s):
    """Keys, values and queries whose strides pass 4 GB."""
    say("long offsets")
    rng = np.random.default_rng(8)
    q, k, v, starts = packed(rng, [(5, 5), (290, 290)], 1, 2, 64, BF16)
    step = 1 << 23
    big = torch.empty(295, step, dtype=BF16, device="cuda")
    far = [big[:, at:at + n * 64].unflatten(1, (n, 64)) for at, n in ((0, 2), (step // 2, 1), (step - 64, 1))]
    for a, b in zip(far, (q, k, v)):
        a.copy_(b)
    assert big.numel() * 2 > 1 << 32
    out = i4s.prompt_attention(*far, *starts, max_q=290, max_k=290)
    assert torch.equal(out, i4s.prompt_attention(q, k, v, *starts, max_q=290, max_k=290))
    check_attention(q, k, v, starts, out, None, True, 64 ** -0.5, BF16)
    token = i4s.prompt_attention(far[0][-1:], far[1], far[2])
    want = [torch.tensor(x, dtype=torch.int32) for x in ([0, 1], [0, 295])]
    check_attention(q[-1:], k, v, want, token, None, True, 64 ** -0.5, BF16)


# ---------------------------------------------------------------------------
# calls together


def prompt_step(i4s, lengths, seed=0):
    import bench
    return bench.PromptStep(i4s, lengths, seed=seed, hidden=512, heads=8, kv_heads=2, mlp=1408, vocab=1000)


def test_prompt_step_then_a_decode_step(i4s):
    """The step that ``bench.py --prompt-step`` times, on a small layer and three requests, each part against the oracle on
    its own inputs; then each request's next token over the cache that the prompts left."""
    say("prompt step")
    s = prompt_step(i4s, [70, 1, 33])
    a, y, scores = s.run()
    torch.cuda.synchronize()
    q, k, v = s.project()
    check_product(i4s, i4s.mx_quantize(s.x), s.qkv, torch.cat([t.flatten(1) for t in (q, k, v)], 1), F16)
    r = s.extend()
    assert int(r.flags) == 0 and r.q_start.tolist() == [0, 70, 71, 104]
    starts = [r.q_start.cpu()] * 2
    check_attention(q, k, v, starts, a.unflatten(1, (8, 64)), None, True, 0.125, F16)
    gate_up = i4s.mx_product(i4s.mx_product(a, s.o), s.gate_up)
    check_product(i4s, i4s.mx_quantize(i4s.mx_product(a, s.o)), s.gate_up, gate_up, F16)
    check_product(i4s, i4s.mx_quantize(gate_up[:, :1408] * gate_up[:, 1408:]), s.down, y, F16)
    logits = i4s.mx_product(y[[69, 70, 103]], s.head)
    lp, ent, ids, top = S.token_logprobs(f64(logits), s.given.cpu().numpy(), 8)
    np.testing.assert_array_equal(scores.top_ids.cpu().numpy(), ids)
    np.testing.assert_allclose(f64(scores.logprobs), lp, rtol=2.0**-20)  # sums of 1000 terms
    # the cache holds what the attention read, in 4 bits
    keys, values = i4s.kv_read(s.cache, r.slots, dtype=F32)
    for got, x in ((keys, k), (values, v)):
        n, f = S.quantize(f64(x), 64)
        np.testing.assert_array_equal(f64(got), n * f.repeat(64, -1))
    # the next token of each
    new = torch.ones(3, dtype=torch.int32, device="cuda")
    q, k, v = s.project(s.x[:3])
    n = i4s.kv_extend(s.table, r.lens, new, s.free, r.free_count, s.PAGE, 3)
    assert int(n.flags) == 0 and n.lens.tolist() == [71, 2, 34]
    i4s.kv_append(s.cache, k, v, n.slots)
    out = i4s.kv_attention(s.cache, q, s.table, n.lens, q_start=n.q_start, max_q=1)
    slots = r.slots.tolist()
    for i, (b, e) in enumerate(((0, 70), (70, 71), (71, 104))):
        held = torch.tensor(slots[b:e] + [n.slots.tolist()[i]], dtype=torch.int32).cuda()
        keys, values = i4s.kv_read(s.cache, held, dtype=F32)
        want, _, spread = S.attention(f64(q[i:i + 1]), f64(keys), f64(values), e - b, 0.125)
        assert (np.abs(f64(out[i:i + 1]) - want) <= half_step(F16) * np.abs(want) + 2.0**-10 * spread).all()


def test_captured_steps_replay(i4s):
    """Two steps in two graphs, replayed in turn with other inputs and eager work in between, against the eager calls."""
    say("captured")
    steps = [prompt_step(i4s, lengths, seed) for seed, lengths in ((1, [300, 20]), (2, [1, 17, 600]))]
    # and a token behind long keys, whose call has a workspace
    q, k, v = (torch.randn(n, h, 128, device="cuda").half() for n, h in ((1, 4), (5000, 1), (5000, 1)))
    graphs, outs = [], []
    for s in steps:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run(), i4s.prompt_attention(q, k, v)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((*s.run()[:2], i4s.prompt_attention(q, k, v)))
        graphs.append(graph)
    for turn in range(4):
        for s in steps:
            s.x.normal_()
        q.normal_(), k.normal_()
        want = [[t.clone() for t in (*s.run()[:2], i4s.prompt_attention(q, k, v))] for s in steps]
        for graph in graphs:
            graph.replay()
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(a, b) for a, b in zip(w, o)), turn


def test_two_streams_at_once(i4s):
    """Calls with workspaces on two streams at the same time."""
    say("two streams")
    torch.manual_seed(3)
    qs = [torch.randn(1, 4, 128, device="cuda").half() for _ in range(2)]
    k, v = (torch.randn(6000, 1, 128, device="cuda").half() for _ in range(2))
    xs = [torch.randn(200, 1024, device="cuda").half() for _ in range(2)]
    w = i4s.mx_quantize(torch.randn(1000, 1024, device="cuda").half())
    want = [(i4s.prompt_attention(q, k, v), i4s.mx_product(x, w)) for q, x in zip(qs, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for s, q, x, g in zip(streams, qs, xs, got):
            with torch.cuda.stream(s):
                g.append((i4s.prompt_attention(q, k, v), i4s.mx_product(x, w)))
    torch.cuda.synchronize()
    for (a, y), g in zip(want, got):
        assert all(torch.equal(a, b) and torch.equal(y, z) for b, z in g)


def test_python_refusals(i4s):
    x, w = torch.zeros(3, 64, dtype=F16, device="cuda"), i4s.mx_quantize(torch.zeros(20, 64, dtype=F16, device="cuda"))
    q = torch.zeros(5, 4, 64, dtype=F16, device="cuda")
    k = q[:, :2]
    i32 = lambda *s: torch.tensor(s, dtype=torch.int32).cuda()  # noqa: E731
    for call in (lambda: i4s.mx_quantize(x.float()), lambda: i4s.mx_quantize(x.cpu()), lambda: i4s.mx_quantize(x[0]),
                 lambda: i4s.mx_quantize(x[:, ::2]), lambda: i4s.mx_quantize(x, out=w), lambda: i4s.mx_read(w, torch.int8),
                 lambda: i4s.mx_product(x.float(), w), lambda: i4s.mx_product(x[:, :32], w), lambda: i4s.mx_product(x.cpu(), w),
                 lambda: i4s.mx_product(x, w, dtype=torch.int32), lambda: i4s.mx_product(x, w, out=x),
                 lambda: i4s.mx_product(x, w, out=torch.zeros(20, 3, dtype=F16, device="cuda").t()),
                 lambda: i4s.mx_product(x, w, dtype=F32, out=torch.zeros(3, 20, dtype=F16, device="cuda")),
                 lambda: i4s.MXTensor(20, 64, w.vals, w.scales[:1]), lambda: i4s.MXTensor(20, 64, w.vals.cpu(), w.scales.cpu()),
                 lambda: i4s.prompt_attention(q.float(), k, k), lambda: i4s.prompt_attention(q, k.bfloat16(), k),
                 lambda: i4s.prompt_attention(q.cpu(), k, k), lambda: i4s.prompt_attention(q, k.cpu(), k),
                 lambda: i4s.prompt_attention(q[0], k, k), lambda: i4s.prompt_attention(q, k, k[:4]),
                 lambda: i4s.prompt_attention(q, k[..., :32], k[..., :32]), lambda: i4s.prompt_attention(q.transpose(1, 2), k, k),
                 lambda: i4s.prompt_attention(q, k, k, k_start=i32(0, 5)), lambda: i4s.prompt_attention(q, k, k, i32(0, 5).long()),
                 lambda: i4s.prompt_attention(q, k, k, i32(0, 5), i32(0, 2, 5)), lambda: i4s.prompt_attention(q, k, k, i32()),
                 lambda: i4s.prompt_attention(q, k, k, out=q.float()), lambda: i4s.prompt_attention(q, k, k, out=q[:4]),
                 lambda: i4s.prompt_attention(q, k, k, lse=torch.zeros(5, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: i4s.mx_quantize(x[:, :40]), lambda: i4s.mx_quantize(x.flatten()[4:68].view(1, 64)),
                 lambda: i4s.mx_product(x, w, out=x.expand(3, 64)[:, :20]), lambda: i4s.mx_product(x[:1].expand(3, 64), w),
                 lambda: i4s.prompt_attention(q[:, :3], k, k), lambda: i4s.prompt_attention(q[..., :32], k[..., :32], k[..., :32]),
                 lambda: i4s.prompt_attention(q, k, k, out=q), lambda: i4s.prompt_attention(q, k, k, scale=0.0),
                 lambda: i4s.prompt_attention(q, k, k, scale=float("nan")), lambda: i4s.prompt_attention(q, k, k, max_q=0),
                 lambda: i4s.prompt_attention(q, k, k, max_k=-1)):
        with pytest.raises(i4s.I4SError):
            call()
