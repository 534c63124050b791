"""Products whose scales lie at the ends of their range, on the GPU.

A block of 32 products is multiplied by two powers of two, 2^(a - 127) and
2^(b - 127) for scale bytes a and b from 0 to 254.  Their product may leave
fp32's range while neither does.
"""

import numpy as np
import pytest

from oracle import prompt_oracle as O
from test_prompt_gpu import BF16, F16, F32, f64, half_step, i4s, least, say  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF = float("inf")


def held(i4s, code, scale):
    """An MXTensor of codes [rows, cols] and scale bytes [rows, cols / 32]."""
    vals, scales = O.mx_pack(code, scale)
    rows, cols = code.shape
    shape = -(-rows // 16), -(-cols // 512)
    return i4s.MXTensor(rows, cols, torch.from_numpy(vals).view(shape[0], -1, 1024).cuda(),
                        torch.from_numpy(scales).view(*shape, 256).cuda())


# tokens, rows: every kernel's shape (few tokens; 64 x 128, 128 x 128, 256 x 256 outputs)
SHAPES = [(1, 40), (16, 300), (40, 77), (100, 16300), (383, 5003), (3900, 3900)]
# scale bytes of tokens and weights, whose powers of two together lie in fp32's normal range, and below it
PAIRS = [(0, 254), (254, 0), (3, 250), (1, 251), (253, 2), (67, 66), (60, 80), (180, 170), (127, 1), (254, 5)]
SMALL = [(60, 60), (64, 59), (0, 120), (100, 10), (30, 70), (0, 0)]


def drawn(rng, rows, cols, byte):
    code = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    scale = np.minimum(byte + rng.integers(0, 2, (rows, cols // 32)), 254).astype(np.uint8)
    return code, scale


@pytest.mark.parametrize("tokens,rows", SHAPES)
@pytest.mark.parametrize("pairs", [PAIRS, SMALL], ids=["normal", "subnormal"])
def test_products_of_large_and_small_scales(i4s, tokens, rows, pairs):
    """Sums that fp32 holds, subnormal ones among them: as near as at any other scale.  There each of the cols / 32 + 8
    additions is off by at most 2^-23 of what it adds up; below the normal range fp32's steps are 2^-149 whatever the
    number's size, so that each addition may be off by one of those as well, and the last rounding by half of one."""
    rng = np.random.default_rng(rows)
    cols = 320
    for a, b in pairs:
        x, w = drawn(rng, tokens, cols, a), drawn(rng, rows, cols, b)
        xt, wt = held(i4s, *x), held(i4s, *w)
        want, size = O.product(O.mx_values(*x), O.mx_values(*w))
        tol = (cols / 32 + 8) * (2.0 ** -23 * size + 2.0 ** -149) + least(F32)
        far = np.abs(f64(i4s.mx_product(xt, wt, dtype=F32)) - want)
        say(tokens, rows, a, b, float((far / tol).max()), float(np.abs(want).max()))
        assert (far <= tol).all()
        got = f64(i4s.mx_product(xt, wt, dtype=BF16))  # the exponents of fp32
        assert (np.abs(got - want) <= tol * 1.01 + half_step(BF16) * np.abs(want) + least(BF16)).all()


@pytest.mark.parametrize("tokens,rows", SHAPES)
@pytest.mark.parametrize("a,b", [(254, 254), (200, 200), (254, 126)])
def test_products_past_the_range(i4s, tokens, rows, a, b):
    """Sums of one sign go to that infinity, sums of zeros stay 0, and no sum that passes the range on its way comes back
    as a number of another size."""
    rng = np.random.default_rng(rows + a)
    cols = 1120
    x, w = drawn(rng, tokens, cols, a), drawn(rng, rows, cols, b)
    x[0][0] = 7                        # 6 in every column
    w[0][::4] = 0
    w[0][1::4] &= 7
    w[0][2::4] |= 8
    y = i4s.mx_product(held(i4s, *x), held(i4s, *w), dtype=F32)
    assert (y[:, ::4] == 0).all()
    assert (y[0, 1::4] == INF).all() and (y[0, 2::4] == -INF).all()
    y = f64(y)
    want, size = O.product(O.mx_values(*x), O.mx_values(*w))
    tol = (cols / 32 + 8) * 2.0 ** -23 * size
    assert (~np.isfinite(y) | (np.abs(y - want) <= tol)).all()
    assert not np.isfinite(y[np.abs(want) > 2.0 ** 128 + tol]).any()


@pytest.mark.parametrize("tokens,rows", SHAPES)
@pytest.mark.parametrize("block", [0, 1, 4, 20, 34])
def test_a_block_of_nan_beside_sums_past_the_range(i4s, tokens, rows, block):
    """Whether the NaN comes before or behind the sum's infinity, of either sign: every product with it is NaN."""
    rng = np.random.default_rng(block)
    cols = 1120
    for sign in (0, 8):
        x, w = (rng.integers(4, 8, (n, cols)).astype(np.uint8) for n in (tokens, rows))
        sx, sw = np.full((tokens, cols // 32), 127, np.uint8), np.full((rows, cols // 32), 127, np.uint8)
        sx[:, 2:30:3] = 254
        sw[:, 2:30:3] = 254
        clean = i4s.mx_product(held(i4s, x | sign, sx), held(i4s, w, sw), dtype=F32)
        assert (clean == (-INF if sign else INF)).all()
        sx[tokens - 1, block] = 255
        sw[rows - 1, block] = 255
        y = i4s.mx_product(held(i4s, x | sign, sx), held(i4s, w, sw), dtype=F32)
        assert y[tokens - 1].isnan().all() and y[:, rows - 1].isnan().all()
        assert torch.equal(y[:tokens - 1, :rows - 1], clean[:tokens - 1, :rows - 1])


@pytest.mark.parametrize("dtype,sizes", [(F16, (2.0 ** -24, 2.0 ** -16, 2.0 ** 14)),
                                         (BF16, (2.0 ** -133, 2.0 ** -120, 2.0 ** 125))])
@pytest.mark.parametrize("tokens", [3, 16, 70])
def test_16_bit_tokens_of_any_size(i4s, tokens, dtype, sizes):
    """The largest and the smallest numbers of a type: quantized within the call as by themselves.  (The largest of bf16
    bring sums past fp32's range: an infinity or NaN, and of the same bits' meaning either way.)"""
    rng = np.random.default_rng(tokens)
    w = i4s.mx_quantize(torch.from_numpy(rng.standard_normal((300, 640))).to(dtype).cuda())
    for size in sizes:
        x = torch.from_numpy(np.clip(rng.standard_normal((tokens, 640)), -3, 3) * size).to(dtype).cuda()
        assert x.isfinite().all() and x.any()
        y, again = i4s.mx_product(x, w, dtype=F32), i4s.mx_product(i4s.mx_quantize(x), w, dtype=F32)
        assert torch.equal(y.isnan(), again.isnan()) and torch.equal(y.nan_to_num(3.0, INF, -INF), again.nan_to_num(3.0, INF, -INF))
        code, scale = O.mx_quantize(f64(x))
        want, spread = O.product(O.mx_values(code, scale), f64(i4s.mx_read(w, F32)))
        assert y.isfinite().all() == (size < 2.0 ** 120)
        y = f64(y)
        near = np.abs(y - want) <= 28 * (2.0 ** -23 * spread + 2.0 ** -149) + least(F32)
        assert (near | (~np.isfinite(y) & (spread > 2.0 ** 127))).all()
