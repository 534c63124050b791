"""The prompt's oracle (``oracle/prompt_oracle.py``) against values worked out by hand and other formulas."""

import numpy as np
import pytest

from oracle import prompt_oracle as O


def block(*values):
    return np.array([list(values) + [0.0] * (32 - len(values))])


@pytest.mark.parametrize("x,byte,codes", [
    # 6 stands at 2^0; ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    ((6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), 127, (7, 0, 2, 2, 4, 4, 6, 6)),
    ((-4.0, 0.26, -0.74, -0.0), 127, (14, 1, 9, 8)),
    ((7.99, 5.01), 127, (7, 7)),            # beyond 6: to 6
    ((8.0, 2.0), 128, (6, 2)),              # the next power of two
    ((0.0, -0.0), 0, (0, 8)),               # nothing: the smallest scale
    ((2.0 ** -126, 2.0 ** -128), 0, (4, 1)),   # 2^-128 is half of the smallest scale 2^-127
    ((2.0 ** 127, 2.0 ** 125), 252, (6, 2)),
    ((1.0, np.nan), 255, (0, 0)), ((1.0, -np.inf), 255, (0, 0))])
def test_blocks(x, byte, codes):
    code, scale = O.mx_quantize(block(*x))
    assert scale.tolist() == [[byte]] and code[0, :len(codes)].tolist() == list(codes)
    assert not code[0, len(codes):].any()
    v = O.mx_values(code, scale)
    if byte == 255:
        assert np.isnan(v).all()
    else:
        again = O.mx_quantize(v)
        np.testing.assert_array_equal(O.mx_values(*again), v)


def test_nearest():
    """No value of the grid is nearer, and the scale leaves the largest below 8 units."""
    x = np.random.default_rng(0).standard_normal((40, 96)) * np.exp(np.random.default_rng(1).standard_normal((40, 1)) * 20)
    code, scale = O.mx_quantize(x)
    unit = np.repeat(np.exp2(scale.astype(float) - 127), 32, 1)
    far = np.abs(np.abs(x)[..., None] - O.GRID * unit[..., None])
    np.testing.assert_array_equal(np.abs(O.mx_values(code, scale) - x), far.min(-1))
    top = (np.abs(x) / unit).reshape(40, 3, 32).max(-1)
    assert (top >= 4).all() and (top < 8).all()


@pytest.mark.parametrize("rows,cols", [(1, 32), (16, 512), (17, 288), (33, 1056)])
def test_places(rows, cols):
    """Every value has a place of its own, and packing and unpacking are inverse."""
    byte, shift, at = O.mx_places(rows, cols)
    assert len(np.unique(byte * 8 + shift)) == rows * cols and len(np.unique(at[:, ::32])) == rows * cols // 32
    rng = np.random.default_rng(cols)
    code = rng.integers(0, 16, (rows, cols), dtype=np.uint8)
    scale = rng.integers(0, 256, (rows, cols // 32), dtype=np.uint8)
    vals, scales = O.mx_pack(code, scale)
    assert byte.max() < vals.size and at.max() < scales.size
    got = O.mx_unpack(vals, scales, rows, cols)
    np.testing.assert_array_equal(got[0], code), np.testing.assert_array_equal(got[1], scale)


def test_first_bytes():
    code = np.zeros((17, 512), np.uint8)
    code[0, 0], code[0, 1], code[1, 0], code[0, 32], code[0, 128], code[16, 0] = 1, 2, 3, 4, 5, 6
    vals, scales = O.mx_pack(code, np.full((17, 16), 9, np.uint8))
    assert (vals[0], vals[16], vals[256], vals[1024], vals[4096]) == (0x21, 3, 4, 5, 6)
    assert np.count_nonzero(vals) == 5 and (scales[:256] == 9).all() and scales.size == 512
    assert (scales[256:].reshape(4, 16, 4)[:, 0] == 9).all() and np.count_nonzero(scales[256:]) == 16


def test_attention_against_a_dense_softmax():
    rng = np.random.default_rng(5)
    for nq, nk in ((4, 4), (3, 7), (5, 2)):
        q, k, v = rng.standard_normal((nq, 4, 8)), rng.standard_normal((nk, 2, 8)), rng.standard_normal((nk, 2, 8))
        for causal in (True, False):
            out, lse, spread = O.attention(q, k, v, causal, 0.3)
            kk, vv = k.repeat(2, 1), v.repeat(2, 1)
            s = 0.3 * np.einsum("qhd,khd->hqk", q, kk)
            if causal:
                s = np.where(np.arange(nk) <= nk - nq + np.arange(nq)[:, None], s, -np.inf)
            with np.errstate(invalid="ignore", divide="ignore"):
                e = np.exp(s)
                want = np.nan_to_num(np.einsum("hqk,khd->qhd", e / e.sum(-1, keepdims=True), vv))
                np.testing.assert_allclose(out, want, atol=1e-12)
                np.testing.assert_allclose(lse, np.log(e.sum(-1)).T, atol=1e-12)
            assert (np.abs(out) <= spread + 1e-12).all()
            if causal and nq > nk:
                assert not out[:nq - nk].any() and np.isneginf(lse[:nq - nk]).all()


def test_attention_does_not_read_what_is_not_seen():
    rng = np.random.default_rng(6)
    q, k, v = (rng.standard_normal((4, 1, 8)) for _ in range(3))
    clean = O.attention(q, k, v, True, 1.0)[0]
    k[3], v[3] = np.nan, np.inf
    np.testing.assert_array_equal(O.attention(q, k, v, True, 1.0)[0][:3], clean[:3])
