"""Pins of the serving oracle (CPU): the cache format word by word, the
quantizer's corners, and the definitions against independent forms."""

import numpy as np
import pytest

from oracle import serve_oracle as O


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_places_are_a_permutation(dim):
    k = {O.k_place(x, dim) for x in range(dim)}
    v = {O.v_place(x, dim) for x in range(dim)}
    every = {(w, 4 * b) for w in range(dim // 8) for b in range(8)}
    assert k == v == every


def test_places_of_some_channels():
    """Worked by hand from the format: dim 128, channel 77 = 32*2 + 8*1 + 5: K word 4*1 + 2, element 5 in slot 6;
    77 = 64*1 + 16*0 + 13: V half 13*2 + 1 = word 13, upper half, e = 0."""
    assert O.k_place(77, 128) == (6, 24)
    assert O.v_place(77, 128) == (13, 16)
    assert O.k_place(0, 64) == (0, 0) and O.k_place(1, 64) == (0, 16)
    assert O.v_place(63, 64) == (7, 28) and O.v_place(255, 256) == (31, 28)


def test_write_then_read():
    rng = np.random.default_rng(0)
    c = O.Cache(3, 16, 2, 64, 32)
    k, v = rng.standard_normal((2, 5, 2, 64)).astype(np.float16).astype(np.float64)
    slots = [0, 47, 17, 3, 30]
    for t, s in enumerate(slots):
        c.write(s, k[t], v[t])
    gk, gv = c.read(slots + [-1, 48])
    for got, x in ((gk, k), (gv, v)):
        q, s = O.quantize(x, 32)
        np.testing.assert_array_equal(got[:5], q * s.repeat(32, -1))
        assert not got[5:].any()
        step = s.repeat(32, -1)
        # |x - s q| is at most half a step, and 3.5 steps of the rounded scale's own half step 2^-11 at the ends
        assert (np.abs(got[:5] - x) <= step * (0.5 + 7 * 2.0**-11)).all()


def test_quantizer_corners():
    q, s = O.quantize(np.array([np.nan, np.inf, -np.inf, 1.0] + [0.0] * 28), 32)
    assert s[0] == O.SCALE_MAX and list(q[:4]) == [0, 7, -7, 0]
    q, s = O.quantize(np.zeros(32), 32)
    assert s[0] == 0 and not q.any()
    q, s = O.quantize(np.array([7.0, 0.5, 1.5, 2.5, -0.5, -3.5] + [0.0] * 26), 32)
    assert s[0] == 1 and list(q[:6]) == [7, 0, 2, 2, 0, -4]  # half to even
    assert np.isfinite(np.float16(7 * O.SCALE_MAX)) and not np.isfinite(np.float16(7 * (O.SCALE_MAX + 8)))


def test_attention_against_a_softmax_matrix():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    out, lse, _ = O.attention(q, k, v, 6, 0.3)
    for h in range(4):
        x = 0.3 * q[:, h] @ k[:, h // 2].T
        x[np.arange(9)[None] > 6 + np.arange(3)[:, None]] = -np.inf
        np.testing.assert_allclose(lse[:, h], np.log(np.exp(x).sum(1)), rtol=1e-12)
        np.testing.assert_allclose(out[:, h], (np.exp(x) / np.exp(x).sum(1, keepdims=True)) @ v[:, h // 2], rtol=1e-12)
    chain = O.attention(q, k, v, 6, 0.3, [1, 3, 7])
    np.testing.assert_array_equal(chain[0], out)
    empty = O.attention(q, k[:3], v[:3], 0, 0.3, [0, 2, 5])
    assert not empty[0][0].any() and np.isneginf(empty[1][0]).all() and np.isfinite(empty[1][1:]).all()


def test_extend_small():
    r = O.extend([[7, -1, -1], [-1, -1, -1]], [10, 0], [8, 17], [3, 4, 5, 6], 4, 16, 27)
    assert r["table"].tolist() == [[7, 6, -1], [5, 4, -1]] and r["free_count"] == 1 and r["flags"] == 0
    assert r["q_start"] == [0, 8, 25] and r["lens"] == [18, 17]
    assert r["slots"] == [7 * 16 + i for i in range(10, 16)] + [96, 97] + [80 + i for i in range(16)] + [64, -1, -1]
    assert r["positions"] == list(range(10, 18)) + list(range(17)) + [0, 0]


def test_token_logprobs_small():
    x = np.array([[0.0, np.log(2.0), np.log(5.0), -np.inf]])
    lp, ent, ids, top = O.token_logprobs(x, np.array([1]), 2)
    p = np.array([1, 2, 5]) / 8
    np.testing.assert_allclose(lp, np.log(2 / 8))
    np.testing.assert_allclose(ent, -(p * np.log(p)).sum())
    assert ids.tolist() == [[2, 1]]
    np.testing.assert_allclose(top, np.log([[5 / 8, 2 / 8]]))
