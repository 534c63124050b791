"""Plain NumPy definitions of the prompt's operators, in float64 and exact
whole numbers.  Test infrastructure only; shares no code with the library.

Values travel as float64 arrays that hold exactly what fp16, bf16 or fp32
inputs hold.  The microscaled buffers are addressed value by value from the
format's rule.
"""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_SCALE = 255


def mx_quantize(x):
    """[rows, cols] -> (codes 0..15 [rows, cols], scale bytes [rows, cols / 32])."""
    x = np.asarray(x, np.float64)
    y = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(y).all(-1)
    y = np.where(bad[..., None], 0.0, y)
    amax = np.abs(y).max(-1) if y.size else np.zeros(y.shape[:2])
    # frexp: amax = m * 2^k with m in [0.5, 1), so floor(log2(amax)) = k - 1
    e = np.where(amax > 0, np.maximum(np.frexp(amax)[1] - 1 - 2, -127), -127)
    size = np.abs(y) / np.exp2(e.astype(np.float64))[..., None]
    code = np.zeros(size.shape, np.uint8)
    best = np.full(size.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):  # of two that are as near the even one stays
        far = np.abs(size - GRID[c])
        code = np.where(far < best, np.uint8(c), code)
        best = np.minimum(best, far)
    code = code | (np.signbit(y).astype(np.uint8) << 3)
    code[bad] = 0
    return code.reshape(x.shape), np.where(bad, NAN_SCALE, e + 127).astype(np.uint8)


def mx_values(code, scale):
    """What codes and scale bytes stand for."""
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    unit = np.where(scale == NAN_SCALE, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return v * np.repeat(unit, 32, axis=1)


def mx_places(rows, cols):
    """(byte of vals, shift, byte of scales) of every value, in the flat buffers."""
    row, col = np.arange(rows)[:, None], np.arange(cols)[None]
    steps, groups = 2 * -(-cols // 256), -(-cols // 512)
    lane = 16 * (col % 128 // 32) + row % 16
    byte = ((row // 16 * steps + col // 128) * 64 + lane) * 16 + col % 32 // 2
    scale = ((row // 16 * groups + col // 512) * 64 + lane) * 4 + col % 512 // 128
    return byte, 4 * (col % 2), scale


def mx_pack(code, scale):
    """The two buffers, zeros where no value lies."""
    rows, cols = code.shape
    tiles = -(-rows // 16)
    vals = np.zeros(tiles * 2 * -(-cols // 256) * 1024, np.uint8)
    scales = np.zeros(tiles * -(-cols // 512) * 256, np.uint8)
    byte, shift, at = mx_places(rows, cols)
    np.bitwise_or.at(vals, byte, code << np.broadcast_to(shift, code.shape).astype(np.uint8))
    scales[at[:, ::32]] = scale
    return vals, scales


def mx_unpack(vals, scales, rows, cols):
    """(codes, scale bytes) of the two buffers."""
    byte, shift, at = mx_places(rows, cols)
    return vals[byte] >> shift & 15, scales[at[:, ::32]]


def product(x, w):
    """(y, sum of magnitudes) of tokens [tokens, cols] and a weight [rows, cols]."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def attention(q, k, v, causal, scale):
    """One sequence: q [nq, heads, D], k and v [nk, kv_heads, D].  (out, lse,
    spread): spread is the probabilities' sum of |v|, what roundings of
    probabilities are relative to.  Keys that a token does not see do not enter."""
    nq, heads, _ = q.shape
    nk, kv_heads, d = k.shape
    out, lse, spread = np.zeros((nq, heads, d)), np.full((nq, heads), -np.inf), np.zeros((nq, heads, d))
    for h in range(heads):
        kh, vh = k[:, h // (heads // kv_heads)], v[:, h // (heads // kv_heads)]
        for t in range(nq):
            n = max(0, min(nk, nk - nq + t + 1)) if causal else nk
            if n == 0:
                continue
            x = scale * (kh[:n] @ q[t, h])
            m = x.max()
            p = np.exp(x - m)
            l = p.sum()
            lse[t, h] = m + np.log(l)
            out[t, h] = (p / l) @ vh[:n]
            spread[t, h] = (p / l) @ np.abs(vh[:n])
    return out, lse, spread
