"""Attention over the 4-bit cache on the GPU where little is left to hide
behind: values next to others that are far larger, scores of nearly one
height, keys in several pieces, masks in the last piece.

The outputs are held against the float64 definition to the last half step of
their type, by its true spacing, and what the arithmetic before that loses:

* key j's score is off by at most d_j = scale (D + D/G + 8) 2^-24 sum |q| (|k_j|
  + 24 s_j) (fp32 sums of products with 16 + u that start from -24 sum q) and, as
  the sum over groups starts from minus the row's reference, a score too, by
  scale (D/G + 2) 2^-24 max |q . k|, which moves its weight by expm1(d_j) of itself, and the sum that divides by at most E
  = sum p_j expm1(d_j): together (sum p_j expm1(d_j) |v_j| + |out| E) / (1 - E);
* a probability times V's scale s is taken in two bf16 terms, of 8 bits each:
  the first leaves 2^-8 of it, the second 2^-8 of that: 2^-16;
* the sums are fp32.  A wave has at most a quarter of the keys, n = l / 128 steps
  of 32; a step adds two products of 32 terms to each output, the value + 24 for
  even tokens and - 23 for odd ones, each product off by at most 2^-23 of what it
  sums, 31 sum p s so far; and 8 times to the sum of the offsets, 24 sum p s so
  far: (2 * 31 2^-23 + 8 * 24 2^-24) (n / 2 + 1) sum p s.  (l + 64) 2^-24 sum p |v|
  for joins, exponentials and the quotient;
* blocks of many rows and groups (row tiles x channel groups >= 8) scale V
  instead, without offsets: fp16 outputs keep 2^-21 of a probability times a
  scaled value (two fp16 terms of either, without the product of the second
  ones), bf16 outputs 2^-11 of either.  The probability is 2^7 at least for the
  key that set the row's offset, so that fp16's smallest step loses at most 2^-32
  |v| of every key's value, whatever other keys and groups hold.  Three products a
  step sum 7 p s each: 3 * 7 2^-23 (n / 2 + 1) sum p s.
"""

import ctypes

import numpy as np
import pytest

from oracle import serve_oracle as O
from test_serving_gpu import BF16, F16, SHAPES, device_cache, f64, filled, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def i4s():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int4_sparse_gemv_amd as I
    return I


def spacing(x, dtype):
    """The distance from |x| to the next larger number of the type."""
    bits, least = (10, -24) if dtype == F16 else (7, -133)
    e = np.frexp(np.where(x == 0, 2.0**-140, np.abs(x)))[1] - 1
    return np.exp2(np.maximum(e - bits, least))


class Definition:
    """out and lse of one sequence, and what its errors are measured by: sum p |v|, sum p s, sum |v| over the keys
    seen, and `moved`, the error that the scores' own errors leave.  ks, vs: the scales of every channel."""

    def __init__(self, q, k, v, ks, vs, group, ctx, scale, masks=None):
        n, heads, dim = q.shape
        length, share = k.shape[0], heads // k.shape[1]
        pos = np.arange(length)
        if masks is None:
            seen = pos[None] <= ctx + np.arange(n)[:, None]
        else:
            bit = np.clip(pos - ctx, 0, 63).astype(np.uint64)
            named = (np.asarray(masks).view(np.uint64)[:, None] >> bit[None]) & np.uint64(1)
            seen = (pos < ctx)[None] | ((named > 0) & (pos - ctx < 64)[None])
        self.out, self.spread, self.p_s, self.sum_v, self.moved = (np.zeros((n, heads, dim)) for _ in range(5))
        self.lse = np.full((n, heads), -np.inf)
        self.d_score = np.zeros((n, heads))
        some = seen.any(1)
        for h in range(heads if length else 0):
            kh, vh, qh = k[:, h // share], v[:, h // share], q[some, h]
            x = np.where(seen[some], scale * (qh @ kh.T), -np.inf)
            m = x.max(1, keepdims=True)
            e = np.exp(x - m)
            p = e / e.sum(1, keepdims=True)
            self.lse[some, h] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
            self.out[some, h] = p @ vh
            self.spread[some, h] = p @ np.abs(vh)
            self.p_s[some, h] = p @ vs[:, h // share]
            self.sum_v[some, h] = seen[some].astype(float) @ np.abs(vh)
            d = scale * (np.abs(qh) @ (np.abs(kh) + 24 * ks[:, h // share]).T) * (dim + dim // group + 8) * 2.0**-24
            d = np.where(seen[some], d + np.abs(np.where(seen[some], x, 0)).max(1, keepdims=True) * (dim // group + 2) * 2.0**-24, 0)
            z = (p * np.expm1(d)).sum(1, keepdims=True)
            assert (z < 0.5).all()
            self.moved[some, h] = ((p * np.expm1(d)) @ np.abs(vh) + np.abs(p @ vh) * z) / (1 - z)
            self.d_score[some, h] = z[:, 0] / (1 - z[:, 0])


def scales_of(c, slots):
    """K's and V's scales of every channel, float64 [tokens, heads, D]."""
    out = np.zeros((2, len(slots), c.heads, c.dim))
    for n, slot in enumerate(slots):
        page, off = divmod(int(slot), c.page_size)
        at = c._at(off)[4]
        out[0, n], out[1, n] = c.k_scales[page][:, at], c.v_scales[page][:, at]
    return out


def int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def pieces_of(d, tokens, q_heads, n, width, max_q, max_len):
    """Into how many pieces a call splits the keys, from its workspace."""
    from int4_sparse_gemv_amd import _serve_binding as S
    a = S.i4s_attention_args()
    a.cache, a.dtype, a.q_heads, a.num_tokens, a.num_seqs = ctypes.addressof(d.descriptor), 0, q_heads, tokens, n
    a.table_width, a.q_start, a.max_q, a.max_len, a.scale = width, 4, max_q, max_len, 1.0
    size = ctypes.c_uint64()
    assert S.i4s_attention_workspace_size(a, size) == 0
    return max(1, size.value // (tokens * q_heads * (d.head_dim + 4) * 4))


def scales_v(c, rows):
    groups = c.dim // c.group
    return (2 if rows > 16 and groups >= 4 and c.dim <= 128 else 1) * groups >= 8


def attend(i4s, rng, c, d, lens, q_lens, share, dtype, q=None, masks=None, scale=None, max_len=0, pieces=None, table=None):
    """One call against the definition; q: numpy [tokens, heads, D], by default normal."""
    page, heads, dim = c.page_size, c.heads, c.dim
    width = max(1, max(-(-l // page) for l in lens))
    if table is None:
        table, order, at = np.zeros((len(lens), width), np.int64), rng.permutation(c.pages), 0
        for i, l in enumerate(lens):
            m = -(-l // page)
            table[i, :m] = order[at:at + m]
            at += m
    total, starts = sum(q_lens), np.concatenate([[0], np.cumsum(q_lens)])
    q = rng.standard_normal((total, heads * share, dim)) if q is None else q
    q = torch.from_numpy(np.asarray(q, np.float64)).to(dtype)
    scale = dim**-0.5 if scale is None else scale
    if pieces is not None:
        n = pieces_of(d, total, heads * share, len(lens), width, max(q_lens), max_len)
        assert pieces(n), f"{n} pieces"
    lse = torch.empty(total, heads * share).cuda()
    args = dict(q_start=int32(starts), max_q=max(q_lens), max_len=max_len, scale=scale, lse=lse,
                tree_mask=None if masks is None else torch.from_numpy(np.asarray(masks)).cuda())
    out = i4s.kv_attention(d, q.cuda(), int32(table), int32(lens), **args)
    torch.cuda.synchronize()
    wide = scales_v(c, max(q_lens) * share)
    kept = 2.0**-16 if not wide else (2.0**-21 if dtype == F16 else 2.0**-10)
    for i, (l, n_q) in enumerate(zip(lens, q_lens)):
        slots = [int(table[i, j // page]) * page + j % page for j in range(l)]
        k, v = c.read(slots)
        ks, vs = scales_of(c, slots)
        a, b = starts[i], starts[i + 1]
        w = Definition(f64(q[a:b]), k, v, ks, vs, c.group, l - n_q, scale, None if masks is None else masks[a:b])
        before = w.moved + 1.01 * ((l + 64) * 2.0**-24 + kept) * w.spread
        before += (3 * 7 if wide else 62 + 96) * 2.0**-23 * (l / 256 + 1) * w.p_s + (2.0**-32 * w.sum_v if wide else 0)
        got = f64(out[a:b])
        tol = before + spacing(np.abs(w.out) + before, dtype) / 2
        bad = ~(np.abs(got - w.out) <= tol)
        assert not bad.any(), (i, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], w.out[bad][:3], tol[bad][:3])
        got_lse, empty = f64(lse[a:b]), np.isneginf(w.lse)
        assert np.array_equal(empty, np.isneginf(got_lse))
        with np.errstate(invalid="ignore"):
            off = ~(np.abs(got_lse - w.lse) <= w.d_score + (l + 64) * 2.0**-24 + 2.0**-22 * np.abs(w.lse))
        assert not (off & ~empty).any()
    for _ in range(2):
        same = torch.equal(out, i4s.kv_attention(d, q.cuda(), int32(table), int32(lens), **args))
        assert same, "two calls differ"
    return out


def random_masks(rng, q_lens):
    """Any subset of a token's earlier candidates and itself."""
    return np.concatenate([[sum(1 << int(b) for b in np.nonzero(rng.random(t + 1) < 0.5)[0]) for t in range(n)]
                           for n in q_lens]).astype(np.uint64).view(np.int64)


# ---------------------------------------------------------------------------
# scales of the scores


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_any_positive_scale(i4s, dim, group, dtype):
    """A scale so small that no score differs from another gives the mean of V; with V of zeros, zeros.

    The output's rounding and those of the weights: at most 2^-8 of the mean and 2^-9 of the mean of |V|."""
    for share, scale in ((1, 1e-38), (24, 1e-38), (3, 2.0**-126), (24, 1e-40), (1, 1e-30)):
        say("any scale", dim, group, dtype, share, scale)
        rng = np.random.default_rng(dim + group + share)
        c, d = filled(i4s, rng, 20, 16, 1, dim, group)
        _, v = c.read(np.arange(300))
        q = torch.from_numpy(rng.standard_normal((2, share, dim))).to(dtype).cuda()
        table, lens = int32(np.arange(20)[None].repeat(2, 0)), int32([1, 300])
        out = f64(i4s.kv_attention(d, q, table, lens, scale=scale))
        for i, n in enumerate((1, 300)):
            mean, size = v[:n, 0].mean(0), np.abs(v[:n, 0]).mean(0)
            assert (np.abs(out[i] - mean) <= 2.0**-8 * np.abs(mean) + 2.0**-9 * size).all()
        c.v_scales[:] = 0
        assert not i4s.kv_attention(device_cache(i4s, c), q, table, lens, scale=scale).any()


# ---------------------------------------------------------------------------
# what the probabilities keep


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_few_keys_to_the_last_half_step(i4s, dim, group, dtype):
    """One to forty keys of nearly one height: a probability's own rounding would show."""
    for share, lens, q_lens in ((1, [1, 2, 3, 40], [1, 1, 1, 1]), (4, [5, 9, 33], [2, 8, 6])):
        say("few keys", dim, group, dtype, share)
        rng = np.random.default_rng(dim + 3 * group + share)
        c, d = filled(i4s, rng, 9, 16, 2, dim, group)
        q = rng.standard_normal((sum(q_lens), 2 * share, dim)) / 128
        attend(i4s, rng, c, d, lens, q_lens, share, dtype, q=q)


def beside(c, rng, keys, at):
    """V positive and small, K of zeros, but for key `at`: it has about half of the probability of a query of ones, and
    V = 0."""
    c.k_scales[:] = 0
    c.v_scales[:] = rng.uniform(0.002, 0.003, c.v_scales.shape)
    c.v_vals |= 0x88  # nibbles 8..15: values of 0 to 7
    put_key(c, at, np.log(keys), 0.0)


def put_key(c, at, score, v_scale):
    """Key `at` (page = its table entry): the score of a query of ones at the default scale, and V's scale."""
    page, off = divmod(at, c.page_size)
    for h in range(c.heads):
        places = c._at(off)[4]
        c.k_scales[page, h, places] = np.float16(abs(score) / 7 / c.dim**0.5)
        c.k_vals[page, h, off * (c.dim // 2):(off + 1) * (c.dim // 2)] = 0xFF if score > 0 else 0x11
        c.v_scales[page, h, places] = v_scale


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 32), (128, 64), (256, 32), (256, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_small_values_beside_a_group_of_large_ones(i4s, dim, group, dtype):
    """One channel group's V is a million times the others', and one key of the wave has half of the probability."""
    for share in (1, 24):
        say("beside a large group", dim, group, dtype, share)
        rng = np.random.default_rng(dim + share)
        c, _ = filled(i4s, rng, 16, 16, 1, dim, group)
        beside(c, rng, 250, 3)
        s = c.v_scales.reshape(16, 1, 4, dim // group, 4)
        s[:, :, :, 0] = np.where(s[:, :, :, 0] == 0, 0, rng.uniform(2000, 3000, s[:, :, :, 0].shape))
        attend(i4s, rng, c, device_cache(i4s, c), [250], [1], share, dtype, q=np.ones((1, share, dim)),
               table=np.arange(16)[None])


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_small_values_beside_an_infinity(i4s, dim, group, dtype):
    """An infinity in V is stored as the largest value; a key that has it and hardly any probability, or that a token
    does not see, takes nothing from the others."""
    for share in (1, 24):
        say("beside an infinity", dim, group, dtype, share)
        rng = np.random.default_rng(dim + group + share)
        c, _ = filled(i4s, rng, 24, 16, 1, dim, group)
        table = np.arange(24)[None]
        beside(c, rng, 250, 3)
        put_key(c, 4, -24.0, O.SCALE_MAX)
        attend(i4s, rng, c, device_cache(i4s, c), [250], [1], share, dtype, q=np.ones((1, share, dim)), table=table)
        # the same at a candidate that the last token does not see
        beside(c, rng, 310, 290)
        put_key(c, 308, -24.0, O.SCALE_MAX)
        masks = np.array([1, 1, 0b101], np.uint64).view(np.int64)
        attend(i4s, rng, c, device_cache(i4s, c), [310], [3], share, dtype, q=np.ones((3, share, dim)), masks=masks,
               table=table)


@pytest.mark.parametrize("dim,group,share", [(64, 32, 1), (128, 64, 4), (128, 32, 24), (256, 128, 16)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tokens_of_one_parity(i4s, dim, group, share, dtype):
    """All the weight on even or on odd tokens: the offsets of the two do not cancel."""
    for odd in (0, 1):
        say("one parity", dim, group, share, dtype, odd)
        rng = np.random.default_rng(dim + share + odd)
        c, _ = filled(i4s, rng, 150, 16, 1, dim, group)
        c.k_scales[:] = 0
        for at in range(odd, 150 * 16, 2):
            put_key(c, at, -60.0, 0.3)
        attend(i4s, rng, c, device_cache(i4s, c), [2395, 33], [1, 1], share, dtype, q=np.ones((2, share, dim)),
               table=np.stack([np.arange(150), np.arange(150)]))


def test_outputs_are_as_near_as_their_rounding(i4s):
    """The mean error of fp16 outputs is that of rounding the exact values to fp16."""
    for lens, share in (([4000], 1), ([700, 33], 4)):
        say("mean error", lens, share)
        rng = np.random.default_rng(sum(lens))
        c, d = filled(i4s, rng, sum(-(-l // 16) for l in lens), 16, 2, 128, 64)
        n = sum(-(-l // 16) for l in lens)
        table, at = np.zeros((len(lens), max(-(-l // 16) for l in lens)), np.int64), 0
        for i, l in enumerate(lens):
            m = -(-l // 16)
            table[i, :m] = np.arange(at, at + m)
            at += m
        assert at == n
        q = rng.standard_normal((len(lens), 2 * share, 128)).astype(np.float16).astype(np.float64)
        out = f64(attend(i4s, rng, c, d, lens, [1] * len(lens), share, F16, q=q, table=table))
        want = []
        for i, l in enumerate(lens):
            slots = [int(table[i, j // 16]) * 16 + j % 16 for j in range(l)]
            k, v = c.read(slots)
            want.append(Definition(q[i:i + 1], k, v, *scales_of(c, slots), 64, l - 1, 128**-0.5).out)
        want = np.concatenate(want)
        rounded = want.astype(np.float16).astype(np.float64)
        norm = lambda x: np.sqrt((x * x).sum())  # noqa: E731
        # before that the 2^-16 of every key, of either sign, adds up as the keys' values themselves do, whose signs are
        # random too: 2^-16 of the output, 2^-5 of its rounding
        assert norm(out - want) <= 1.04 * norm(rounded - want)


# ---------------------------------------------------------------------------
# keys in pieces


def held(i4s, rng, lens, page, heads, dim, group):
    return filled(i4s, rng, sum(-(-l // page) for l in lens) + 1, page, heads, dim, group)


@pytest.mark.parametrize("dim,group,heads,share,lens,q_lens,most", [
    (128, 64, 1, 4, [2300], [1], False), (128, 64, 1, 4, [1500, 40, 1100], [1, 1, 1], True), (128, 32, 2, 1, [3000], [2], False),
    (64, 32, 2, 8, [4100], [1], False), (64, 64, 1, 3, [1300, 9], [5, 2], True), (256, 128, 1, 4, [2000], [2], False),
    (256, 64, 1, 1, [900], [3], True), (256, 32, 1, 2, [2100], [1], False)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_pieces_of_few_rows(i4s, dtype, dim, group, heads, share, lens, q_lens, most):
    """Up to 16 rows: joined by rows (up to 8 pieces) and by blocks (more), every type and channel count."""
    say("pieces", dim, group, heads, share, lens, q_lens, dtype)
    rng = np.random.default_rng(dim + sum(lens))
    c, d = held(i4s, rng, lens, 32, heads, dim, group)
    attend(i4s, rng, c, d, lens, q_lens, share, dtype, pieces=lambda n: 2 <= n <= 8 if most else n > 8)


@pytest.mark.parametrize("dim,group,lens,q_lens,most", [
    (128, 32, [900, 130], [5, 3], True), (128, 32, [1900], [5], False), (256, 64, [800], [4], True), (256, 64, [1500], [4], False),
    (256, 32, [700, 3], [3, 3], True), (256, 32, [1400], [6], False), (128, 64, [1800], [7], True), (64, 32, [3000], [9], False)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_pieces_of_many_rows(i4s, dtype, dim, group, lens, q_lens, most):
    """Several row tiles and blocks of rows, with V's scales on the values and on the probabilities."""
    say("pieces of many rows", dim, group, lens, q_lens, dtype)
    rng = np.random.default_rng(dim + sum(lens) + 1)
    c, d = held(i4s, rng, lens, 16, 1, dim, group)
    attend(i4s, rng, c, d, lens, q_lens, 8, dtype, pieces=lambda n: 2 <= n <= 8 if most else n > 8)


@pytest.mark.parametrize("dim,group,share,lens,q_lens", [
    (128, 128, 1, [2047], [16]), (128, 64, 2, [2100, 70], [64, 64]), (64, 32, 1, [3001], [64]), (128, 32, 8, [1200], [7]),
    (256, 64, 1, [2070, 1], [40, 1]), (128, 64, 1, [2049, 2080], [3, 64])])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tree_masks_over_pieces(i4s, dtype, dim, group, share, lens, q_lens):
    """The candidates lie in the last piece of the keys, or across the last two; some rows see none of a piece."""
    say("tree over pieces", dim, group, share, lens, q_lens, dtype)
    rng = np.random.default_rng(dim + sum(lens) + 2)
    c, d = held(i4s, rng, lens, 32, 1, dim, group)
    attend(i4s, rng, c, d, lens, q_lens, share, dtype, masks=random_masks(rng, q_lens), pieces=lambda n: n > 1)


@pytest.mark.parametrize("dim,group,share,max_len", [(128, 64, 1, 1500), (128, 64, 4, 1100), (128, 32, 24, 700), (64, 32, 2, 2400),
                                                     (256, 128, 1, 600)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_lengths_beyond_max_len(i4s, dtype, dim, group, share, max_len):
    """Keys in pieces by a largest length that is too small: the last piece takes what is left, in any sequence."""
    for tree in (False, True):
        say("beyond max_len", dim, group, share, max_len, dtype, tree)
        lens, q_lens = [2500, max_len, 5, max_len + 1, 3300], [2, 1, 2, 2, 1]
        rng = np.random.default_rng(dim + max_len)
        c, d = held(i4s, rng, lens, 32, 1, dim, group)
        attend(i4s, rng, c, d, lens, q_lens, share, dtype, max_len=max_len, pieces=lambda n: n > 1,
               masks=random_masks(rng, q_lens) if tree else None)


# ---------------------------------------------------------------------------
# scores far from zero


@pytest.mark.parametrize("dim,group,share,n_q,length,page", [(64, 32, 1, 1, 40, 16), (128, 64, 4, 1, 300, 32), (128, 32, 8, 4, 2000, 32),
                                                            (128, 64, 8, 4, 700, 16), (256, 32, 2, 3, 900, 64), (256, 128, 1, 1, 3000, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_billions(i4s, dtype, dim, group, share, n_q, length, page, sign):
    """Scores that are whole multiples of 2^26 or more, exact in fp32: the largest one alone has a weight, and two equal
    ones have a half each, wherever they lie; all of them far above or far below zero."""
    say("billions", dim, group, share, n_q, length, dtype, sign)
    for power in ((11, 13, 15) if dtype == F16 else (12, 20, 60)):
        rng = np.random.default_rng(dim + length + power)
        c, _ = filled(i4s, rng, -(-length // page), page, 1, dim, group)
        c.k_scales[:] = 8192
        c.k_vals[:] = 0x88
        height = rng.integers(-7, 6, length)            # channel 0 of K, in steps of the scale
        best = sorted(rng.choice(length - n_q, 2, replace=False)) if length > 50 else [3, 3]
        height[best] = 6
        height += sign                                  # all of one sign at the top
        height = np.clip(height, -7, 7)
        if sign < 0:
            height = np.where(np.isin(np.arange(length), best), -1, np.minimum(height, -2))
        for at, h in enumerate(height):
            byte = c._at(at % page)[0][0]
            c.k_vals[at // page, 0, byte] = 0x80 | int(h + 8)  # channel 0 is the word's first nibble
        q = np.zeros((n_q, share, dim))
        q[:, :, 0] = 2.0**power
        d = device_cache(i4s, c)
        _, v = c.read(np.arange(length))
        lse = torch.empty(n_q, share).cuda()
        out = f64(i4s.kv_attention(d, torch.from_numpy(q).to(dtype).cuda(), int32(np.arange(-(-length // page))[None]), int32([length]),
                                   q_start=int32([0, n_q]), max_q=n_q, scale=4.0, lse=lse))
        want = v[best, 0].mean(0)
        assert np.isfinite(out).all() and (np.abs(out - want) <= 2.0**-8 * np.abs(v[best, 0]).max(0)).all(), (power, best)
        top = 4.0 * 2.0**power * 8192 * (height.max() if sign > 0 else -1)
        assert (np.abs(f64(lse) - top) <= 2.0**-21 * abs(top)).all()


@pytest.mark.parametrize("dim,group,share,length", [(64, 64, 1, 300), (128, 64, 4, 2000), (128, 32, 24, 300), (256, 32, 1, 900)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_any_finite_scale(i4s, dim, group, share, length, dtype):
    """A scale so large that the largest score alone has a weight."""
    for scale in (1e30, 2.3e38, 3.4e38):
        say("large scale", dim, group, share, length, dtype, scale)
        rng = np.random.default_rng(dim + share + length)
        pages = -(-length // 32)
        c, d = filled(i4s, rng, pages, 32, 1, dim, group)
        k, v = c.read(np.arange(length))
        q = torch.from_numpy(rng.standard_normal((1, share, dim))).to(dtype)
        x = f64(q)[0] @ k[:, 0].T
        two = np.sort(x, 1)[:, -2:]
        assert (two[:, 1] - two[:, 0] > 1e-3).all()  # fp32 tells them apart
        out = f64(i4s.kv_attention(d, q.cuda(), int32(np.arange(pages)[None]), int32([length]), scale=scale))
        best = x.argmax(1)
        want, scales = v[best, 0], scales_of(c, best)[1][:, 0]
        # the output's rounding, half a step of at most 2^-8, and 2^-10 for a probability and a scaled value of one term
        # each; the offsets' additions (see the top) leave something of a value of 0 too
        tol = (2.0**-8 + 2.0**-10) * np.abs(want) + (62 + 96) * 2.0**-23 * (length / 256 + 1) * scales
        assert (np.abs(out[0] - want) <= tol).all(), scale
