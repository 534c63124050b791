"""Attention of whole prompts where values are not finite, on the GPU.

The rule: every key that a token sees counts, whatever its probability.  A NaN
among their values, or infinities of both signs, make the channel NaN, another
infinity makes it that infinity.  So the answer depends neither on the launch's
shape, nor on the tile that a key lies in, nor on where the keys are split;
channels whose values are finite keep their bits.
"""

import numpy as np
import pytest

from test_prompt_gpu import BF16, F16, i4s, say  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")

# (query tokens, keys) of every sequence, KV heads, query heads of one: the launch's shapes, each with long and ragged keys
SHAPES = {
    "wave": ([(2, 203), (1, 64)], 1, 3),                              # 32 rows or fewer: waves with tiles of their own
    "wave_split": ([(2, 3001), (1, 700)], 1, 3),
    "block": ([(61, 203), (90, 90)], 2, 3),                           # 128 rows
    "block_split": ([(50, 3001), (9, 700)], 1, 4),
    "large": ([(300, 6200)] + [(n, n + 70) for n in range(46)], 2, 4),  # 256 rows, head dimension 128
}
CASES = [(s, d, t) for s in SHAPES for d, t in ((64, F16), (128, BF16), (256, BF16)) if s != "large" or d == 128]


def make(shape, dim, dtype, seed=0):
    lengths, heads, share = SHAPES[shape]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    nq, nk = sum(a for a, _ in lengths), sum(b for _, b in lengths)
    q, k, v = (torch.randn(n, h, dim, generator=g, device="cuda").to(dtype)
               for n, h in ((nq, heads * share), (nk, heads), (nk, heads)))
    starts = [torch.tensor([0] + list(np.cumsum(x)), dtype=torch.int32).cuda() for x in zip(*lengths)]
    return q, k, v, starts, lengths


def attend(i4s, q, k, v, starts, lengths, causal=True, scale=1.0):
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    out = i4s.prompt_attention(q, k, v, *starts, max_q=max(a for a, _ in lengths), max_k=max(b for _, b in lengths),
                               causal=causal, scale=scale, lse=lse)
    return out, lse


def test_the_shapes_are_split_as_said(i4s):
    from int4_sparse_gemv_amd.prompt import _attention_workspace
    for shape, (lengths, heads, share) in SHAPES.items():
        nq, nk = (sum(x) for x in zip(*lengths))
        n = _attention_workspace(0, 128, heads * share, heads, nq, nk, len(lengths), *(max(x) for x in zip(*lengths)))
        assert (n > 0) == shape.endswith("split"), shape


@pytest.mark.parametrize("shape,dim,dtype", CASES)
@pytest.mark.parametrize("where", [0, 40, 150])
@pytest.mark.parametrize("below", [300.0, INF])
def test_a_nan_of_no_weight_counts(i4s, shape, dim, dtype, where, below):
    """A NaN among the values of keys whose scores lie 300 below the others', or are -inf: whole pieces of them."""
    say(shape, dim, dtype, where, below)
    q, k, v, starts, lengths = make(shape, dim, dtype)
    some = 600 if lengths[0][1] > 600 else 160  # keys of no weight, in all of a wave's or a piece's tiles
    q[..., 0], k[..., 0], k[:some, :, 0] = 1, 0, -below * dim ** 0.5
    clean, clean_lse = attend(i4s, q, k, v, starts, lengths, True, dim ** -0.5)
    v[where, :, 3] = NAN
    out, lse = attend(i4s, q, k, v, starts, lengths, True, dim ** -0.5)
    assert torch.equal(lse, clean_lse)
    nq, nk = lengths[0]
    hit = slice(max(0, where - (nk - nq)), nq)  # the tokens of the first sequence that see it
    assert out[hit, :, 3].isnan().all()
    out[hit, :, 3] = clean[hit, :, 3]
    assert torch.equal(out, clean)


# ---------------------------------------------------------------------------
# the rule for all values that are not finite, at every place of the keys


def sees(starts, lengths, key, tokens, causal):
    """Which query tokens see key number ``key`` of the first sequence."""
    nq, nk = lengths[0]
    hit = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    hit[max(0, key - (nk - nq)) if causal else 0:nq] = True
    return hit


def poison(i4s, q, k, v, starts, lengths, key, causal, scale=1.0):
    """One key's values in three channels, NaN and both infinities: the rows that see it get those, all else stays."""
    clean, clean_lse = attend(i4s, q, k, v, starts, lengths, causal, scale)
    v = v.clone()
    for channel, bad in ((3, NAN), (17, INF), (40, -INF)):
        v[key, :, channel] = bad
    out, lse = attend(i4s, q, k, v, starts, lengths, causal, scale)
    hit = sees(starts, lengths, key, q.shape[0], causal)
    assert hit.any() and torch.equal(lse, clean_lse)
    got = out[hit].float()
    assert got[..., 3].isnan().all(), "NaN"
    assert (got[..., 17] == INF).all(), "inf"
    assert (got[..., 40] == -INF).all(), "-inf"
    out = out.clone()
    for channel in (3, 17, 40):
        out[hit, :, channel] = clean[hit, :, channel]
    assert torch.equal(out, clean)


KEYS = ("first", 40, "middle", "block", "last")


def key_of(where, lengths):
    nq, nk = lengths[0]
    return {"first": 0, "middle": nk // 2, "block": nk - nq, "last": nk - 1}.get(where, where)


@pytest.mark.parametrize("shape,dim,dtype", CASES)
@pytest.mark.parametrize("where", KEYS)
@pytest.mark.parametrize("causal", [True, False])
def test_a_key_of_no_weight_counts(i4s, shape, dim, dtype, where, causal):
    """Its score lies 300 below the others: its probability is less than fp32 holds."""
    say(shape, dim, dtype, where, causal)
    q, k, v, starts, lengths = make(shape, dim, dtype)
    key = key_of(where, lengths)
    q[..., 0], k[..., 0], k[key, :, 0] = 1, 0, -300 * dim ** 0.5
    poison(i4s, q, k, v, starts, lengths, key, causal, dim ** -0.5)


@pytest.mark.parametrize("shape,dim,dtype", CASES)
def test_a_key_whose_weight_fades_counts(i4s, shape, dim, dtype):
    """The first key's probability is the largest at its time; later scores rise step by step until it is less than fp32
    holds."""
    say(shape, dim, dtype)
    q, k, v, starts, lengths = make(shape, dim, dtype)
    q[..., 0] = 1
    k[:, :, 0] = (torch.arange(k.shape[0], device="cuda") * (400.0 * dim ** 0.5 / lengths[0][1]))[:, None].to(dtype)
    poison(i4s, q, k, v, starts, lengths, 0, True, dim ** -0.5)


@pytest.mark.parametrize("shape,dim,dtype", CASES)
@pytest.mark.parametrize("where", KEYS)
def test_a_key_of_score_minus_infinity_counts(i4s, shape, dim, dtype, where):
    say(shape, dim, dtype, where)
    q, k, v, starts, lengths = make(shape, dim, dtype)
    key = key_of(where, lengths)
    q[..., 0], k[key, :, 0] = 1, -INF
    poison(i4s, q, k, v, starts, lengths, key, True, dim ** -0.5)


@pytest.mark.parametrize("shape,dim,dtype", CASES)
@pytest.mark.parametrize("where", KEYS)
def test_only_scores_of_minus_infinity(i4s, shape, dim, dtype, where):
    """0 and -inf where the values are finite, and the rule where they are not."""
    say(shape, dim, dtype, where)
    q, k, v, starts, lengths = make(shape, dim, dtype)
    q[..., 0], k[..., 0] = 1, -INF
    for causal in (True, False):
        out, lse = attend(i4s, q, k, v, starts, lengths, causal, dim ** -0.5)
        assert (out == 0).all() and torch.isneginf(lse).all()
        poison(i4s, q, k, v, starts, lengths, key_of(where, lengths), causal, dim ** -0.5)


@pytest.mark.parametrize("shape,dim,dtype", CASES)
def test_infinities_of_both_signs(i4s, shape, dim, dtype):
    """Of keys far apart, in either order, one of them of no weight: NaN for the rows that see both."""
    say(shape, dim, dtype)
    q, k, v, starts, lengths = make(shape, dim, dtype)
    a, b = key_of("first", lengths), key_of("last", lengths)
    q[..., 0], k[..., 0], k[a, :, 0] = 1, 0, -300 * dim ** 0.5
    clean, _ = attend(i4s, q, k, v, starts, lengths, False, dim ** -0.5)
    v[a, :, 5], v[b, :, 5], v[a, :, 9], v[b, :, 9] = INF, -INF, -INF, INF
    out, _ = attend(i4s, q, k, v, starts, lengths, False, dim ** -0.5)
    nq = lengths[0][0]
    assert out[:nq, :, 5].isnan().all() and out[:nq, :, 9].isnan().all()
    keep = out.clone()
    keep[:nq, :, 5], keep[:nq, :, 9] = clean[:nq, :, 5], clean[:nq, :, 9]
    assert torch.equal(keep, clean)


@pytest.mark.parametrize("shape,dim,dtype", CASES)
def test_scores_that_are_not_finite(i4s, shape, dim, dtype):
    """A score of NaN or +inf makes its token's row NaN, and no other."""
    say(shape, dim, dtype)
    for bad in (NAN, INF):
        q, k, v, starts, lengths = make(shape, dim, dtype)
        q[..., 0], k[..., 0] = 1, 0
        key = lengths[0][1] - 1
        clean, clean_lse = attend(i4s, q, k, v, starts, lengths, True, dim ** -0.5)
        k[key, :, 0] = bad
        out, lse = attend(i4s, q, k, v, starts, lengths, True, dim ** -0.5)
        hit = sees(starts, lengths, key, q.shape[0], True)
        assert out[hit].isnan().all() and lse[hit].isnan().all()
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("shape,dim,dtype", CASES)
def test_infinities_of_both_signs_the_last_of_no_weight(i4s, shape, dim, dtype):
    say(shape, dim, dtype)
    q, k, v, starts, lengths = make(shape, dim, dtype)
    a, b = key_of("first", lengths), key_of("last", lengths)
    q[..., 0], k[..., 0], k[b, :, 0] = 1, 0, -300 * dim ** 0.5
    v[a, :, 5], v[b, :, 5], v[a, :, 9], v[b, :, 9], v[a, :, 11], v[b, :, 11] = INF, -INF, -INF, INF, INF, NAN
    nq = lengths[0][0]
    for causal in (True, False):
        out, _ = attend(i4s, q, k, v, starts, lengths, causal, dim ** -0.5)
        both = slice(nq - 1 if causal else 0, nq)
        assert out[both, :, 5].isnan().all() and out[both, :, 9].isnan().all() and out[both, :, 11].isnan().all()
        if causal:  # the tokens before do not see the last key
            assert (out[:nq - 1, :, 5] == INF).all() and (out[:nq - 1, :, 9] == -INF).all() and (out[:nq - 1, :, 11] == INF).all()
        assert out[:nq, :, 12:].isfinite().all() and out[nq:].isfinite().all()


@pytest.mark.parametrize("shape,dim,dtype", CASES)
@pytest.mark.parametrize("where", KEYS)
def test_scores_that_are_not_finite_anywhere(i4s, shape, dim, dtype, where):
    """A score of NaN or +inf, far above or below the others' tiles: its rows are NaN, beside values that are not finite too."""
    say(shape, dim, dtype, where)
    q, k, v, starts, lengths = make(shape, dim, dtype)
    q[..., 0], k[..., 0] = 1, 0
    key = key_of(where, lengths)
    hit = sees(starts, lengths, key, q.shape[0], True)
    for bad in (NAN, INF):
        for values in (False, True):
            kk, vv = k.clone(), v.clone()
            if values:
                vv[lengths[0][1] // 3, :, 7], vv[key, :, 9] = INF, NAN
            clean, clean_lse = attend(i4s, q, kk, vv, starts, lengths, True, dim ** -0.5)
            kk[key, :, 0] = bad
            out, lse = attend(i4s, q, kk, vv, starts, lengths, True, dim ** -0.5)
            assert out[hit].isnan().all() and lse[hit].isnan().all()
            assert torch.equal(out[~hit].nan_to_num(3.0, INF, -INF), clean[~hit].nan_to_num(3.0, INF, -INF))
            assert torch.equal(lse[~hit], clean_lse[~hit])


def test_a_captured_call_with_values_that_are_not_finite(i4s):
    """Replayed with finite and other values in turn: each replay is the eager call's result."""
    say("captured")
    q, k, v, starts, lengths = make("block", 128, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attend(i4s, q, k, v, starts, lengths)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = attend(i4s, q, k, v, starts, lengths)
    for value in (1.0, INF, NAN, 2.0, -INF, 0.5):
        v[7, :, 3], v[202, 0, 100] = value, value
        want, _ = attend(i4s, q, k, v, starts, lengths)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(3.0), want.nan_to_num(3.0)), value
