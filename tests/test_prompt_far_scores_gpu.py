"""Attention of whole prompts whose scores lie far from 0, on the GPU."""

import numpy as np
import pytest

from oracle import prompt_oracle as O
from test_prompt_gpu import BF16, F16, f64, half_step, i4s, least, say  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def far_scores(dim, keys, tokens, dtype, seed):
    """Whole-number scores around 1000 per channel, rising by about 30 over the keys at scale 0.01, spread by about 1."""
    rng = np.random.default_rng(seed)
    rise = np.arange(keys) * 6 // keys
    k = 1000 + 8 * (rng.integers(-2, 3, (keys, 1, dim)) + rise[:, None, None])
    q = rng.integers(0, 2, (tokens, 2, dim))
    v = rng.standard_normal((keys, 1, dim))
    return [torch.from_numpy(x.astype(np.float64)).to(dtype).cuda() for x in (q, k, v)]


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, F16)])
@pytest.mark.parametrize("tokens,keys", [(1, 60), (3, 3001), (16, 700), (90, 90), (40, 3001), (300, 400)])
def test_far_scores(i4s, tokens, keys, dim, dtype):
    """Exponents are exact differences however far from 0 the scores lie: whole numbers below 2^24 are exact in fp32, in
    any order of sums and from any whole reference on.  What is left: scale log2(e) and its product with a difference, a
    rounding each of an exponent that is at most 64 where it matters, the exponential (2^-22), and the roundings that
    every call has (probabilities, n + 8 steps of 2^-23 for sums, the output).  The logarithm of a sum near 1000: 2^-22
    of it for scale, product, sum and the factor of the natural logarithm, and the sum's own."""
    say("far scores", tokens, keys, dim, dtype)
    q, k, v = far_scores(dim, keys, tokens, dtype, dim + keys)
    kn, qn = f64(k), f64(q)
    assert len(np.unique(kn)) > 8 and np.abs(qn).sum(-1).max() * np.abs(kn).max() < 2 ** 24
    scale = float(np.float32(0.01))
    lse = torch.empty(q.shape[:2], device="cuda")
    out = i4s.prompt_attention(q, k, v, scale=scale, lse=lse)
    want, want_lse, spread = O.attention(qn, kn, f64(v), True, scale)
    assert want_lse.max() > 200 and (spread[-1] < np.abs(f64(v)).max(0)).any()
    u = half_step(dtype)
    rel = u + 2 * 64 * 2.0 ** -23 + 2.0 ** -22 + (keys + 8) * 2.0 ** -23
    tol = spread * rel * 1.01 + u * np.abs(want) + least(dtype)
    if dtype == F16:
        tol = tol + 2.0 ** -32 * keys * np.abs(f64(v)).max()
    far = np.abs(f64(out) - want)
    assert (far <= tol).all(), float((far / tol).max())
    tol = 2.0 ** -22 * np.abs(want_lse) + 2.0 ** -22 + (keys + 8) * 2.0 ** -23 + 2 * 64 * 2.0 ** -23
    far = np.abs(f64(lse) - want_lse)
    assert (far <= tol).all(), float((far / tol).max())


def test_far_scores_have_a_softmax_of_several_keys(i4s):
    """What the cases above need to be worth anything: no key has all of the weight, and equal weights would be far off."""
    q, k, v = far_scores(128, 700, 16, BF16, 828)
    want, _, _ = O.attention(f64(q), f64(k), f64(v), True, 0.01)
    flat, _, _ = O.attention(f64(q), f64(k), f64(v), True, 1e-9)
    one, _, _ = O.attention(f64(q), f64(k), f64(v), True, 10.0)
    assert np.abs(want - flat).max() > 0.3 and np.abs(want - one).max() > 0.3
