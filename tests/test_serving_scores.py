"""Token scores against their float64 definition, each value by the errors
that can enter it: a masked value, as low as its type has, widens nothing.

With m the row's maximum, p the probabilities, l = sum exp(x - m), E1 = sum p
|x - m| and E2 = sum p (x - m)^2, all errors relative to l or absolute in nats:

* an exponential: the difference, its product with log2 e and that constant are
  rounded, 2^-22.5 |x - m| in all with the steps by which a thread's reference
  rises, and v_exp's 2^-22: 2^-22 (1 + E1) of l;
* l's sum in fp32, in partial sums of at most n / 256 + 96 additions: that
  times 2^-24;
* a log probability: l's error, 2^-22 (1 + ln l) of the logarithm, and 2^-23 |x -
  m| of the given or listed value's own difference;
* the entropy, ln l - sum (x - m) p: l's error 1 + 1.5 E1 times (sum in units of
  log2 e), and 2^-21 (1 + ln l + E1 + E2) of the logarithm, of the products' own
  exponentials and of the quotient."""

import numpy as np
import pytest

from oracle import serve_oracle as O

torch = pytest.importorskip("torch")

TYPES = [torch.float16, torch.bfloat16, torch.float32]


def wrong(x, tokens, k, got):
    """The names of what is off in got = (logprobs, entropy, ids, top logprobs) for float64 logits x."""
    n = x.shape[1]
    want = O.token_logprobs(x, tokens, k)
    bad = [] if np.array_equal(got[2], want[2]) else ["ids"]
    with np.errstate(all="ignore"):
        m = x.max(1, keepdims=True)
        d = np.abs(x - m)
        p = np.exp(x - m)
        l = p.sum(1, keepdims=True)
        live = p > 0
        e1, e2 = (np.where(live, p * np.where(live, d, 0)**i, 0).sum(1) / l[:, 0] for i in (1, 2))
        rel = (n / 256 + 96) * 2.0**-24 + 2.0**-22 * (1 + e1)
        of_log = rel + 2.0**-22 * (1 + np.log(l[:, 0]))
        at = np.clip(tokens, 0, n - 1)
        tol = (of_log + 2.0**-23 * d[np.arange(len(x)), at],
               rel * (1 + 1.5 * e1) + 2.0**-21 * (1 + np.log(l[:, 0]) + e1 + e2),
               None,
               of_log[:, None] + 2.0**-23 * np.take_along_axis(d, want[2], 1))
        for i, name in ((0, "logprobs"), (1, "entropy"), (3, "top_logprobs")):
            a, b = got[i].astype(np.float64), want[i]
            same = (a == b) | (np.isnan(a) & np.isnan(b))  # infinities and NaN as they are
            if a.shape != b.shape or not (same | (np.abs(a - b) <= tol[i])).all():
                bad.append(name)
    return bad


def rows_of(dtype, vocab, seed):
    """Normal logits, peaked and flat, and the masks of a vocabulary; the tokens to score."""
    g = torch.Generator().manual_seed(seed)
    low = torch.finfo(dtype).min
    x = torch.randn(16, vocab, generator=g)
    x[0] *= 3
    x[1] *= 20                              # peaked
    x[2] *= 0.01                            # flat
    x[3] = x[3] * 3 + 50
    x[4] = x[4] * 3 - 3000
    x = x.to(dtype)
    some = torch.randperm(vocab, generator=g)[:7]
    for r, mask in ((5, low), (6, -float("inf"))):
        keep = x[r, some].clone()
        x[r] = mask                         # a few tokens are left
        x[r, some] = keep
    x[7, ::2] = low                         # every other one
    x[8, :vocab // 2] = low                 # the first half
    x[9] = low                              # all of them
    x[10] = -float("inf")
    x[11] = low
    x[11, vocab - 1] = 4.0                  # one is left
    x[12] = low
    x[12, 0] = -3.0e4                       # one, low itself
    x[13] = x[13].float().clamp(max=-1e4).to(dtype)  # all equal, below 0
    x[14, vocab // 2] = 30.0                # one far above the others
    tokens = torch.randint(vocab, (16,), generator=g)
    tokens[5], tokens[11], tokens[12], tokens[14] = some[3], vocab - 1, 0, vocab // 2
    return x, tokens


@pytest.mark.parametrize("dtype", TYPES)
def test_a_wrong_result_is_seen(dtype):
    """The exact result, rounded to fp32, passes; a thousandth off in any finite value of any row does not."""
    x, tokens = rows_of(dtype, 50, 0)
    x, tokens = x.double().numpy(), tokens.numpy()
    with np.errstate(over="ignore"):
        want = [a.astype(np.float32) if a.dtype == np.float64 else a for a in O.token_logprobs(x, tokens, 5)]
    assert wrong(x, tokens, 5, want) == []
    for i, name in ((0, "logprobs"), (1, "entropy"), (3, "top_logprobs")):
        for r in range(16):
            if not np.isfinite(want[i][r]).all() or np.abs(want[i][r]).max() > 1e30:
                continue
            off = [a.copy() for a in want]
            off[i][r] += 1e-3 + 1e-3 * np.abs(off[i][r])
            assert wrong(x, tokens, 5, off) == [name], r
    off = [a.copy() for a in want]
    off[2][3, 1:3] = off[2][3, 2:0:-1]
    assert wrong(x, tokens, 5, off) == ["ids"]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [33, 1000, 8193, 32000, 50257, 151643])
def test_scores_of_masked_vocabularies(dtype, vocab):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int4_sparse_gemv_amd as i4s
    print("scores", dtype, vocab, flush=True)
    x, tokens = rows_of(dtype, vocab, vocab)
    for repeat, k in ((1, 8), (1, 0), (20, 32)):  # 320 rows are not split
        y, t = x.repeat(repeat, 1).cuda(), tokens.repeat(repeat).cuda()
        r = i4s.token_logprobs(y, t, top_k=k)
        torch.cuda.synchronize()
        got = [a.cpu().numpy() for a in r]
        for b in range(repeat):  # copies begin elsewhere in a line of memory, where sums have another order
            bad = wrong(x.double().numpy(), tokens.numpy(), k, [a[16 * b:16 * b + 16] for a in got])
            assert not bad, (k, b, bad)
