"""Attention of whole prompts where values are not finite, on the GPU: what a
token sees counts, whatever its probability and wherever the keys are split."""

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
