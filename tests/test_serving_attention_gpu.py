"""Attention over the 4-bit cache on the GPU where little is left to hide
behind."""

import numpy as np
import pytest

from test_serving_gpu import BF16, F16, SHAPES, device_cache, f64, filled, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def i4s():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int4_sparse_gemv_amd as I
    return I


def int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


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
