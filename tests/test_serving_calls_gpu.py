"""The serving operators on the GPU: calls at the edges of what the header
allows."""

import numpy as np
import pytest

from oracle import serve_oracle as O
from test_serving_gpu import BF16, F16, F32, f64, filled, say

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
# reading tokens


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_read_into_outputs_of_16_byte_alignment(i4s, dim, group, dtype):
    """Outputs that begin between two multiples of 32 bytes, and what lies around them stays."""
    say("read alignment", dim, group, dtype)
    from int4_sparse_gemv_amd import _serve_binding as S
    rng = np.random.default_rng(dim)
    c, d = filled(i4s, rng, 3, 16, 3, dim, group)
    slots = int32([47, 0, 17, -1, 48, 5, 31])
    n = 7 * 3 * dim
    size = torch.empty(0, dtype=dtype).element_size()
    bufs = [torch.full((n * size + 64,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert all(b.data_ptr() % 32 == 0 for b in bufs)
    number = {F16: S.I4S_F16, BF16: S.I4S_BF16, F32: S.I4S_F32}[dtype]
    stream = torch.cuda.current_stream().cuda_stream
    assert S.i4s_kv_read(d.descriptor, slots.data_ptr(), 7, number, bufs[0].data_ptr() + 16, bufs[1].data_ptr() + 16, stream) == 0
    torch.cuda.synchronize()
    for b, want in zip(bufs, c.read(slots.cpu().numpy())):
        got = b[16:16 + n * size].view(dtype).view(7, 3, dim)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype))
        assert (b[:16] == 0x55).all() and (b[16 + n * size:] == 0x55).all()


# ---------------------------------------------------------------------------
# attention


def test_tree_masks_of_many_sequences_need_no_max_q(i4s):
    """More than 64 tokens in all, few of each sequence; more than 64 of one sequence are refused."""
    say("tree default")
    rng = np.random.default_rng(1)
    c, d = filled(i4s, rng, 12, 16, 1, 64, 32)
    q = torch.from_numpy(rng.standard_normal((100, 2, 64))).to(F16).cuda()
    table, lens, starts = int32(rng.integers(0, 12, (5, 4))), int32([60, 20, 33, 45, 21]), int32([0, 20, 40, 60, 80, 100])
    mask = torch.from_numpy(np.concatenate([(1 << np.arange(20)) | 1] * 5)).cuda()
    got = i4s.kv_attention(d, q, table, lens, q_start=starts, tree_mask=mask)
    assert torch.equal(got, i4s.kv_attention(d, q, table, lens, q_start=starts, max_q=20, tree_mask=mask))
    with pytest.raises(i4s.I4SError):
        i4s.kv_attention(d, q[:65], table[:1], lens[:1], q_start=int32([0, 65]), tree_mask=mask[:65])


# ---------------------------------------------------------------------------
# numbers that 32 bits do not hold


def test_numbers_beyond_32_bits_are_refused(i4s):
    """The C ABI takes 32-bit numbers; none is cut down to its lower half."""
    say("32 bits")
    big = 1 << 32
    d = i4s.kv_cache(4, 16, 2, 64, 32)
    t, l, one = int32([[0, 1]]), int32([20]), int32([1])
    q = torch.zeros(2, 2, 64, dtype=F16).cuda()
    for call in (lambda: i4s.kv_extend(t, l, one, one, one, big + 16, 1), lambda: i4s.kv_extend(t, l, one, one, one, 16, big + 1),
                 lambda: i4s.kv_extend(t, l, one, one, one, 16, -big + 1),
                 lambda: i4s.kv_attention(d, q, t, l, q_start=int32([0, 2]), max_q=big + 1),
                 lambda: i4s.kv_attention(d, q, t, l, q_start=int32([0, 2]), max_len=big),
                 lambda: i4s.kv_attention(d, q, t, l, q_start=int32([0, 2]), max_len=-big),
                 lambda: i4s.token_logprobs(torch.zeros(1, 9).cuda(), torch.zeros(1, dtype=torch.int64).cuda(), top_k=big + 1),
                 lambda: i4s.kv_cache(4, big + 16, 2, 64, 32), lambda: i4s.kv_cache(big + 4, 16, 2, 64, 32),
                 lambda: i4s.KVCache(16, 2 + big, 64, 32, d.k_vals, d.v_vals, d.k_scales, d.v_scales)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
