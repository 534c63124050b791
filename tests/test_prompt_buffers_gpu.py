"""Buffers of the microscaled format on the GPU: the smallest alignment that the header asks for."""

import ctypes

import numpy as np
import pytest

from oracle import prompt_oracle as O
from test_prompt_gpu import BF16, F16, F32, draw, f64, i4s, say  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype,number", [(F16, 0), (BF16, 1), (F32, 2)])
@pytest.mark.parametrize("rows,cols", [(3, 96), (40, 544), (1100, 8224)])
def test_read_to_an_address_of_16_bytes(i4s, rows, cols, dtype, number):
    """Every buffer begins 16 bytes past one of 32, and nothing before or behind the values changes."""
    from int4_sparse_gemv_amd import _binding as B
    from int4_sparse_gemv_amd import _prompt_binding as P
    say(rows, cols, dtype)
    m = i4s.mx_quantize(draw(np.random.default_rng(rows), rows, cols, F16))
    held = []
    for t in (m.vals, m.scales):
        held.append(torch.full((t.numel() + 64,), 0xA5, dtype=torch.uint8, device="cuda"))
        held[-1][16:16 + t.numel()] = t.flatten()
    size = rows * cols
    out = torch.full((size + 64,), 7.0, dtype=dtype, device="cuda")
    first = 16 // out.element_size()
    assert all(x.data_ptr() % 32 == 0 for x in (*held, out))
    part = P.i4s_mx(rows, cols, held[0].data_ptr() + 16, held[1].data_ptr() + 16)
    B.check(P.i4s_mx_read(ctypes.byref(part), number, out.data_ptr() + 16, torch.cuda.current_stream().cuda_stream), "i4s_mx_read")
    assert torch.equal(out[first:first + size].view(rows, cols), i4s.mx_read(m, dtype))
    assert (out[:first] == 7.0).all() and (out[first + size:] == 7.0).all()
    if dtype == F32:
        code, scale = O.mx_unpack(m.vals.cpu().numpy().reshape(-1), m.scales.cpu().numpy().reshape(-1), rows, cols)
        np.testing.assert_array_equal(f64(out[first:first + size]).reshape(rows, cols), O.mx_values(code, scale))
