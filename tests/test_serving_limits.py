"""CPU tests of the serving ABI: its binding, and each size at the border that the header gives it."""

import os

import pytest

from int4_sparse_gemv_amd import _binding as B
from int4_sparse_gemv_amd import _serve_binding as S


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from int4_sparse_gemv_amd import build
        build.build()
    return S.load()


def test_binding_has_the_library_s_functions_and_no_others(lib):
    for name in S.SIGNATURES:
        assert getattr(S, name) is getattr(lib, name), name
    with pytest.raises(AttributeError):
        S.i4s_run
