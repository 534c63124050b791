"""CPU tests of the serving ABI: its binding, and each size at the border that the header gives it."""

import os
import subprocess

import pytest

from int4_sparse_gemv_amd import _binding as B
from int4_sparse_gemv_amd import _serve_binding as S
from test_host_sanitized import CSRC, ENV, HERE, ROOT, SAN, gxx


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


def test_sizes_at_their_borders(tmp_path):
    """In a CPU build of the host layer with sanitizers, against stand-ins: nothing is launched."""
    out, host = str(tmp_path / "limits"), os.path.join(HERE, "host")
    cmd = [gxx(), "-std=c++17", "-g", "-O1", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", host,
           *[os.path.join(CSRC, f) for f in ("i4s_api.cpp", "i4s_plan.cpp", "i4s_serve_api.cpp")],
           *[os.path.join(host, f) for f in ("i4s_hip_stub.cpp", "i4s_serve_stub.cpp", "limits_driver.cpp")], "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([out], capture_output=True, text=True, env=ENV, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
