"""The serving operators' host layer (``i4s_serve_api.cpp``) built for the CPU
with AddressSanitizer and UndefinedBehaviorSanitizer against stand-ins for the
HIP runtime and the launchers: arguments, launch shapes, refusals."""

import os
import subprocess

import pytest

from test_host_sanitized import CSRC, ENV, HERE, ROOT, SAN, gxx


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("serve_host") / "serve_driver")
    host = os.path.join(HERE, "host")
    cmd = [gxx(), "-std=c++17", "-g", "-O1", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", host,
           *[os.path.join(CSRC, f) for f in ("i4s_api.cpp", "i4s_plan.cpp", "i4s_serve_api.cpp")],
           *[os.path.join(host, f) for f in ("i4s_hip_stub.cpp", "i4s_serve_stub.cpp", "serve_driver.cpp")], "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return out


@pytest.mark.parametrize("arch", [None, "gfx942", "gfx90a"])
def test_every_entry_point(driver, arch):
    r = subprocess.run([driver] + (["--arch", arch] if arch else []), capture_output=True, text=True, env=ENV, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]
    assert r.stdout.startswith("ok "), r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
