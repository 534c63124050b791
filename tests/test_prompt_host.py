"""The prompt's operators without a GPU: their host layer
(``i4s_prompt_api.cpp``) built for the CPU with AddressSanitizer and
UndefinedBehaviorSanitizer against stand-ins for the HIP runtime and the
launchers, the package's names, and the arguments of the step's benchmark."""

import os
import subprocess
import sys

import pytest

from test_host_sanitized import CSRC, ENV, HERE, ROOT, SAN, gxx


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("prompt_host") / "prompt_driver")
    host = os.path.join(HERE, "host")
    cmd = [gxx(), "-std=c++17", "-g", "-O1", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", host,
           *[os.path.join(CSRC, f) for f in ("i4s_api.cpp", "i4s_plan.cpp", "i4s_serve_api.cpp", "i4s_prompt_api.cpp")],
           *[os.path.join(host, f) for f in ("i4s_hip_stub.cpp", "i4s_serve_stub.cpp", "i4s_prompt_stub.cpp", "prompt_driver.cpp")],
           "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return out


@pytest.mark.parametrize("arch", [None, "gfx942", "gfx90a"])
def test_every_entry_point(driver, arch):
    r = subprocess.run([driver] + (["--arch", arch] if arch else []), capture_output=True, text=True, env=ENV, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]
    assert r.stdout.startswith("ok "), r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr


def test_package_names():
    pytest.importorskip("torch")
    code = ("from int4_sparse_gemv_amd import *\nimport int4_sparse_gemv_amd as i\n"
            "print(prompt_attention.__module__, MXTensor.__name__, mx_quantize is i.mx_quantize, mx_read is i.mx_read, "
            "mx_product is i.mx_product)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.stdout.split() == ["int4_sparse_gemv_amd.prompt", "MXTensor", "True", "True", "True"], r.stderr[-2000:]


def test_names_without_torch_say_what_is_missing():
    code = ("import sys; sys.modules['torch'] = None\nimport int4_sparse_gemv_amd as i\ntry:\n    i.mx_product\n"
            "except ImportError as e:\n    print(e.name)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.stdout.strip() == "torch", r.stderr[-2000:]


@pytest.mark.parametrize("args,ok", [(["--prompt-step", "1"], True), (["--prompt-step", "65536"], True),
                                     (["--prompt-step", "0"], False), (["--prompt-step", "65537"], False)])
def test_prompt_step_range(monkeypatch, capsys, args, ok):
    import bench
    monkeypatch.setattr(sys, "argv", ["bench.py", *args])
    if ok:
        assert bench.parse().prompt_step >= 1
    else:
        with pytest.raises(SystemExit) as e:
            bench.parse()
        assert e.value.code == 2 and "takes 1 to 65536" in capsys.readouterr().err


def test_a_matrix_keeps_its_buffers():
    """The descriptor has the addresses of the tensors that a matrix was made of: another tensor in their place is refused,
    where the calls would go on with the old one's memory."""
    torch = pytest.importorskip("torch")
    from int4_sparse_gemv_amd import prompt
    vals, scales = torch.zeros(2, 2, 1024, dtype=torch.uint8), torch.zeros(2, 1, 256, dtype=torch.uint8)
    m = prompt.MXTensor.__new__(prompt.MXTensor)._hold(20, 64, vals, scales, -1)
    for name, value in (("vals", vals.clone()), ("scales", scales.clone()), ("rows", 5), ("cols", 32), ("shape", (5, 32)),
                        ("index", 0), ("descriptor", None), ("address", 0), ("other", 1)):
        with pytest.raises(AttributeError):
            setattr(m, name, value)
    assert m.vals is vals and m.scales is scales and (m.rows, m.cols, m.shape) == (20, 64, (20, 64))
    assert (m.descriptor.vals, m.descriptor.scales) == (vals.data_ptr(), scales.data_ptr())
    m.vals[:] = 7  # what they hold is the caller's
