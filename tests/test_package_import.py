"""What importing the package needs: its own names do without torch, which the serving operators bring in."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HIDDEN = "import sys; sys.modules['torch'] = None"
# a finder that knows no torch, as where it is not installed
ABSENT = """import sys
class No:
    def find_spec(self, name, path=None, target=None):
        if name == 'torch' or name.startswith('torch.'):
            raise ModuleNotFoundError("No module named 'torch'", name='torch')
sys.meta_path.insert(0, No())"""


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


@pytest.mark.parametrize("without", [HIDDEN, ABSENT], ids=["hidden", "absent"])
def test_star_import_without_torch(without):
    out = python(without + "\nfrom int4_sparse_gemv_amd import *\nprint(pack_sizes.__name__, I4SError.__name__, 'kv_cache' in dir())")
    assert out.split() == ["pack_sizes", "I4SError", "False"]


def test_serving_names_without_torch_say_what_is_missing():
    out = python(HIDDEN + "\nimport int4_sparse_gemv_amd as i\ntry:\n    i.kv_cache\nexcept ImportError as e:\n    print(e.name)")
    assert out.strip() == "torch"


def test_star_import_with_torch():
    pytest.importorskip("torch")
    out = python("from int4_sparse_gemv_amd import *\nprint(kv_attention.__module__, KVCache.__name__, run.__name__)")
    assert out.split() == ["int4_sparse_gemv_amd.serving", "KVCache", "run"]


def test_import_alone_leaves_torch_out():
    assert python("import sys\nimport int4_sparse_gemv_amd\nprint('torch' in sys.modules)").strip() == "False"
