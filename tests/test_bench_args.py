"""Arguments that ``bench.py`` refuses before it touches a GPU."""

import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args,ok", [(["--verify-step", "1"], True), (["--verify-step", "16", "--context", "0"], True),
                                     (["--verify-step", "0"], False), (["--verify-step", "17"], False),
                                     (["--verify-step", "4", "--context", "-1"], False), ([], True)])
def test_verify_step_range(monkeypatch, capsys, args, ok):
    sys.path.insert(0, ROOT)
    import bench
    monkeypatch.setattr(sys, "argv", ["bench.py", *args])
    if ok:
        assert bench.parse().context >= 0
    else:
        with pytest.raises(SystemExit) as e:
            bench.parse()
        err = capsys.readouterr().err
        assert e.value.code == 2 and ("takes 1 to 16" in err or "takes 0 or more" in err)
