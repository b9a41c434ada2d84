"""What the build makes, with a compiler that only notes its calls."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch  # noqa: F401  (imported before a test hides it)

from block_scaled_fp8_act_gb300 import build as fp8build


@pytest.fixture
def calls(monkeypatch, tmp_path):
    for name, path in (("BUILD_DIR", tmp_path), ("LIB_PATH", tmp_path / "libfp8act.so"), ("EXT_PATH", tmp_path / "_fp8act.so")):
        monkeypatch.setattr(fp8build, name, str(path))
    made = []

    def run(cmd, **_):
        made.append(cmd)
        fails = getattr(run, "fails", None)
        if fails and fails(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(fp8build.subprocess, "run", run)
    return made, run


def test_library_without_torch(calls, monkeypatch):
    """The C ABI needs no PyTorch, and neither does its build."""
    made, _ = calls
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        assert fp8build.build() == fp8build.LIB_PATH and os.path.exists(fp8build.LIB_PATH)
        assert len(made) == len(fp8build.sources()) + 1 and not os.path.exists(fp8build.EXT_PATH)
        fp8build.build()
        assert len(made) == len(fp8build.sources()) + 1  # nothing is stale
    fp8build.build()
    assert os.path.exists(fp8build.EXT_PATH)  # made once PyTorch is there


def test_library_is_there_if_the_binding_does_not_compile(calls):
    made, run = calls
    run.fails = lambda cmd: cmd[0] == "g++"
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        fp8build.build()
    assert os.path.exists(fp8build.LIB_PATH) and not os.path.exists(fp8build.EXT_PATH)
