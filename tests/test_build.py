"""The build's two products do not depend on each other."""
import pathlib
import subprocess

import pytest

from grouped_mixed_input_amd import build


def test_the_library_is_linked_without_the_python_module(monkeypatch, tmp_path):
    # no g++ or no torch headers: the C library is there all the same, and the failure is still reported
    def fails():
        raise RuntimeError("g++ failed")

    def link(cmd, **kw):
        pathlib.Path(cmd[cmd.index("-o") + 1]).write_bytes(b"linked")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "OBJDIR", tmp_path)
    monkeypatch.setattr(build, "LIB", tmp_path / "libgmi.so")
    monkeypatch.setattr(build, "_compile", lambda src, obj: None)
    monkeypatch.setattr(build, "_build_calls", fails)
    monkeypatch.setattr(subprocess, "run", link)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert build.LIB.read_bytes() == b"linked"
