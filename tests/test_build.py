"""The build's order, on the CPU with the compilers' calls replaced: the C-ABI
library needs no torch, and what goes wrong with the torch extension does not
take the library away."""
import importlib.util
import subprocess

import pytest

from byte_level_bpe_amd import build as libbuild


@pytest.fixture
def dry(tmp_path, monkeypatch):
    """build() into tmp_path, whose compiler writes empty outputs."""
    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")
    for name in ("OUT", "SERVING", "BUILD"):
        monkeypatch.setattr(libbuild, name, str(tmp_path / name))
    monkeypatch.setattr(libbuild.subprocess, "run", run)
    return tmp_path


def test_library_without_torch(dry, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))

    def serving():
        raise ModuleNotFoundError("No module named 'torch'")
    monkeypatch.setattr(libbuild, "_serving", serving)
    assert libbuild.build() == libbuild.OUT
    assert (dry / "OUT").exists() and not (dry / "SERVING").exists()
    assert "torch is not installed" in capsys.readouterr().err


def test_library_before_a_failing_extension(dry, monkeypatch):
    def serving():
        raise RuntimeError("compile failed")
    monkeypatch.setattr(libbuild, "_serving", serving)
    with pytest.raises(RuntimeError):
        libbuild.build()
    assert (dry / "OUT").exists()
