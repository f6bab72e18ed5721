"""The build's steps on machines that hold less than this one: the C library
needs hipcc alone, the Python binding torch's headers.  Compiles nothing."""
import sys

import pytest

from bit_gemm_block_amd import build as b


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """What a build would compile and link, in order."""
    done = []
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(b, "_compile", lambda src, extra: done.append(src) or src + ".o")
    monkeypatch.setattr(b, "_link", lambda out, args: done.append(out))
    return done


def test_library_without_torch(steps, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)      # as where it is not installed
    monkeypatch.setitem(sys.modules, "torch.utils", None)
    assert b.build() == b.LIB
    assert sorted(steps[:-1]) == sorted(b.SOURCES) and steps[-1] == b.LIB
    assert "torch" in capsys.readouterr().out            # says what is missing


def test_library_and_binding_with_torch(steps, monkeypatch):
    commands = []
    ok = type("Done", (), {"returncode": 0})
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: commands.append(cmd) or ok)
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(b.shutil, "which", lambda name: None)     # no g++: hipcc compiles host code as well
    assert b.build() == b.LIB
    assert steps[-2:] == [b.LIB, b.BINDING]
    assert [c[0] for c in commands] == [b.hipcc()]


def test_a_binding_that_does_not_compile_is_an_error(steps, monkeypatch):
    bad = type("Done", (), {"returncode": 1, "stdout": "", "stderr": "no such header"})
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: bad)
    with pytest.raises(RuntimeError, match="no such header"):
        b.build()
    assert steps[-1] == b.LIB                             # the library is there all the same
