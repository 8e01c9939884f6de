"""The build of the compiled binding (no GPU): libra.so does not depend on it, and one made for another torch or
Python is made anew."""
import os
import shutil
import subprocess
import warnings

import pytest


@pytest.fixture()
def b(monkeypatch, tmp_path):
    from int4_quantized_flashattention_b200 import _build
    _build.build()                                      # what is there already stays
    objects = [f for f in os.listdir(_build.OBJDIR) if f.endswith(".o")]
    for f in objects:
        shutil.copy2(os.path.join(_build.OBJDIR, f), tmp_path / f)   # with its time
    monkeypatch.setattr(_build, "OBJDIR", str(tmp_path))
    monkeypatch.setattr(_build, "BIND", str(tmp_path / "_bind.so"))
    return _build


def _compiler(monkeypatch, b, error=None):
    """A stand-in for g++ that counts its calls and writes an empty file."""
    calls = []

    def run(cmd, check=True):
        assert cmd[0] == "g++", cmd
        calls.append(cmd)
        if error is not None:
            raise error
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
    monkeypatch.setattr(b.subprocess, "run", run)
    return calls


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), subprocess.CalledProcessError(1, "g++")])
def test_library_without_the_binding(b, monkeypatch, error):
    calls = _compiler(monkeypatch, b, error)
    with open(b.BIND, "w"):
        pass                                            # a binding that does not fit
    with pytest.warns(RuntimeWarning, match="binding"):
        assert b.build() == b.LIB
    assert len(calls) == 1 and os.path.exists(b.LIB) and not os.path.exists(b.BIND)


def test_made_anew_for_another_torch(b, monkeypatch):
    import torch
    calls = _compiler(monkeypatch, b)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        b.build()
        b.build()
        assert len(calls) == 1
        monkeypatch.setattr(torch, "__version__", "0.0")
        b.build()
        b.build()
        assert len(calls) == 2
