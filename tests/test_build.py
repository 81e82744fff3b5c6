"""Building: libssd.so does not depend on torch, and the compiled calls follow
the torch that they were built against.  Nothing in the tree is rebuilt here."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import mamba_ssd_sequence_b200 as ssd
from mamba_ssd_sequence_b200 import build as ssd_build


@pytest.fixture
def built(monkeypatch, tmp_path):
    """A built tree whose compiled calls may be replaced or removed."""
    ssd_build.build()
    copy = tmp_path / "_binding.so"
    shutil.copy2(ssd_build.BINDING, copy)
    monkeypatch.setattr(ssd_build, "BINDING", str(copy))
    return copy


def test_without_torch_the_library_is_built(built, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    with pytest.warns(UserWarning, match="recurrence and the norms"):
        assert ssd_build.build() == ssd_build.LIB
    assert os.path.exists(ssd_build.LIB) and not built.exists()
    with pytest.raises(ImportError):
        ssd_build.build_binding()


def test_without_a_compiler_for_the_calls_the_library_is_built(built, monkeypatch):
    monkeypatch.setenv("CXX", shutil.which("false"))
    os.utime(built, (0, 0))  # out of date
    with pytest.warns(UserWarning, match="failed"):
        assert ssd_build.build() == ssd_build.LIB
    assert not built.exists()
    with pytest.raises(RuntimeError, match="failed"):
        ssd_build.build_binding()


def test_another_torch_rebuilds_the_calls(built, monkeypatch):
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "")

    monkeypatch.setattr(ssd_build.subprocess, "run", run)
    assert ssd_build.build_binding() == str(built) and not runs  # up to date
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(RuntimeError):
        ssd_build.build_binding()
    assert len(runs) == 1


def test_calls_of_another_torch_are_refused(monkeypatch):
    ssd_build.build()
    monkeypatch.setattr(ssd, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(RuntimeError, match="built against torch"):
        ssd.load_binding()
