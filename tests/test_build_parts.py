"""The build's two parts: the library, which needs nvcc alone, and the binding,
which is of one torch and one Python."""
import importlib.util
import os
import subprocess

import pytest

from fibonacci_spaced_sparse_gb300 import _lib, build

TINY = '#include "sfa.h"\nextern "C" int sfa_version(void) { return 1; }\n'


@pytest.fixture
def place(monkeypatch, tmp_path):
    """A build of one small source file in a folder of its own; counts the compilers' runs."""
    src = tmp_path / "tiny.cu"
    src.write_text(TINY)
    out = tmp_path / "_build"
    monkeypatch.setattr(build, "BUILD", str(out))
    monkeypatch.setattr(build, "LIB", str(out / "libsfa.so"))
    monkeypatch.setattr(build, "BIND", str(out / "_sfa_bind.so"))
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    runs = []
    real = subprocess.run

    def run(cmd, **kw):
        runs.append(os.path.basename(cmd[0]))
        return real(cmd, **kw)

    monkeypatch.setattr(subprocess, "run", run)
    return out, runs


def _refuse():
    raise RuntimeError("g++ failed")


def test_the_library_is_built_without_the_binding(place, monkeypatch):
    out, runs = place
    monkeypatch.setattr(build, "_compile_bind", _refuse)
    assert build.build(binding=False) == str(out / "libsfa.so")
    assert (out / "libsfa.so").exists() and not (out / "_sfa_bind.so").exists()
    assert runs == ["nvcc", "nvcc"]
    build.build(binding=False)                      # nothing to do
    assert len(runs) == 2


def test_no_torch_no_binding(place, monkeypatch):
    out, runs = place
    monkeypatch.setattr(build, "_compile_bind", _refuse)
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    build.build()
    build.build()
    assert (out / "libsfa.so").exists() and runs == ["nvcc", "nvcc"]


def test_a_binding_that_fails_leaves_the_library(place, monkeypatch):
    out, runs = place
    monkeypatch.setattr(build, "_compile_bind", _refuse)
    for _ in range(2):                              # loud each time, the library built once
        with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
            build.build()
        assert (out / "libsfa.so").exists() and runs == ["nvcc", "nvcc"]


def test_another_torch_is_noticed(place, monkeypatch):
    out, runs = place
    made = []

    def compile_bind():
        made.append(build.binding_key())
        obj = out / "bind.o"
        subprocess.run(["g++", "-fPIC", "-x", "c++", "-c", "-o", str(obj), "/dev/null"], check=True)
        return str(obj)

    monkeypatch.setattr(build, "_compile_bind", compile_bind)
    build.build()
    build.build()
    assert len(made) == 1 and build.built_for(build.BIND) == build.binding_key()
    monkeypatch.setattr(_lib, "_bind", None)
    monkeypatch.setattr(_lib, "BIND_PATH", build.BIND)
    here = build.binding_key()
    monkeypatch.setattr(build, "binding_key", lambda: "torch 9.9 elsewhere, Python 3.12")
    with pytest.raises(RuntimeError, match="built for " + here.replace("+", "\\+")):
        _lib.bind()
    build.build()
    assert made == [here, build.binding_key()]
    os.remove(build.BIND + ".key")                  # of a build before keys were kept
    with pytest.raises(RuntimeError, match="another torch"):
        _lib.bind()
