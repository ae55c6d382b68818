"""What is left where the extension module cannot be built or loaded: the library, and the calls that go to it directly."""
import importlib
import subprocess
import types

import pytest

import gemm_rtn_sym_gb300 as w4
from gemm_rtn_sym_gb300 import build as b


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The commands of a build, none of which runs; those of `failing` compilers fail."""
    log = types.SimpleNamespace(run=[], placed=[], failing=set())

    def run(cmd, **kw):
        log.run.append(cmd[0].rsplit("/", 1)[-1])
        return subprocess.CompletedProcess(cmd, int(log.run[-1] in log.failing), "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b.os, "replace", lambda old, new: log.placed.append(new))
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    return log


def test_the_library_is_built_without_torch(commands, monkeypatch):
    monkeypatch.setattr(b, "_have_torch", lambda: False)
    assert b.build() == b.LIB
    assert commands.placed == [b.LIB] and set(commands.run) == {"nvcc"} and len(commands.run) == len(b.sources()) + 1


def test_the_library_is_there_where_the_module_does_not_compile(commands):
    commands.failing.add("g++")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        b.build()
    assert commands.placed == [b.LIB]


def test_both_are_built(commands):
    b.build()
    assert commands.placed == [b.LIB, b.BINDING] and commands.run.count("g++") == 2


def test_calls_of_the_library_do_without_the_module(monkeypatch):
    w4.load()
    real = importlib.import_module

    def no_module(name, *package):
        if name == "._binding":
            raise ImportError("undefined symbol")
        return real(name, *package)

    monkeypatch.setattr(importlib, "import_module", no_module)
    for name in ("_lib", "_fast", "_fast_error"):
        monkeypatch.setattr(w4, name, None)
    assert w4.w4_packed_bytes(4, 256) == 512 and w4.w4_status_string(0)
    for call in (w4._compiled, lambda: w4.w4_kv_copy(None, None, None)):
        with pytest.raises(RuntimeError, match="_binding.so"):
            call()
