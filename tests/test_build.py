"""What is left where the extension module cannot be built or loaded: the library, and the calls that go to it directly."""
import importlib
import os
import re
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


SAID = """ptxas info    : Compiling entry function '_ZN2w418attn_prefix_kernelILi128ELb1EEEvNS_10PrefixArgsENS0_5BoxesE' for 'sm_103a'
ptxas info    : Function properties for _ZN2w418attn_prefix_kernelILi128ELb1EEEvNS_10PrefixArgsENS0_5BoxesE
    64 bytes stack frame, 156 bytes spill stores, 496 bytes spill loads
ptxas info    : Used %d registers, used 2 barriers, 64 bytes cumulative stack size, 5440 bytes smem
"""


def test_a_compiler_that_gives_other_registers_is_reported(commands, monkeypatch):
    """The kernel's warps share registers out: with another number of them at launch its calls are refused.  The build says so,
    with everything in place."""
    said = [96]
    run = b.subprocess.run
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(run(cmd, **kw), 0, "", SAID % said[0]))
    b.build()
    said[0] = 88
    commands.placed.clear()
    with pytest.raises(RuntimeError, match="registers"):
        b.build()
    assert commands.placed == [b.LIB, b.BINDING]


def test_registers_of_the_kernels_that_share_them_out():
    """As built, and as the source counts on them."""
    path = os.path.join(b.BUILD, "kernels.txt")
    if not os.path.exists(path):
        b.build()
    with open(path) as f:
        have = b.registers(f.read())
    with open(os.path.join(b.CSRC, "w4_attn_prefix.cu")) as f:
        wanted = int(re.search(r"kLaunchRegs = (\d+)", f.read())[1])
    for part, n in b.SHARED_OUT.items():
        assert n == wanted and [m for name, m in have.items() if part in name] == [n]
    # no other kernel shares registers out
    sources = [f for f in os.listdir(b.CSRC) if "setmaxnreg" in open(os.path.join(b.CSRC, f)).read()]
    assert sources == ["w4_attn_prefix.cu"]
