"""Builds libw4.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu file under csrc/ is compiled in parallel to an object under _build/,
then linked into gemm_rtn_sym_gb300/libw4.so.  csrc/binding.cpp becomes the
extension module gemm_rtn_sym_gb300/_binding.so, which calls the library; it is
left out where torch is not there, as for a user of the C library alone
(``python gemm_rtn_sym_gb300/build.py``).  IEEE division and no
flush-to-zero are required by the quantiser, so no fast-math flags are used.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libw4.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=true",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libw4.so")
    return path


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(src: str, extra: list[str]) -> tuple[str, str]:
    """The object of a source, and what the assembler says about its kernels."""
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + extra + ["-Xptxas", "-v", "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


#: Kernels whose warps hand registers to one another, by their name in the object, and what a thread has to be launched with
#: (kLaunchRegs beside them): with fewer, the warps that ask for more would wait for ever, so that the calls refuse to launch.
SHARED_OUT = {"attn_prefix_kernelILi64ELb1E": 96, "attn_prefix_kernelILi128ELb1E": 96}


def registers(text: str) -> dict[str, int]:
    """Registers of each kernel in what the assembler says."""
    found = re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", text, re.S)
    return {name: int(n) for name, n in found}


def _check_registers(text: str) -> None:
    have = registers(text)
    for part, wanted in SHARED_OUT.items():
        got = {n for name, n in have.items() if part in name}
        if got - {wanted}:
            raise RuntimeError(f"this compiler gives {part} {sorted(got)} registers instead of {wanted}: attention over shared "
                               "prefixes in 8 bits will be refused (the library is there for all else)")


def _have_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _compile_binding() -> str:
    """Object of the extension module (host code against torch's headers)."""
    import torch

    obj = os.path.join(BUILD, "binding.o")
    home = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    top = os.path.join(os.path.dirname(torch.__file__), "include")
    includes = [os.path.join(ROOT, "include"), top, os.path.join(top, "torch", "csrc", "api", "include"),
                os.path.join(home, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [x for i in includes for x in ("-isystem", i)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libw4.so", "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile and link libw4.so and the extension module; returns the library's path.  The library is there also where
    the module cannot be built, which raises."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(12, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding) if _have_torch() else None
        made = list(ex.map(lambda s: _compile(s, list(extra or [])), srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-Xlinker", "-soname=libw4.so", "-o", tmp] + [obj for obj, _ in made]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding is not None:
        _link_binding(binding.result())
    said = "".join(text for _, text in made)
    with open(os.path.join(BUILD, "kernels.txt"), "w") as f:
        f.write(said)
    _check_registers(said)
    if verbose:
        print(f"built {LIB}" + ("" if binding is not None else " (no torch: without the extension module)"))
    return LIB


if __name__ == "__main__":
    build(verbose=True)
