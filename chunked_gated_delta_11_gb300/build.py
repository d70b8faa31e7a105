"""Build libkda.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ compiles to an object in parallel, then nvcc links them
into ``chunked_gated_delta_11_gb300/_build/libkda.so``.  ``-Xptxas -v``
register and shared-memory reports go to ``_build/ptxas.log``.  The Python
extension of the softmax-attention calls, ``_build/attn_binding.so``, is compiled
beside them with g++ against torch's and Python's headers and linked to libkda.
It belongs to the torch and the Python that it was built with (named in
``_build/attn_binding.tag``).  Where it cannot be built the rest can: build()
warns, and the attention calls raise.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libkda.so")
BINDING = os.path.join(BUILD, "attn_binding.so")
BINDING_SRC = os.path.join(CSRC, "attn_binding.cpp")
BINDING_TAG = os.path.join(BUILD, "attn_binding.tag")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC,-O2", "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libkda cannot be built")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def _lib_up_to_date() -> bool:
    deps = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                        if f.endswith((".cuh", ".h"))]
    return _newer(LIB, [*deps, os.path.join(INCLUDE, "kda.h"), os.path.abspath(__file__)])


def binding_tag() -> str:
    """What the binding's binary interface depends on."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def binding_built_for() -> str:
    """The binding_tag() that the binding was built with; "" if it is not there."""
    if not (os.path.exists(BINDING) and os.path.exists(BINDING_TAG)):
        return ""
    with open(BINDING_TAG) as f:
        return f.read()


def _binding_up_to_date() -> bool:
    return (binding_built_for() == binding_tag()
            and _newer(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "kda.h"), os.path.abspath(__file__)]))


def up_to_date() -> bool:
    return _lib_up_to_date() and _binding_up_to_date()


def _compile_binding() -> str:
    import torch  # noqa: F401  (its headers and libraries belong to this interpreter's torch)
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [INCLUDE, os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    obj = os.path.join(BUILD, "attn_binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for d in inc for x in ("-I", d)], "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-lkda", "-Wl,-rpath,$ORIGIN", "-L", libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _remove_binding()
    os.replace(tmp, BINDING)
    with open(BINDING_TAG, "w") as f:
        f.write(binding_tag())


def _remove_binding() -> None:
    for old in (BINDING_TAG, BINDING):
        if os.path.exists(old):
            os.remove(old)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_binding) if force or not _binding_up_to_date() else None
        if force or not _lib_up_to_date():
            _build_lib(verbose)
        if binding is not None:
            try:
                _link_binding(binding.result())
            except Exception as e:  # the KDA calls do without it
                _remove_binding()
                warnings.warn(f"the attention binding was not built: {e}")
    return LIB


def _build_lib(verbose: bool) -> None:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, sources()))
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for obj, log in results:
            f.write(f"== {os.path.basename(obj)}\n{log}\n")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(open(os.path.join(BUILD, "ptxas.log")).read())


if __name__ == "__main__":
    print(build(force=True, verbose=True))
