"""Build the in-tree C-ABI library libzero_step.so for sm_103a.

The translation units (the step's CUDA kernels and entry points, the
language-model operators' six, and the host-only plan and checkpoint code)
are compiled in parallel by nvcc and linked into one shared library with the
CUDA runtime linked statically, so the library needs no libcudart at load time
and can be loaded (and its host-only entry points called) on a machine without
a GPU.

The Python module _lm (csrc/lm_binding.cpp, the tensors' checks of the
language-model operators) is compiled beside it with the host compiler against
the installed torch's headers.  The library needs neither: without a torch that
has CUDA the module is left out, and if it fails to compile the library is in
place all the same.
"""
from __future__ import annotations

import fcntl
import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libzero_step.so")
BUILD_DIR = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]
SOURCES = [os.path.join(CSRC, "zero_step.cu"), os.path.join(CSRC, "plan.cpp"),
           os.path.join(CSRC, "ckpt.cpp"), os.path.join(CSRC, "lm_embed.cu"),
           os.path.join(CSRC, "lm_norm.cu"), os.path.join(CSRC, "lm_xent.cu"),
           os.path.join(CSRC, "lm_layer_norm.cu"), os.path.join(CSRC, "lm_loss.cu"),
           os.path.join(CSRC, "lm_clip.cu")]
EXT = os.path.join(PKG, "_lm.so")
EXT_SOURCE = os.path.join(CSRC, "lm_binding.cpp")
HEADERS = [os.path.join(INCLUDE, "zero_step.h")] + sorted(
    os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh"))


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def torch_dir():
    """Where a torch with CUDA is installed, or None."""
    spec = importlib.util.find_spec("torch")
    for d in (spec and spec.submodule_search_locations) or ():
        if os.path.exists(os.path.join(d, "lib", "libc10_cuda.so")):
            return d
    return None


def _older(built, sources) -> bool:
    if not os.path.exists(built):
        return True
    t = os.path.getmtime(built)
    return any(os.path.getmtime(p) > t for p in [*sources, *HEADERS, __file__])


def _lib_stale() -> bool:
    return _older(LIB, SOURCES)


def _ext_for() -> str:
    """What the module is tied to: the torch and the Python it was built against."""
    version = runpy.run_path(os.path.join(torch_dir(), "version.py"))["__version__"]
    return f"{torch_dir()} {version} {sysconfig.get_config_var('EXT_SUFFIX')}\n"


def _ext_stale() -> bool:
    if torch_dir() is None:
        return False
    if _older(EXT, [EXT_SOURCE]) or not os.path.exists(EXT + ".for"):
        return True
    with open(EXT + ".for") as f:
        return f.read() != _ext_for()


def _stale() -> bool:
    return _lib_stale() or _ext_stale()


def compile_commands():
    os.makedirs(BUILD_DIR, exist_ok=True)
    cmds, objs = [], []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmds.append([nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj])
        objs.append(obj)
    link = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", LIB + ".tmp", *objs]
    return cmds, link


def ext_command():
    torch = torch_dir()
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    include = [INCLUDE, os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_path("include"), cuda]
    libs = os.path.join(torch, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            *(x for i in include for x in ("-I", i)), EXT_SOURCE, "-o", EXT + ".tmp", "-L", libs,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{libs}"]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    # several processes may find it stale at once: one builds, the others wait
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(os.path.join(BUILD_DIR, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        lib, ext = force or _lib_stale(), _ext_stale() or (force and torch_dir() is not None)
        if torch_dir() is None:
            print("no torch with CUDA here: the module _lm of the language-model operators is "
                  "left out", file=sys.stderr)
        _build(lib, ext, verbose)
    return LIB


def _build(lib: bool, ext: bool, verbose: bool) -> None:
    cmds, link = compile_commands() if lib else ([], None)
    ext_cmds = [ext_command()] if ext else []
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for c in cmds + ext_cmds]
    failed = {}
    for i, (c, p) in enumerate(zip(cmds + ext_cmds, procs)):
        out, _ = p.communicate()
        if verbose and out:
            sys.stdout.write(out)
        if p.returncode != 0:
            failed[i] = f"$ {' '.join(c)}\n{out}"
    if lib and not any(i < len(cmds) for i in failed):
        subprocess.run(link, check=True)
        os.replace(LIB + ".tmp", LIB)
    if failed:
        raise RuntimeError("the build failed:\n" + "\n".join(failed.values()))
    if ext:
        os.replace(EXT + ".tmp", EXT)
        with open(EXT + ".for", "w") as f:
            f.write(_ext_for())


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
