"""Build libvsd.so (the C-ABI CUDA library) in-tree for sm_103a.

Each translation unit under ``csrc/`` is compiled in parallel with nvcc, then linked
into ``libvsd.so`` next to this file.  Objects go to ``_build/`` (not committed).
``csrc/binding.cpp``, the Python calls of the 8-bit cache, becomes the extension module
``_binding.so`` beside it, for the torch and the Python that are installed.  The library
needs neither; where the module cannot be built (no torch headers) the library is built all
the same, with a warning, and those calls raise.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libvsd.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_FOR = os.path.join(BUILD, "binding.txt")  # what the module was built for
HEADER = os.path.join(ROOT, "include", "vsd.h")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-Wall", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + [HEADER, os.path.abspath(__file__)]


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, _deps())


def _installed() -> str:
    import torch
    return "torch %s, python %s" % (torch.__version__, sys.version.split()[0])


def binding_up_to_date() -> bool:
    if not _newer(BINDING, [BINDING_SRC, HEADER, os.path.abspath(__file__)]):
        return False
    try:
        with open(BINDING_FOR) as f:
            return f.read() == _installed()
    except (ImportError, OSError):
        return False


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def build_binding() -> str:
    """Compile csrc/binding.cpp against the installed torch; returns the module's path."""
    import torch
    os.makedirs(BUILD, exist_ok=True)
    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = BINDING + ".%d.tmp" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           "-DVSD_BUILT_FOR=\"%s\"" % _installed(),
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    for p in include:
        cmd += ["-isystem", p]
    cmd += [BINDING_SRC, "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-L" + os.path.join(os.path.dirname(os.path.dirname(nvcc())), "lib64"), "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(_installed())
    return BINDING


def _binding_or_warning(wait) -> None:
    try:
        wait()
    except Exception as e:  # noqa: BLE001 (no torch, no headers, no compiler)
        warnings.warn("the calls of the 8-bit cache are not available: _binding.so was not built: %s" % e,
                      RuntimeWarning, stacklevel=3)


def build(force: bool = False, verbose: bool = False, extra_flags=(), out: str = None,
          objdir: str = None) -> str:
    """Compile and link libvsd.so, and the binding beside it, where they are not up to date;
    returns the library's path.  `out` / `objdir` build a separate copy of the library (e.g.
    with other -D settings in `extra_flags`) without touching the main one."""
    with_binding = out is None and (force or not binding_up_to_date())
    if out is None and not force and library_up_to_date():
        if with_binding:
            _binding_or_warning(build_binding)
        return LIB
    lib_path = out or LIB
    objdir = objdir or BUILD
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        binding = ex.submit(build_binding) if with_binding else None
        objs = list(ex.map(compile_one, srcs))
    tmp = lib_path + ".%d.tmp" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, lib_path)
    if binding is not None:
        _binding_or_warning(binding.result)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
