"""Build libprism.so in-tree for sm_103a (nvcc and g++; no cmake).

Each ``csrc/*.cu`` translation unit is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a`` and linked into
``deterministic_w8a8_int8_gb300/libprism.so`` against the shared CUDA runtime.
``csrc/decode_py.cpp``, the Python side of the decode-step entry points, becomes
the extension module ``_decode.so`` beside it (g++; Python's and torch's headers).
Without these the library is built all the same, with a warning.
Set ``PRISM_PTXAS_VERBOSE=1`` to print ptxas register and spill reports.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libprism.so")
MODULE_SRC = os.path.join(CSRC, "decode_py.cpp")
MODULE_PATH = os.path.join(PKG, "_decode.so")
STAMP_PATH = os.path.join(BUILD_DIR, "decode_py.stamp")   # what the module was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _cxx() -> str | None:
    for cand in (os.environ.get("CXX"), shutil.which("g++"), shutil.which("c++")):
        if cand:
            return cand
    return None


def _cuda_lib_dir(nvcc: str) -> str:
    root = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    for sub in ("lib64", "lib", "targets/sbsa-linux/lib", "targets/x86_64-linux/lib"):
        d = os.path.join(root, sub)
        if os.path.isdir(d):
            return d
    return os.path.join(root, "lib64")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec is not None and spec.submodule_search_locations else None


def _module_lacks() -> str | None:
    """What is missing here that the extension module cannot be built without."""
    if _cxx() is None:
        return "g++"
    torch_dir = _torch_dir()
    if torch_dir is None or not os.path.isdir(os.path.join(torch_dir, "include", "torch", "csrc")):
        return "torch's headers"
    return None if os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")) else "Python's headers"


def _module_stamp() -> str:
    """The torch and the Python that the module is built for."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sysconfig.get_config_var('EXT_SUFFIX')}\n{_torch_dir()}\n{f.read()}"


def _module_up_to_date() -> bool:
    if not os.path.exists(MODULE_PATH) or not os.path.exists(STAMP_PATH):
        return False
    with open(STAMP_PATH) as f:
        if f.read() != _module_stamp():
            return False
    return os.path.getmtime(MODULE_PATH) >= max(os.path.getmtime(MODULE_SRC), os.path.getmtime(os.path.join(INCLUDE, "prism.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps()) and (_module_lacks() is not None or _module_up_to_date())


def _run(what: str, cmd: list[str]) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")


def _compile_module(nvcc: str) -> str:
    obj = os.path.join(BUILD_DIR, "decode_py.o")
    torch_include = os.path.join(_torch_dir(), "include")
    dirs = [INCLUDE, torch_include, os.path.join(torch_include, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
    _run("g++ on decode_py.cpp", [_cxx(), "-O2", "-std=c++17", "-fPIC", *(a for d in dirs for a in ("-I", d)),
                                  "-c", MODULE_SRC, "-o", obj])
    return obj


def _link_module(obj: str, libdir: str) -> None:
    torch_lib = os.path.join(_torch_dir(), "lib")
    tmp = MODULE_PATH + f".tmp{os.getpid()}"
    _run("link of _decode.so", [_cxx(), "-shared", obj, "-o", tmp, "-L", PKG, "-lprism", "-L", torch_lib, "-lc10", "-lc10_cuda",
                                "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
                                f"-Wl,-rpath,$ORIGIN:{torch_lib}:{libdir},-rpath-link,{libdir}"])
    os.replace(tmp, MODULE_PATH)
    with open(STAMP_PATH, "w") as f:
        f.write(_module_stamp())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if os.environ.get("PRISM_PTXAS_VERBOSE"):
        flags += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose or os.environ.get("PRISM_PTXAS_VERBOSE"):
            print(r.stderr, end="")
        return obj

    lacks = _module_lacks()
    if lacks is not None:
        warnings.warn(f"_decode.so is not built, for want of {lacks}: the decode-step entry points need it")
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        module = ex.submit(_compile_module, nvcc) if lacks is None else None
        objs = list(ex.map(compile_one, srcs))
    libdir = _cuda_lib_dir(nvcc)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp,
           "-Xlinker", f"-rpath,{libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, LIB_PATH)
    if module is not None:
        _link_module(module.result(), libdir)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
