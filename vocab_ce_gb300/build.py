"""Build libtpce.so in-tree with nvcc for sm_103a.

Translation units are compiled in parallel, then linked into
``vocab_ce_gb300/lib/libtpce.so``; beside it the host binding of the
training-step calls (g++ and torch's headers), under a name of its own for each
torch and Python. Run ``python -m vocab_ce_gb300.build``.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build", "tpce")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libtpce.so")

SOURCES = ["runtime.cu", "mlp.cu", "linear.cu", "ce.cu", "ce_static.cu", "step/norm.cu", "step/experts.cu",
           "step/adamw.cu"]
BINDING_SOURCE = os.path.join(CSRC, "step", "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def _deps_mtime() -> float:
    files = [os.path.join(d, f) for top in (CSRC, INCLUDE) for d, _, names in os.walk(top) for f in names]
    return max(os.path.getmtime(f) for f in files)


def binding_path() -> str:
    """The step binding for the torch and the Python that run: it is compiled against torch's C++ classes, whose
    layout another version may change."""
    import torch

    return os.path.join(LIB_DIR, f"_step_binding-torch{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _build_binding(force: bool = False) -> None:
    import torch

    path = binding_path()
    if not force and _is_current(path):
        return
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    lib = os.path.join(home, "lib")
    tmp = path + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE]
    for d in (os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include"), sysconfig.get_paths()["include"]):
        cmd += ["-isystem", d]
    cmd += [BINDING_SOURCE, "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
            "-lc10_cuda", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on step/binding.cpp:\n" + r.stderr)
    os.replace(tmp, path)


def _is_current(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()


def build(force: bool = False, verbose: bool = False, extra_flags=None, out_path: str = None,
          build_dir: str = None) -> str:
    """Compile and link libtpce.so (default: in-tree, with the step binding beside it). extra_flags are added to
    every nvcc compile (e.g. -DTPCE_EPI_WARPS=8 tuning knobs)."""
    os.makedirs(os.path.dirname(out_path or LIB_PATH), exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = None if out_path else ex.submit(_build_binding, force)
        lib_path = _build_library(force, verbose, extra_flags, out_path or LIB_PATH, build_dir or BUILD_DIR)
    if binding is not None:
        binding.result()  # raises only here: the library needs neither g++ nor torch's headers
    return lib_path


def _build_library(force: bool, verbose: bool, extra_flags, lib_path: str, bdir: str) -> str:
    if not force and _is_current(lib_path):
        return lib_path
    os.makedirs(bdir, exist_ok=True)
    exe = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(bdir, src.replace("/", "_").replace(".cu", ".o"))
        cmd = [exe] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    for src, _, r in results:
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    tmp = lib_path + ".tmp"
    cmd = [exe] + ARCH + ["-shared", "-o", tmp] + [obj for _, obj, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
