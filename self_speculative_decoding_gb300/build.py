"""Builds libssd.so in-tree for sm_103a with nvcc (no cmake).

Each translation unit is compiled in parallel to an object file under
``_build/`` and linked into ``libssd.so`` next to this file.  The CUDA
runtime is linked statically.  ``csrc/binding.cpp``, the tree-decoding and several sequences' calls'
Python module, is compiled against the installed PyTorch's headers into
``_binding.so``; where that fails the library is built all the same, and those
calls raise the reason.
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
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libssd.so")
BINDING = os.path.join(HERE, "_binding.so")
STAMP = os.path.join(HERE, "_binding.txt")  # what it was built against; the reason if that failed
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newest_input(files) -> float:
    paths = [os.path.join(CSRC, f) for f in files]
    paths.append(os.path.join(os.path.dirname(HERE), "include", "ssd.h"))
    paths.append(os.path.join(os.path.dirname(HERE), "include", "ssd_ops.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths if os.path.exists(p))


def _current(path: str, files) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _newest_input(files)


def binding_key() -> str:
    """What _binding.so is built against (its C++ interfaces change with both)."""
    import torch
    return f"PyTorch {torch.__version__} in {os.path.dirname(torch.__file__)}, Python {sys.version.split()[0]}"


def _stamp():
    """(what _binding.so, or the attempt at it, was built against, why it failed)."""
    if not os.path.exists(STAMP):
        return "", ""
    with open(STAMP) as f:
        key, _, reason = f.read().partition("\n")
    return key, reason


def binding_failure() -> str:
    """Why there is no _binding.so for this PyTorch; empty if there is one."""
    key, reason = _stamp()
    if key and key != binding_key():
        return f"it was built against {key}, and this is {binding_key()}"
    return reason or ("" if os.path.exists(BINDING) else "it has not been built")


def _binding_current() -> bool:
    """Whether it, or an attempt that failed, is of this PyTorch and these sources."""
    key, reason = _stamp()
    return (key == binding_key() and (bool(reason) or os.path.exists(BINDING)) and
            _current(STAMP, ["binding.cpp"]))


def _build_binding() -> None:
    """_binding.so, or the reason why not, in STAMP."""
    key = binding_key()
    try:
        _compile_binding()
        reason = ""
    except Exception as e:
        reason = str(e)
        if os.path.exists(BINDING):
            os.remove(BINDING)  # of other sources, or another PyTorch
        warnings.warn(f"no tree-decoding calls and none of several sequences, the rest of the library is built: {reason}")
    with open(STAMP, "w") as f:
        f.write(key + "\n" + reason)


def _compile_binding() -> None:
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    libs = os.path.join(root, "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for i in inc for x in ("-isystem", i)], os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    with ThreadPoolExecutor(max_workers=1) as ex:
        os.makedirs(BUILD, exist_ok=True)
        binding = None
        if force or not _binding_current():
            binding = ex.submit(_build_binding)
        if force or not _current(LIB, [f for f in os.listdir(CSRC) if f != "binding.cpp"]):
            _build_library(verbose, extra_flags)
        if binding:
            binding.result()
    return LIB


def _build_library(verbose: bool, extra_flags) -> None:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build_variant(tag: str, flags) -> str:
    """Builds a copy of the library with extra compile flags (tuning sweeps)
    under _build/<tag>/; returns the path of its .so."""
    out_dir = os.path.join(BUILD, tag)
    os.makedirs(out_dir, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(out_dir, src[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, sources()))
    lib = os.path.join(out_dir, "libssd.so")
    r = subprocess.run([cc, *ARCH, "-shared", "-o", lib, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
