"""Build libpa.so in-tree with nvcc for sm_100a (B200), and _pa_torch.so with the C++ compiler.

Usage: python -m paged_kv_cache_442_b200.build [--force] [--ptxas-verbose]
Each .cu (device and host code) and .cpp (host-only code) under csrc/ is compiled to
an object in _build/ by nvcc (in parallel), then the
objects are linked into paged_kv_cache_442_b200/libpa.so with the CUDA runtime
linked statically. csrc/torch/binding.cpp (torch tensors to C pointers, for the Python
binding) becomes _pa_torch.so, linked against libpa.so and torch; it holds the names of the torch
and the Python it was built for. Without torch only libpa.so is built. Rebuilds only when a
source or header is newer than the libraries, or torch or Python are others.
"""
from __future__ import annotations

import argparse
import glob
import importlib.metadata
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpa.so")
BINDING_SRC = os.path.join(CSRC, "torch", "binding.cpp")
BINDING = os.path.join(PKG, "_pa_torch.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) +
                               glob.glob(os.path.join(CSRC, "*.cuh")) +
                               glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def _newer_than(target, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _binding_deps():
    return [BINDING_SRC, os.path.abspath(__file__)] + sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def binding_target() -> str | None:
    """The torch and the Python that _pa_torch.so has to be built for; None without torch."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return f"torch {version}, Python {sys.version_info.major}.{sys.version_info.minor}"


def built_for() -> str | None:
    """What the _pa_torch.so that is there was built for (read, not loaded: a module of another
    torch may not load); None if it does not say."""
    if not os.path.exists(BINDING):
        return None
    with open(BINDING, "rb") as f:
        name = re.search(rb"pa_built_for{([^}]*)}", f.read())
    return name.group(1).decode() if name else None


def _binding_up_to_date() -> bool:
    target = binding_target()
    return target is None or (built_for() == target and _newer_than(BINDING, _binding_deps()))


def up_to_date() -> bool:
    return _newer_than(LIB, _deps()) and _binding_up_to_date()


def _compile_binding() -> str:
    """Object file of the torch binding (host C++; torch's headers, no CUDA code)."""
    import torch
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler: g++ is required to build _pa_torch.so")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    obj = os.path.join(BUILD_DIR, "binding.cpp.o")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DPA_BUILT_FOR="{binding_target()}"',
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-I", INCLUDE,
           "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the torch binding does not compile:\n" + r.stdout + r.stderr)
    return obj


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    tmp = BINDING + ".tmp"
    cmd = [cxx, "-shared", "-o", tmp, obj, "-L", PKG, "-l:libpa.so", "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of _pa_torch.so failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, BINDING)


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int = 8) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *common, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=jobs) as ex:
        wanted = binding_target() is not None and (force or not _binding_up_to_date())
        binding = ex.submit(_compile_binding) if wanted else None
        results = [] if not force and _newer_than(LIB, _deps()) else \
            list(ex.map(compile_one, _sources()))
    failed = [(s, r) for s, _, r in results if r.returncode != 0]
    for s, _, r in results:
        if r.stdout or r.stderr:
            sys.stderr.write(f"--- {os.path.basename(s)}\n{r.stdout}{r.stderr}")
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(os.path.basename(s) for s, _ in failed))
    if results:
        _link_library(nvcc, [o for _, o, _ in results])
    if binding is not None:
        _link_binding(binding.result())
    return LIB


def _link_library(nvcc, objects) -> None:
    tmp = LIB + ".tmp"
    link = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp,
            "-Xlinker", "-soname=libpa.so", *objects, "-cudart", "static"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, ptxas_verbose=a.ptxas_verbose))


if __name__ == "__main__":
    main()
