"""Build the CUDA library (csrc/*.cu -> _build/libmoe_gb300.so) for sm_103a.

Every translation unit is compiled in parallel with one -gencode
(compute_103a / sm_103a) and linked into a shared library with the static
CUDA runtime. csrc/tensors.cpp, the Python side's fast way from torch tensors
to the library's calls, becomes an extension module beside it where torch is
installed (the library needs none, and the package does without); nothing is
installed outside this folder.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import re
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
# MOE_BUILD_DIR / MOE_NVCC_DEFINES build a variant elsewhere (for example
# with -DMOE_TRACE); MOE_LIBRARY makes the binding load a given build.
BUILD = os.environ.get("MOE_BUILD_DIR", os.path.join(HERE, "_build"))
LIBRARY = os.environ.get("MOE_LIBRARY", os.path.join(BUILD, "libmoe_gb300.so"))
DEFINES = os.environ.get("MOE_NVCC_DEFINES", "").split()
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-ffp-contract=off", "-I", os.path.join(ROOT, "include")]


def _torch_folder():
    """The folder of the installed torch (found, not imported), None without one or with one for CPUs only."""
    spec = importlib.util.find_spec("torch")
    folder = os.path.dirname(spec.origin) if spec is not None and spec.origin else None
    return folder if folder and all(os.path.exists(os.path.join(folder, f)) for f in ("version.py", "lib/libc10_cuda.so")) else None


def _tensors_path():
    """The extension module's file, named by the torch and the Python that it is bound to: another's is not taken for it."""
    torch = _torch_folder()
    if torch is None:
        return None
    with open(os.path.join(torch, "version.py"), encoding="utf-8") as f:
        version = re.search(r"__version__\s*=\s*['\"]([^'\"]+)", f.read())
    name = f"_tensors.{sysconfig.get_config_var('SOABI')}.torch-{version.group(1) if version else 'unknown'}"
    return os.path.join(os.path.dirname(LIBRARY), re.sub(r"[^\w.-]", "-", name) + ".so")


TENSORS = _tensors_path()


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _dependencies():
    deps = _sources() + [os.path.join(CSRC, "tensors.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    return deps + [os.path.join(ROOT, "include", "moe.h")]


def up_to_date() -> bool:
    made = [LIBRARY] if TENSORS is None else [LIBRARY, TENSORS]
    if not all(os.path.exists(m) for m in made):
        return False
    built = min(os.path.getmtime(m) for m in made)
    return all(os.path.getmtime(d) <= built for d in _dependencies())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIBRARY
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, *DEFINES, *extra, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stderr}")
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    def compile_tensors():
        if TENSORS is None:
            return
        torch = _torch_folder()
        tmp = TENSORS + f".{os.getpid()}.tmp"
        cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
        include = [os.path.join(ROOT, "include"), sysconfig.get_path("include"), os.path.join(torch, "include"),
                   os.path.join(torch, "include", "torch", "csrc", "api", "include"), cuda]
        lib = os.path.join(torch, "lib")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *[f"-I{i}" for i in include], os.path.join(CSRC, "tensors.cpp"),
               "-o", tmp, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{lib}"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"g++ failed for tensors.cpp:\n{res.stderr}")
        os.replace(tmp, TENSORS)

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(_sources()) + 1) as pool:
        tensors = pool.submit(compile_tensors)
        objects = list(pool.map(compile_one, _sources()))
        tensors.result()
    tmp = LIBRARY + f".{os.getpid()}.tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objects]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose="-v" in sys.argv))
