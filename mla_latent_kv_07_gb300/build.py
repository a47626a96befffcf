"""Build libmla.so in-tree with nvcc for sm_103a (one -gencode, parallel TUs), and
_mla_native.so, the host path of some calls as a Python extension, with g++
against the installed torch.

    python -m mla_latent_kv_07_gb300.build [--verbose]

Objects and the library land in mla_latent_kv_07_gb300/_build/ (git-ignored).
The library links the CUDA runtime statically and resolves driver entry points
at run time, so it loads on a machine without a GPU driver.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmla.so")
NATIVE = os.path.join(BUILD, "_mla_native.so")
ROOT = os.path.dirname(HERE)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(obj: str, src: str, headers=None) -> bool:
    if not os.path.exists(obj):
        return True
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) if headers is None else headers
    deps = [src, *headers, os.path.join(ROOT, "include", "mla.h")]
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def torch_version() -> str:
    """torch.__version__, without the import."""
    with open(os.path.join(torch_dir(), "version.py")) as f:
        return re.search(r"^__version__ = '([^']+)'", f.read(), re.M).group(1)


def native_command(out: str):
    torch = torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(torch, "include"), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden", f'-DMLA_TORCH_VERSION="{torch_version()}"',
            *(f"-I{d}" for d in inc),
            os.path.join(CSRC, "native.cpp"), "-o", out, f"-L{torch}/lib", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10", "-lc10_cuda"]


def native_stamp() -> str:
    """What the extension is built against, beside its sources."""
    return f"torch {torch_version()} in {torch_dir()}, Python {sys.version}"


def native_stale() -> bool:
    try:
        with open(NATIVE + ".stamp") as f:
            if f.read() != native_stamp():
                return True
    except FileNotFoundError:
        return True
    return _stale(NATIVE, os.path.join(CSRC, "native.cpp"), [])


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, src):
            jobs.append([cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj])
    kernels = bool(jobs)
    native_tmp = NATIVE + f".{os.getpid()}.tmp"
    native = force or native_stale()
    if native:
        jobs.append(native_command(native_tmp))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"nvcc failed: {' '.join(cmd)}")
    if native:
        os.replace(native_tmp, NATIVE)
        with open(NATIVE + ".stamp", "w") as f:
            f.write(native_stamp())
    if kernels or not os.path.exists(LIB):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lrt", "-ldl", "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
