"""Build libpa.so in-tree with nvcc for sm_103a, and the compiled host calls beside it.

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into
``lib/libpa.so`` with the CUDA runtime linked statically.  A rebuild happens
only when a source or header is newer than the library.  ptxas resource
reports (registers, spills, shared memory) are kept next to the objects.
``csrc/fast_calls.cpp`` becomes ``lib/_pa_fast.so``, a Python module against the
installed torch's headers that calls into libpa.so.  It only saves host time:
where it cannot be compiled (no g++, no Python or torch headers) the build says
so and libpa.so stands alone, with the checks in Python.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import platform
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIBDIR = os.path.join(HERE, "lib")
OBJDIR = os.path.join(LIBDIR, "obj")
LIBPATH = os.path.join(LIBDIR, "libpa.so")
FASTSRC = os.path.join(CSRC, "fast_calls.cpp")
FASTPATH = os.path.join(LIBDIR, "_pa_fast.so")

ARCH = "-gencode=arch=compute_103a,code=sm_103a"
NVCC_FLAGS = ["-std=c++17", "-O3", ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              f"-I{INCLUDE}"]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libpa.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [
        FASTSRC, os.path.abspath(__file__)]


STAMP = os.path.join(LIBDIR, "host-arch.txt")


NO_FAST = ", host calls not compiled"          # at the end of the stamp


def _stamp() -> str:
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "none"
    return f"{platform.machine()} torch {torch}"


def up_to_date() -> bool:
    """The libraries exist (_pa_fast.so unless it could not be compiled), were
    built on this machine's architecture with the installed torch, and are
    newer than every source."""
    if not all(os.path.exists(p) for p in (LIBPATH, STAMP)):
        return False
    with open(STAMP) as f:
        stamp = f.read().strip()
    built = [LIBPATH] if stamp == _stamp() + NO_FAST else [LIBPATH, FASTPATH]
    if stamp.removesuffix(NO_FAST) != _stamp() or not all(os.path.exists(p) for p in built):
        return False
    t = min(os.path.getmtime(p) for p in built)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(obj + ".ptxas.txt", "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
    return obj


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    return spec.submodule_search_locations[0]


def _compile_fast() -> str:
    torch_dir = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    obj = os.path.join(OBJDIR, "fast_calls.o")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", f"-I{torch_dir}/include",
           f"-I{torch_dir}/include/torch/csrc/api/include", f"-I{sysconfig.get_paths()['include']}", f"-I{cuda}/include",
           "-c", FASTSRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {FASTSRC}:\n{r.stderr[-4000:]}")
    return obj


def _link_fast(obj: str) -> None:
    torch_dir = _torch_dir()
    tmp = FASTPATH + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{LIBDIR}", "-lpa", f"-L{torch_dir}/lib", "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, FASTPATH)


def build(force: bool = False, jobs: int | None = None) -> str:
    """Compile and link libpa.so and, where that is possible, _pa_fast.so;
    returns the former's path."""
    if not force and up_to_date():
        return LIBPATH
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = _sources()
    jobs = jobs or min(len(srcs), max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(max_workers=jobs + 1) as ex:
        fast = ex.submit(_compile_fast)
        objs = list(ex.map(_compile, srcs))
    tmp = LIBPATH + ".tmp"
    cmd = [nvcc(), ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIBPATH)
    without = ""
    try:
        _link_fast(fast.result())
    except (RuntimeError, OSError) as e:
        without = NO_FAST
        if os.path.exists(FASTPATH):
            os.remove(FASTPATH)                  # of other sources
        warnings.warn(f"{os.path.basename(FASTPATH)} was not built: the tree-speculation calls do their checks in Python, "
                      f"about 10 microseconds a call; build(force=True) tries again.  {e}", RuntimeWarning, stacklevel=2)
    with open(STAMP, "w") as f:
        f.write(_stamp() + without + "\n")
    return LIBPATH


if __name__ == "__main__":
    print(build(force=True))
