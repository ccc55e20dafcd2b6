"""Build libpa.so (the C-ABI library) from csrc/ with nvcc for sm_103a, and
_binding.so (csrc/binding.cpp, the compiled part of the torch binding).

Each translation unit is compiled in parallel into _build/ at the repository
root, then linked into paged_kv_cache_108_gb300/libpa.so (static CUDA runtime);
_binding.so links against it and the installed torch, and is left out where
there is none.  Each is rebuilt only when a source or header of its own is
newer, the binding also when torch or Python is another than it was built for.
Run ``python -m paged_kv_cache_108_gb300.build`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import fcntl
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpa.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BUILT_FOR = os.path.join(PKG, "_binding.built_for")  # the torch and Python that BINDING is for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libpa.so")
    return cand


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _built_for() -> str:
    """The installed torch's version and this Python's ABI, by which the
    layouts that the binding's code relies on go."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        version = re.search(r"__version__\s*=\s*['\"](.+?)['\"]", f.read())
    return f"torch {version.group(1) if version else '?'} {sysconfig.get_config_var('SOABI')}\n"


def binding_fits() -> bool:
    """Whether there is a binding, built for this torch and Python."""
    if _torch_dir() is None or not os.path.exists(BINDING) or not os.path.exists(BUILT_FOR):
        return False
    with open(BUILT_FOR) as f:
        return f.read() == _built_for()


def sources():
    """The library's translation units."""
    cpp = [s for s in glob.glob(os.path.join(CSRC, "*.cpp")) if s != BINDING_SRC]
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + cpp)


def _newer_than_all(out: str, deps) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in deps)


def library_up_to_date() -> bool:
    headers = [h for e in ("*.h", "*.cuh") for h in glob.glob(os.path.join(CSRC, e))]
    return _newer_than_all(LIB, [*sources(), *headers, os.path.join(INCLUDE, "pa.h"), __file__])


def binding_up_to_date() -> bool:
    return (_newer_than_all(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "pa.h"), __file__])
            and binding_fits())


def up_to_date() -> bool:
    return library_up_to_date() and (_torch_dir() is None or binding_up_to_date())


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if src.endswith(".cu"):
        cmd = [_nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
               "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose_ptxas:
            cmd[1:1] = ["-Xptxas", "-v"]
    else:
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-I", CSRC,
               "-c", src, "-o", obj]
        if src == BINDING_SRC:
            inc = os.path.join(_torch_dir(), "include")
            cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
            for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"),
                      sysconfig.get_path("include"), cuda):
                cmd[1:1] = ["-isystem", d]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    """Build what is stale of libpa.so and, where torch is installed, of
    _binding.so; returns libpa.so's path."""
    if not force and not verbose_ptxas and up_to_date():
        return LIB  # (nothing is written, not the lock either)
    with _alone(), cf.ThreadPoolExecutor(max_workers=1) as ex:  # the binding beside the library
        obj = None
        if _torch_dir() is not None and (force or not binding_up_to_date()):
            obj = ex.submit(_compile, BINDING_SRC, False)
        _library(force, verbose_ptxas, jobs)
        if obj is not None:
            _link_binding(obj.result())
    return LIB


def build_library(force: bool = False, verbose_ptxas: bool = False,
                  jobs: int | None = None) -> str:
    """Compile and link libpa.so (needs the CUDA toolkit alone); returns its path."""
    if not force and not verbose_ptxas and library_up_to_date():
        return LIB
    with _alone():
        return _library(force, verbose_ptxas, jobs)


def _library(force: bool, verbose_ptxas: bool, jobs: int | None) -> str:
    if not force and not verbose_ptxas and library_up_to_date():
        return LIB
    srcs = sources()
    jobs = jobs or min(len(srcs), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    _link([_nvcc(), *ARCH, "-shared"], [*objs, "-lpthread"], LIB)
    return LIB


def build_binding() -> str:
    """Build _binding.so if it is stale and link it against libpa.so, which it
    leaves as it is: a process that has libpa.so loaded goes on with that one."""
    if _torch_dir() is None:
        raise RuntimeError("torch not found: the binding is compiled against its headers")
    with _alone():
        if not binding_up_to_date():
            _link_binding(_compile(BINDING_SRC, False))
    return BINDING


@contextlib.contextmanager
def _alone():
    """One build at a time, over the threads and processes of this machine:
    they share object files and outputs."""
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, "lock"), "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)
        yield


def _link_binding(obj: str) -> None:
    torch_lib = os.path.join(_torch_dir(), "lib")
    _link(["g++", "-shared"],
          [obj, "-L", PKG, "-l:libpa.so", "-L", torch_lib, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"], BINDING)
    with open(BUILT_FOR, "w") as f:
        f.write(_built_for())


def _link(cmd, inputs, out: str) -> None:
    tmp = out + f".tmp{os.getpid()}"
    cmd = [*cmd, "-o", tmp, *inputs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
