"""Builds ``libgrpo.so`` (the C-ABI CUDA library) in-tree for sm_103a, and
``_ops.so`` (the marshalling of PyTorch tensors for the operators around the
loss, host code linked to it).

Each ``csrc/*.cu`` file is compiled to an object in ``_build/`` in parallel,
then linked into ``vocab_wide_logprob_gb300/libgrpo.so`` against the shared
CUDA runtime (so the process keeps a single runtime instance with PyTorch).
Run as ``python -m vocab_wide_logprob_gb300.build`` or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBRARY = os.path.join(PKG, "libgrpo.so")
BINDING = os.path.join(PKG, "_ops.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def cuda_home() -> str:
    env = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if env:
        return env
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def nvcc() -> str:
    return os.path.join(cuda_home(), "bin", "nvcc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def compile_flags(verbose_ptxas: bool = False):
    flags = ["-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
             "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]
    return flags


def _compile(src: str, verbose_ptxas: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if verbose_ptxas or _stale(obj, [src, *_headers()]):
        cmd = [nvcc(), *compile_flags(verbose_ptxas), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr
    return obj, ""


def _torch_dir() -> str:
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def binding_target() -> str:
    """What ``_ops.so`` has to be compiled against: this PyTorch and this Python."""
    version = runpy.run_path(os.path.join(_torch_dir(), "version.py"))["__version__"]
    return f"torch {version}, {sys.implementation.cache_tag}"


def _binding_stale(obj: str) -> bool:
    """Whether the object is older than its sources or was compiled against
    another PyTorch or Python (noted in a file beside it)."""
    if _stale(obj, [BINDING_SOURCE, *glob.glob(os.path.join(INCLUDE, "*.h"))]):
        return True
    try:
        with open(obj + ".target") as f:
            return f.read() != binding_target()
    except OSError:
        return True


def _compile_binding() -> str:
    obj = os.path.join(BUILD, "binding.o")
    if _binding_stale(obj):
        target, inc = binding_target(), os.path.join(_torch_dir(), "include")
        dirs = [INCLUDE, inc, os.path.join(inc, "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda_home(), "include")]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
               f'-DGRPO_BUILT_FOR="{target}"',
               *[x for d in dirs for x in ("-isystem" if d != INCLUDE else "-I", d)],
               "-c", BINDING_SOURCE, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {BINDING_SOURCE}:\n{r.stderr}")
        with open(obj + ".target", "w") as f:
            f.write(target)
    return obj


def _link_binding(obj: str, force: bool) -> None:
    if not force and not _stale(BINDING, [obj, LIBRARY]):
        return
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libgrpo.so",
           "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-L", os.path.join(cuda_home(), "lib64"), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {BINDING} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = True) -> str:
    """Compiles the library if any source is newer than it; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(9, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    objs = [o for o, _ in results]
    if verbose_ptxas and not quiet:
        for _, log in results:
            sys.stderr.write(log)
    if force or _stale(LIBRARY, objs):
        tmp = LIBRARY + f".tmp{os.getpid()}"
        lib64 = os.path.join(cuda_home(), "lib64")
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
               "-Xlinker", f"-rpath,{lib64}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIBRARY)
    # (after the library: the loss calls work without the binding)
    _link_binding(binding.result(), force)
    return LIBRARY


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(force="--force" in sys.argv, verbose_ptxas=v, quiet=not v))
