"""Builds ``libssd_gb300.so`` in-tree with nvcc for sm_103a.

Each translation unit under ``csrc/`` is compiled in parallel into
``_build/``; the shared library links the CUDA runtime statically so it
loads on a machine without a GPU driver (nothing touches the driver until
the first CUDA call).  Usage: ``python -m state_space_model_gb300.build``.

The compiled Python binding of the attention entry points
(``binding/attn_ext.cpp`` -> ``_attn_ext.so``) is built beside it with the host
compiler against the installed torch, again when that torch or the Python
changes.  Without torch or g++ the library is built alone.

``--debug-bounds`` builds ``libssd_gb300_debug.so`` instead (objects in
``_build_debug/``), compiled with ``-DSSD_DEBUG_BOUNDS``: the kernels check
every index, shared-memory offset and tensor-memory column range they compute
and report failures through ssd_device_status (see csrc/ssd_debug.cuh).
Python loads it when SSD_DEBUG_BOUNDS=1 is set.
"""
from __future__ import annotations

import concurrent.futures as cf
import errno
import glob
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libssd_gb300.so")
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libssd_gb300_debug.so")
BINDING_SRC = os.path.join(PKG, "binding", "attn_ext.cpp")
BINDING_TYPES = os.path.join(PKG, "binding", "scalar_types.h")
BINDING = os.path.join(PKG, "_attn_ext.so")
BINDING_STAMP = os.path.join(BUILD, "attn_ext.stamp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _run(cmd: list[str]) -> subprocess.CompletedProcess:
    """A compiler's run.  Starting one while other threads start theirs has failed with EFAULT
    once (aarch64), which is not the command's fault: it is tried again."""
    for last in (False, False, True):
        try:
            return subprocess.run(cmd, capture_output=True, text=True)
        except OSError as e:
            if e.errno != errno.EFAULT or last:
                raise


def _nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libssd_gb300")
    return exe


def _flags(verbose_ptxas: bool, debug_bounds: bool = False) -> list[str]:
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                "--expt-relaxed-constexpr"]
    if debug_bounds:
        f += ["-DSSD_DEBUG_BOUNDS"]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) +
                  glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps() -> list[str]:
    return (_sources() + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(CSRC, "*.cuh")) +
            [os.path.join(ROOT, "include", "ssd.h"), os.path.abspath(__file__)])


def up_to_date(debug_bounds: bool = False) -> bool:
    lib = LIB_DEBUG if debug_bounds else LIB
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _binding_stamp() -> str | None:
    """What the binding is built against, or None without a torch: the Python, and the place and
    date of torch's library (found without importing it)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    torch_lib = os.path.join(os.path.dirname(spec.origin), "lib", "libtorch_python.so")
    if not os.path.exists(torch_lib):
        return None
    return "\n".join([sys.version, str(sysconfig.get_config_var("SOABI")), platform.machine(),
                      torch_lib, str(os.stat(torch_lib).st_mtime_ns)])


def _binding_up_to_date() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_STAMP):
        return False
    with open(BINDING_STAMP) as f:
        if f.read() != _binding_stamp():
            return False
    t = os.path.getmtime(BINDING)
    return all(os.path.getmtime(p) <= t for p in (
        BINDING_SRC, BINDING_TYPES, os.path.join(ROOT, "include", "ssd.h"), os.path.abspath(__file__)))


def build_binding() -> str | None:
    """Compiles ``_attn_ext.so``.  It links the torch that is installed and calls the
    library through addresses that ``attn`` gives it.  None, with a line on stderr, where
    torch or the host compiler is missing: only ``attn`` needs it, and says so when called."""
    stamp = _binding_stamp()
    missing = "torch" if stamp is None else None if shutil.which("g++") else "g++"
    if missing:
        sys.stderr.write(f"_attn_ext.so not built: {missing} not found\n")
        return None
    import torch
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", BINDING_SRC, "-o", tmp,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(troot, "include"),
           "-I", os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-L", os.path.join(troot, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath," + os.path.join(troot, "lib")]
    r = _run(cmd)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on attn_ext.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(stamp)
    return BINDING


def build(force: bool = False, verbose_ptxas: bool | None = None,
          debug_bounds: bool = False) -> str:
    lib = LIB_DEBUG if debug_bounds else LIB
    out_dir = BUILD_DEBUG if debug_bounds else BUILD
    if force or not _binding_up_to_date():
        binding = cf.ThreadPoolExecutor(max_workers=1).submit(build_binding)
    else:
        binding = None
    if not force and up_to_date(debug_bounds):
        if binding:
            binding.result()
        return lib
    if verbose_ptxas is None:
        verbose_ptxas = os.environ.get("SSD_PTXAS_VERBOSE", "0") == "1"
    os.makedirs(out_dir, exist_ok=True)
    nvcc = _nvcc()
    flags = _flags(verbose_ptxas, debug_bounds)

    def compile_one(src: str) -> str:
        obj = os.path.join(out_dir, os.path.basename(src) + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = _run(cmd)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = _run(cmd)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if binding:
        binding.result()
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv,
                debug_bounds="--debug-bounds" in sys.argv))
