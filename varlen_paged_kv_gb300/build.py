"""Build libpagedattn.so in-tree for sm_103a (GB300).

Each translation unit under csrc/ is compiled by nvcc in parallel, then linked into a
shared library next to this file. Rebuilds only when a source or header is newer than
the library. The CUDA runtime is linked statically, so the library depends on the
driver only. Beside it, g++ builds csrc/binding.cpp against the installed torch: the
Python calls of the operators around the attention call. Only their host time depends on
it (step.py makes the same calls), so where it cannot be built the library still is.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libpagedattn.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))


# the coverage-counting debug library (pa_debug_coverage), built on demand by its test
COV_LIB = os.path.join(HERE, "libpagedattn_cov.so")


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def binding_path(folder: str = HERE) -> str:
    """The compiled Python calls for this interpreter and torch. They build torch's objects by its
    headers, so the name holds what they were compiled against: another torch or Python looks
    for another file."""
    import sysconfig

    import torch

    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(folder, f"_step_binding.torch-{torch.__version__}-abi{abi}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_binding(force: bool = False) -> str:
    """csrc/binding.cpp against the torch that imports it."""
    out = binding_path()
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src, os.path.join(INCLUDE, "pagedattn.h")]
    if not force and os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps):
        return out
    import sysconfig

    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    tmp = out + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(base, "include"),
           "-I" + os.path.join(base, "include", "torch", "csrc", "api", "include"), "-I" + cuda, src, "-o", tmp,
           "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stderr}")
    os.replace(tmp, out)
    return out


def _try_binding(force: bool = False) -> None:
    """build_binding, or a warning; a binding that is out of date does not stay."""
    out = None
    try:
        out = binding_path()
        build_binding(force)
    except Exception as e:  # noqa: BLE001 (no torch, no compiler, no headers, ...)
        if out is not None and os.path.exists(out):
            os.unlink(out)
        warnings.warn(f"the compiled calls were not built, each call takes some microseconds longer: {e}", RuntimeWarning)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False, coverage: bool = False) -> str:
    lib = COV_LIB if coverage else LIB
    if not force and not ptxas_info and up_to_date(lib):
        _try_binding()
        return lib
    build_dir = os.path.join(BUILD, "cov") if coverage else BUILD
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    if coverage:
        extra = extra + ["-DPA_COVERAGE=1"]

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_try_binding, force)
        results = list(ex.map(compile_one, sources()))
        binding.result()
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                print(log)
    objs = [o for o, _ in results]
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    build(force=True, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
