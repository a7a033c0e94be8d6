"""Build libmpadamw.so in-tree with nvcc for GB300 (sm_103a), and _binding, a
CPython extension, with gcc where that and Python's headers are there.

Each .cu translation unit is compiled in parallel, then linked into one
shared library (CUDA runtime linked statically, so the library needs only the
driver at run time). Arithmetic flags: no fast-math, IEEE division and square
root, no flush-to-zero, no FMA contraction (the kernels also spell every
rounding step with explicit intrinsics).
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmpadamw.so")
# The ordinary calls of include/mp_block.h from Python without ctypes. The name has
# the interpreter's tag, so that no other Python takes it for its own.
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
# compute-free stream probes, a separate library that only the benchmark loads
PROBE_LIB = os.path.join(PKG, "libmpprobe.so")

SOURCES = ["mp_api.cu", "mp_step.cu", "mp_norm.cu", "mp_sr.cu", "mp_outlier.cu", "mp_small.cu", "mp_copy.cu",
           "mp_layernorm.cu", "mp_logprob.cu", "mp_distill.cu", "mp_rmsnorm.cu", "mp_rope.cu", "mp_gated.cu"]
PROBE_SOURCES = ["mp_probe.cu"]
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo", *GENCODE,
    "-fmad=false", "-prec-div=true", "-prec-sqrt=true", "-ftz=false",
    "-Xcompiler", "-fPIC,-O2,-Wall",
    "-Xptxas", "-warn-spills",
    "-I", INCLUDE, "-I", CSRC,
]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmpadamw.so")
    return path


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def is_stale() -> bool:
    built = [LIB, PROBE_LIB] + ([BINDING] if _binding_needs() is None else [])
    if not all(os.path.exists(f) for f in built):
        return True
    return any(_outdated(f) for f in built)


def _outdated(built: str) -> bool:
    return any(os.path.getmtime(f) > os.path.getmtime(built) for f in _inputs())


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libmpadamw.so if missing or older than its sources."""
    if not (force or is_stale()):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + len(PROBE_SOURCES) + 1) as ex:
        binding = ex.submit(_binding)
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES + PROBE_SOURCES))
        binding.result()
    _link(objs[:len(SOURCES)], LIB)
    _link(objs[len(SOURCES):], PROBE_LIB)
    return LIB


def _cc():
    return shutil.which("gcc") or shutil.which("cc")


def _binding_needs():
    """What keeps _binding from being built; None if nothing does."""
    include = sysconfig.get_paths()["include"]
    if _cc() is None:
        return "a C compiler"
    return None if os.path.exists(os.path.join(include, "Python.h")) else f"{include}/Python.h"


def _binding():
    needs = _binding_needs()
    if needs is not None:  # the package works without it, through ctypes
        sys.stderr.write(f"_binding not built: {needs} not found; small calls of mp_block.h cost twice as much\n")
        if os.path.exists(BINDING) and _outdated(BINDING):
            _remove(BINDING)
        return
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [_cc(), "-O2", "-std=c11", "-Wall", "-Wextra", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"],
           "-I", INCLUDE, os.path.join(CSRC, "mp_binding.c"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on mp_binding.c:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    os.replace(tmp, BINDING)
    untagged = os.path.join(PKG, "_binding.so")  # an earlier build's, which any Python would take
    if untagged != BINDING:
        _remove(untagged)


def _remove(path):
    try:
        os.remove(path)
    except FileNotFoundError:  # another process was first
        pass


def _link(objs, out):
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc(), "-shared", *GENCODE, "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
