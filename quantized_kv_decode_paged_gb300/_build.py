"""Builds libdecode_attn.so in-tree with nvcc for sm_103a.

The translation units are compiled in parallel and linked into one shared
library next to this file (``_lib/libdecode_attn.so``).  Beside it the host
compiler makes ``_lib/decode_attn_call.torch<version><ABI tag>.so``, the Python
module that marshals the calls that take torch tensors in C++.  Only it needs
torch: the library is there without it, and the calls then go through Python.
A rebuild happens only when a source or header is newer than what it makes.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libdecode_attn.so")
CALL_SRC = os.path.join(CSRC, "call.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _newer(path, deps) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in deps)


def call_path():
    """Where the marshalling module for this interpreter and its torch is, or
    belongs; None without torch."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return os.path.join(LIB_DIR, f"decode_attn_call.torch{version}"
                                 + sysconfig.get_config_var("EXT_SUFFIX"))


def _call_up_to_date() -> bool:
    path = call_path()
    return path is None or _newer(path, [CALL_SRC, os.path.join(INCLUDE, "decode_attn.h"),
                                         os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _newer(LIB_PATH, _deps()) and _call_up_to_date()


def _build_call() -> None:
    """The marshalling module, against this interpreter's torch.  Where it
    cannot be made, the calls do without it: a warning says why."""
    try:
        _compile_call(call_path())
    except Exception as e:
        warnings.warn(f"the norm, append and shared-prefix calls go through Python, slower: {e}",
                      RuntimeWarning)


def _compile_call(path) -> None:
    import torch
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    top = os.path.dirname(os.path.abspath(torch.__file__))
    include = [sysconfig.get_paths()["include"], os.path.join(top, "include"),
               os.path.join(top, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), INCLUDE]
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for d in include for x in ("-I", d)], CALL_SRC, "-o", tmp,
           "-L" + os.path.join(top, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {CALL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every CUDA translation unit and link libdecode_attn.so; make the
    marshalling module if there is a torch."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    stale = call_path() is not None and (force or not _call_up_to_date())
    if not force and _newer(LIB_PATH, _deps()):
        _build_call()
        return LIB_PATH
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    srcs = _sources()
    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        call = ex.submit(_build_call) if stale else None
        results = list(ex.map(compile_one, srcs))
        if call:
            call.result()
    if verbose or ptxas_verbose:
        for _, log in results:
            if log:
                print(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
