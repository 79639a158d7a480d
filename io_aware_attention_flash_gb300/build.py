"""Build libfa_gb300.so in-tree with nvcc for sm_103a.

Each translation unit is compiled in its own nvcc process (in parallel), then
linked into ``io_aware_attention_flash_gb300/lib/libfa_gb300.so`` with the
CUDA runtime linked statically.  Beside it, the host compiler builds
``lib/_fa_torch.so``, the calls from PyTorch that do without the interpreter
(linked against libfa_gb300.so next to it); ``lib/_fa_torch.txt`` names the
PyTorch and Python it is for.  A rebuild happens only when a source or header is
newer than the libraries, or PyTorch or Python is another one.

    python -m io_aware_attention_flash_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libfa_gb300.so")
TORCH_LIB_PATH = os.path.join(LIB_DIR, "_fa_torch.so")
TORCH_STAMP_PATH = os.path.join(LIB_DIR, "_fa_torch.txt")
TORCH_SOURCE = "fa_torch.cpp"

SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_decode.cu", "fa_cache8.cu", "fa_microbench.cu"]
HEADERS = ["ptx.cuh", "fa_kernels.cuh", "cache8_phases.h", "cache8_tiles.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
          "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libfa_gb300")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS + [TORCH_SOURCE]]
    files.append(os.path.join(INCLUDE, "fa.h"))
    files.append(os.path.abspath(__file__))
    return files


def torch_stamp() -> str:
    """What _fa_torch.so depends on beside the sources: the layout of PyTorch's
    C++ objects, the compiler's ABI and the Python."""
    import sysconfig

    import torch

    return (f"torch {torch.__version__} {torch.version.git_version} cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"python {sysconfig.get_config_var('SOABI')}")


def torch_built_for() -> str:
    """The stamp of the _fa_torch.so that is there; empty if it has none."""
    try:
        with open(TORCH_STAMP_PATH) as f:
            return f.read()
    except FileNotFoundError:
        return ""


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(TORCH_LIB_PATH) or torch_built_for() != torch_stamp():
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(TORCH_LIB_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _compile(nvcc: str, src: str, verbose: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, *ARCH, *CFLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    log = r.stdout + r.stderr
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{log}")
    if verbose:
        print(log, file=sys.stderr)
    return obj, log


def _compile_torch(verbose: bool) -> str:
    """The PyTorch calls' object file, with the compiler ABI PyTorch has."""
    import sysconfig

    import torch

    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    obj = os.path.join(BUILD_DIR, "fa_torch.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE]
    for inc in (root, os.path.join(root, "torch", "csrc", "api", "include"), cuda, sysconfig.get_paths()["include"]):
        cmd += ["-isystem", inc]
    cmd += ["-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {TORCH_SOURCE}:\n{' '.join(cmd)}\n{r.stdout}{r.stderr}")
    return obj


def _link_torch(obj: str) -> None:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_LIB_PATH + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", LIB_DIR, "-l:libfa_gb300.so", "-L", libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}{r.stderr}")
    if os.path.exists(TORCH_STAMP_PATH):  # at no time beside a library that it is not of
        os.remove(TORCH_STAMP_PATH)
    os.replace(tmp, TORCH_LIB_PATH)
    with open(TORCH_STAMP_PATH + ".tmp", "w") as f:
        f.write(torch_stamp())
    os.replace(TORCH_STAMP_PATH + ".tmp", TORCH_STAMP_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library if needed; returns its path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_obj = ex.submit(_compile_torch, verbose)
        results = list(ex.map(lambda s: _compile(nvcc, s, verbose), SOURCES))
        torch_obj = torch_obj.result()
    objs = [o for o, _ in results]
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        for _, log in results:
            f.write(log)
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_torch(torch_obj)
    return LIB_PATH


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
