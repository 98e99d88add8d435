"""Builds libfa.so in-tree with nvcc for sm_103a.

Each CUDA translation unit compiles in its own nvcc process (in parallel),
then the objects link into one shared library with the CUDA runtime linked
statically, so the library only needs the driver at run time.  The PyTorch
binding of the paged-cache calls (csrc/fa_torch.cpp) is a second, small library
beside it, compiled by the host compiler against the installed PyTorch.  Each
is rebuilt for its own sources alone, and the library does not depend on the
binding: where that cannot be compiled (a PyTorch without CUDA or without its
headers) the rest works, and the paged-cache calls say that it is missing.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libfa.so")
HEADER = os.path.join(PKG, "..", "include", "fa.h")
SOURCES = ["fa_api.cu", "fa_simt.cu", "fa_bwd_sm103.cu", "fa_bwd_sm103_count.cu", "fa_bwd_d256_sm103.cu",
           "fa_fwd_sm103.cu", "fa_noalloc.cu", "fa_host.cu", "fa_tma.cu", "fa_decode.cu", "fa_decode_fp32.cu", "fa_cache.cu", "fa_pages.cu",
           "fa_cache_e4m3.cu", "fa_decode_e4m3.cu", "fa_decode_e4m3_sm103.cu"]
TORCH_SOURCE = "fa_torch.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3",
    "-lineinfo",
    "-std=c++17",
    "-Xcompiler",
    "-fPIC",
    "--expt-relaxed-constexpr",
    "-Xptxas",
    "-warn-spills",
]


def torch_binding_path() -> str:
    """The binding for this Python and PyTorch: its name says which, so that
    another version does not load it."""
    import torch

    return os.path.join(OUT_DIR, f"_fa_torch_{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_torch_binding(force: bool = False) -> str:
    """Compile (if stale) and return the path of the binding.  One that cannot
    be compiled again is not left behind."""
    import torch

    root = os.path.dirname(torch.__file__)
    out = torch_binding_path()
    if not force and not _stale(out, [HEADER, os.path.join(CSRC, TORCH_SOURCE)]):
        return out
    os.makedirs(OUT_DIR, exist_ok=True)
    if os.path.exists(out):
        os.remove(out)
    tmp = out + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-fPIC", "-O2", "-std=c++17", os.path.join(CSRC, TORCH_SOURCE),
           "-o", tmp, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f"-I{os.path.join(root, 'include')}", f"-I{os.path.join(root, 'include', 'torch', 'csrc', 'api', 'include')}",
            f"-I{sysconfig.get_paths()['include']}", f"-I{cuda_include()}"]
    lib = os.path.join(root, "lib")
    cmd += [f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {TORCH_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def cuda_include() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(lib: str, deps: list[str]) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps)


def _deps() -> list[str]:
    """What libfa.so is made from."""
    return [HEADER] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile what is stale and return the path of libfa.so.  A binding that
    cannot be compiled is a warning."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(build_torch_binding, force)
        if force or _stale(LIB, _deps()):
            _build_library(verbose, extra_flags)
        try:
            binding.result()
        except Exception as e:
            warnings.warn(f"libfa.so is built, the PyTorch binding of the paged-cache calls is not: {e}")
    return LIB


def _build_library(verbose: bool, extra_flags: list[str] | None) -> None:
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = nvcc_path()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, "-c", os.path.join(CSRC, src), "-o", obj] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            if log.strip():
                sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", "-o", tmp] + [o for o, _ in results] + ARCH + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
