"""Builds the CUDA library ``libmoe_mxfp4.so`` in-tree with nvcc for sm_103a, and, where
torch with CUDA is installed, the torch binding of the dense operators ``_dense_ext.so``
over it.  The library is in place before the binding is, and without it.

Each translation unit is compiled in parallel into ``_build/`` next to this file
and linked into ``libmoe_mxfp4.so`` beside it; nothing is installed elsewhere.
A rebuild happens only when a source or header is newer than the library.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libmoe_mxfp4.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
EXT_PATH = os.path.join(HERE, "_dense_ext.so")
EXT_SOURCE = "dense_binding.cpp"

SOURCES = ["moe_route.cu", "moe_gemm.cu", "moe_aux.cu", "moe_api.cu", "moe_noalloc.cu", "moe_peak.cu",
           "moe_blocknorm.cu", "moe_thin.cu", "moe_dense_gemm.cu", "moe_dense_api.cu"]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_mxfp4.so")


def _inputs():
    return (glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _targets():
    return [LIB_PATH] + ([EXT_PATH] if _torch_has_cuda() else [])


def is_stale() -> bool:
    if not all(os.path.exists(p) for p in _targets()):
        return True
    t = min(os.path.getmtime(p) for p in _targets())
    if any(os.path.getmtime(p) > t for p in _inputs()):
        return True
    return _torch_has_cuda() and _read(_stamp_path()) != _binding_stamp()


def _read(path: str) -> str | None:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _stamp_path() -> str:
    return os.path.join(BUILD_DIR, "binding.txt")


def _binding_stamp() -> str:
    """The Python and the torch that a binding is good for: both have an ABI of their own."""
    torch_dir = _torch_dir()
    return "\n".join((str(sysconfig.get_config_var("SOABI")), torch_dir, _read(os.path.join(torch_dir, "version.py")) or ""))


def _torch_dir() -> str | None:
    """torch's install folder (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _torch_has_cuda() -> bool:
    torch_dir = _torch_dir()
    return torch_dir is not None and os.path.exists(os.path.join(torch_dir, "lib", "libtorch_cuda.so"))


def _run(what: str, cmd) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")
    return res.stderr


def _compile_ext() -> str:
    """The torch binding's object file (host code only)."""
    torch_dir = _torch_dir()
    obj = os.path.join(BUILD_DIR, os.path.splitext(EXT_SOURCE)[0] + ".o")
    includes = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include/torch/csrc/api/include"),
                os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"), sysconfig.get_paths()["include"]]
    _run(f"g++ on {EXT_SOURCE}", ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-DUSE_CUDA",
                                  *[f"-isystem{d}" for d in includes], "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj])
    return obj


def _link_ext(obj: str) -> None:
    lib_dir = os.path.join(_torch_dir(), "lib")
    tmp = EXT_PATH + ".tmp"
    _run("link of the torch binding", ["g++", "-shared", obj, LIB_PATH, f"-L{lib_dir}", "-ltorch_python", "-ltorch_cuda",
                                       "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib_dir}",
                                       "-o", tmp])
    os.replace(tmp, EXT_PATH)


def _compile(nvcc: str, src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose:
        print(res.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link the shared library; returns its path."""
    if not force and not is_stale():
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(_compile_ext) if _torch_has_cuda() else None
        objs = list(ex.map(lambda s: _compile(nvcc, s, verbose), SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-Xcompiler", "-fPIC", "-Xlinker", f"-soname={LIB_NAME}", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    if ext:
        _link_ext(ext.result())
        with open(_stamp_path(), "w") as f:
            f.write(_binding_stamp())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
