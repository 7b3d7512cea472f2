"""Builds liblightning_attn.so (and the Python binding of the softmax layers'
operators) in-tree with nvcc for sm_103a.

Every ``csrc/*.cu`` is compiled in parallel to an object file, then linked
into one shared library (CUDA runtime linked statically, so loading the
library needs no GPU driver; the driver is only touched by the first CUDA
call).  ``csrc/binding.cpp`` is compiled against the installed torch into
_lightning_binding.so, which is linked to the library beside it.  The library
needs neither torch nor Python's headers: without torch it is built alone, and
where the binding cannot be built it is in place before the error is raised.  A
content hash of each one's sources, flags and versions skips rebuilds that would
produce the same file.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "liblightning_attn.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
BINDING_PATH = os.path.join(BUILD_DIR, "_lightning_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _fingerprint(files, *words) -> str:
    h = hashlib.sha256()
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(words).encode())
    return h.hexdigest()


def _library_fingerprint(extra) -> str:
    files = _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h")))
    return _fingerprint(files, *ARCH, *NVCC_FLAGS, *extra)


def _binding_fingerprint() -> str:
    import torch
    files = [os.path.join(CSRC, "binding.cpp")] + sorted(glob.glob(os.path.join(INCLUDE, "*.h")))
    return _fingerprint(files, torch.__version__, sys.version)


def _current(path: str, stamp: str, fingerprint: str) -> bool:
    return os.path.exists(path) and os.path.exists(stamp) and open(stamp).read().strip() == fingerprint


def _binding_commands(obj: str, out: str) -> list[list[str]]:
    """Compile and link commands of the binding (host code only)."""
    import torch
    root = os.path.dirname(torch.__file__)
    cxx = shutil.which("c++") or shutil.which("g++") or "g++"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [INCLUDE, os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    lib = os.path.join(root, "lib")
    return [[cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
             *[f"-I{i}" for i in inc], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj],
            [cxx, "-shared", "-o", out, obj, f"-L{BUILD_DIR}", "-l:" + LIB_NAME,
             "-Wl,-rpath,$ORIGIN", f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10",
             "-lc10_cuda", "-ltorch_cuda", f"-Wl,-rpath,{lib}"]]


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False, extra_flags=(),
          jobs: int | None = None) -> str:
    """Compile and link the library (and, where torch is installed, the binding);
    returns the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(8, len(srcs) + 1)) as ex:
        binding = None
        if importlib.util.find_spec("torch") is not None:
            binding_stamp, binding_fp = BINDING_PATH + ".fingerprint.txt", _binding_fingerprint()
            if force or not _current(BINDING_PATH, binding_stamp, binding_fp):
                compile_, link = _binding_commands(os.path.join(BUILD_DIR, "binding.o"), BINDING_PATH + ".tmp")
                binding = ex.submit(_run, compile_, "binding")
        elif verbose:
            print("torch is not installed: the library without its Python binding")

        stamp, fp = os.path.join(BUILD_DIR, "fingerprint.txt"), _library_fingerprint(extra_flags)
        if force or not _current(LIB_PATH, stamp, fp):
            cc = nvcc()

            def compile_one(src):
                obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
                cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
                if verbose:
                    cmd.insert(1, "-Xptxas=-v")
                return obj, _run(cmd, f"nvcc for {src}")

            results = list(ex.map(compile_one, srcs))
            if verbose:
                for _, log in results:
                    if log.strip():
                        print(log)
            tmp = LIB_PATH + ".tmp"
            _run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in results], "link")
            os.replace(tmp, LIB_PATH)
            with open(stamp, "w") as f:
                f.write(fp)

        if binding is not None:
            binding.result()
            _run(link, "binding link")
            os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
            with open(binding_stamp, "w") as f:
                f.write(binding_fp)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
