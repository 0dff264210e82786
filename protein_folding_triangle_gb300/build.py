"""In-tree build of libtriattn (nvcc, sm_103a only) and of the Python binding's
native part.

Each translation unit is compiled in parallel with
``nvcc -gencode arch=compute_103a,code=sm_103a -lineinfo -O3`` and linked
into ``_build/libtriattn_<machine>.so`` next to this file.  No cmake, no
torch extension machinery: the library exports a plain C ABI
(include/triattn.h).  ``csrc/host.cpp``, which reads torch tensors for the
binding, is compiled with g++ against the installed torch's headers into
``_build/triattn_host_<torch version>.<Python's ABI tag>.so``; the library does
not depend on it, and where it cannot be compiled the binding does without.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import platform
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
SOURCES = ["api.cu", "fwd.cu", "bwd.cu", "noalloc.cu", "module.cu", "trimul.cu", "gemm.cu", "transition.cu",
           "transition_fwd.cu", "transition_rows.cu", "transition_bwd.cu", "transition_wgrad.cu", "gradnorm.cu",
           "qknorm.cu", "relpos.cu", "relpos_pairs.cu", "orthogonalize.cu", "orth_solo.cu"]
HEADERS = ["ptx.cuh", "kernels.cuh", "pairops.cuh", "transition.cuh", "relpos.cuh", "orthogonalize.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtriattn")
    return exe


def lib_path() -> str:
    return os.path.join(BUILD, f"libtriattn_{platform.machine()}.so")


def host_path() -> str:
    import torch
    # the tag (cpython-312-x86_64-linux-gnu, say) names the interpreter and the machine
    return os.path.join(BUILD, f"triattn_host_{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libtriattn and the binding's native part where a source is newer;
    the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        host = ex.submit(_build_host, force, verbose)
        out = _build_lib(force, verbose)
        try:
            host.result()
        except (RuntimeError, OSError) as e:
            warnings.warn(f"the binding's native part is not built: {e}", RuntimeWarning)
    return out


def _build_host(force: bool, verbose: bool) -> None:
    import torch
    out, src = host_path(), os.path.join(CSRC, "host.cpp")
    if not force and not _stale(out, [src, os.path.join(INCLUDE, "triattn.h"), __file__]):
        return
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    lib = os.path.join(root, "lib")
    tmp = out + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", src, "-o", tmp,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [x for d in include for x in ("-I", d)]
    cmd += ["-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(out):
            os.remove(out)  # of an older source
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        print(r.stdout, r.stderr)
    os.replace(tmp, out)


def _build_lib(force: bool, verbose: bool) -> str:
    out = lib_path()
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = srcs + [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "triattn.h"), __file__]
    if not force and not _stale(out, deps):
        return out
    exe = nvcc()
    objs = [os.path.join(BUILD, f"{os.path.splitext(s)[0]}_{platform.machine()}.o") for s in SOURCES]

    def compile_one(src_obj):
        src, obj = src_obj
        cmd = [exe] + NVCC_FLAGS + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        list(ex.map(compile_one, zip(srcs, objs)))
    tmp = out + f".tmp{os.getpid()}"
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(exe))), "lib64")
    cmd = [exe] + ARCH + ["-shared", "-o", tmp] + objs + ["-L", cuda_lib, "-Xlinker", "-rpath=" + cuda_lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(force=True, verbose=True))
