"""Build liblp.so (the C-ABI library) in-tree with nvcc for sm_103a.

Every translation unit is compiled for ``-gencode arch=compute_103a,code=sm_103a``
only, with ``--fmad=false`` (no multiply-add contraction: the arithmetic that
fixes the result bits is written with explicit rounding intrinsics), in
parallel, then linked into ``_build/liblp.so`` next to this file.  The build is
skipped only when ``_build/liblp.so.sha256`` records the SHA-256 of exactly the
current sources, headers, this file and the compiler flags: a library that was
copied in from elsewhere, or built from other sources, is rebuilt.  build()
prints whether it compiled.
"""

from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "liblp.so")
SOURCES = ["lp_api.cu", "lp_logits.cu", "lp_linear.cu", "lp_backward.cu", "lp_train_api.cu",
           "lp_norm.cu", "lp_norm_backward.cu", "lp_policy.cu", "lp_adamw.cu", "lp_tune_api.cu",
           "lp_layer_norm.cu", "lp_layer_norm_backward.cu", "lp_preference.cu",
           "lp_muon.cu"]
HEADERS = [os.path.join(ROOT, "include", f) for f in ("lp.h", "lp_train.h", "lp_tune.h")] + [
    os.path.join(CSRC, f) for f in ("lp_device.cuh", "lp_internal.h", "lp_tcgen05.cuh",
                                    "lp_check.cuh", "lp_train_internal.h", "lp_norm.cuh", "lp_layer_norm.cuh",
                                    "lp_args.h", "lp_tune_internal.h")
]
# the Python calls of train.py and tune.py: host code against torch's headers, no part of liblp
CALLS_MODULES = ("train", "tune")
# the checked build (-DLP_CHECKED: index and coordinate tests in every kernel)
BUILD_CHECKED = os.path.join(PKG, "_build_checked")
LIB_CHECKED = os.path.join(BUILD_CHECKED, "liblp.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17", "--fmad=false",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", os.path.join(ROOT, "include"),
]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path is None:
        cand = "/usr/local/cuda/bin/nvcc"
        if os.path.exists(cand):
            return cand
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblp")
    return path


def _paths(checked: bool):
    return (BUILD_CHECKED, LIB_CHECKED) if checked else (BUILD, LIB)


def source_hash(checked: bool = False) -> str:
    """SHA-256 over the sources, headers, this build script and the flags."""
    h = hashlib.sha256()
    if checked:
        h.update(b"LP_CHECKED")
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS + [os.path.abspath(__file__)]
    for path in deps:
        h.update(os.path.basename(path).encode())
        with open(path, "rb") as f:
            h.update(f.read())
    h.update(" ".join(NVCC_FLAGS).encode())
    return h.hexdigest()


def _stale(checked: bool = False) -> bool:
    _, lib = _paths(checked)
    stamp = lib + ".sha256"
    if not (os.path.exists(lib) and os.path.exists(stamp)):
        return True
    with open(stamp) as f:
        return f.read().strip() != source_hash(checked)


def _compile(src: str, extra: list[str], build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def _calls_paths(module: str) -> tuple[str, str]:
    """The source and the library of a module's compiled calls."""
    return os.path.join(CSRC, f"{module}_calls.cpp"), os.path.join(BUILD, f"_{module}_calls.so")


def _calls_command(module: str, out: str) -> list[str]:
    import torch
    root = os.path.dirname(torch.__file__)
    include = os.path.join(root, "include")
    libs = os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    return [shutil.which("g++") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", sysconfig.get_paths()["include"], "-I", include,
            "-I", os.path.join(include, "torch", "csrc", "api", "include"), "-I", cuda,
            _calls_paths(module)[0], "-o", out, "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", f"-Wl,-rpath,{libs}"]


def calls_hash(module: str = "train") -> str:
    """SHA-256 over a module's compiled calls: their source, the headers, the command (which names
    the flags and torch) and the versions of torch and Python."""
    import torch
    source, library = _calls_paths(module)
    h = hashlib.sha256()
    for path in (source, os.path.join(CSRC, "calls.h"), *HEADERS[:3]):
        with open(path, "rb") as f:
            h.update(f.read())
    h.update(" ".join(_calls_command(module, library)).encode())
    h.update(f"{torch.__version__} {sys.version}".encode())
    return h.hexdigest()


def build_calls(force: bool = False, quiet: bool = False, module: str = "train") -> str:
    """Compile a module's calls (_train_calls.so, _tune_calls.so) unless they were built from exactly
    this source; return their path."""
    library = _calls_paths(module)[1]
    digest, stamp = calls_hash(module), library + ".sha256"
    if not force and os.path.exists(library) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == digest:
                return library
    os.makedirs(BUILD, exist_ok=True)
    tmp = f"{library}.{os.getpid()}.tmp"
    res = subprocess.run(_calls_command(module, tmp), capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {module}_calls.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, library)
    with open(stamp, "w") as f:
        f.write(digest + "\n")
    if not quiet:
        print(f"{module} calls: compiled", flush=True)
    return library


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = False,
          checked: bool = False) -> str:
    """Compile liblp.so unless it was built from exactly these sources; return its path.
    checked=True builds the checked library (_build_checked/liblp.so) instead."""
    build_dir, lib = _paths(checked)
    what = "checked liblp" if checked else "liblp"
    if not force and not _stale(checked):
        if not quiet:
            print(f"{what}: up to date (sources sha256 {source_hash(checked)[:16]})", flush=True)
        return lib
    os.makedirs(build_dir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    if checked:
        extra += ["-DLP_CHECKED"]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra, build_dir), SOURCES))
    tmp = lib + ".tmp"
    cmd = [nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, lib)
    digest = source_hash(checked)
    with open(lib + ".sha256", "w") as f:
        f.write(digest + "\n")
    if not quiet:
        print(f"{what}: compiled {len(SOURCES)} sources for sm_103a (sources sha256 {digest[:16]})",
              flush=True)
    return lib


if __name__ == "__main__":
    print(build(force=True))
