"""Builds libspecverify.so (sm_103a) in-tree with nvcc.

Each CUDA translation unit is compiled in parallel, then linked into one
shared library next to this file; beside them g++ compiles the bindings' tensor
checks (``csrc/tensors.cpp``, against the installed torch's headers).  Usage: ``python -m
mtp_speculative_decoding_qmv_gb300.build [--force] [--debug]``.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = PKG / "_build"
LIB = PKG / "libspecverify.so"
CHECKS = PKG / "_tensors.so"
CHECKS_FOR = BUILD / "_tensors.for"  # what _tensors.so was compiled for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify")


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def _stale(target: Path, deps: list[Path]) -> bool:
    if not target.exists():
        return True
    t = target.stat().st_mtime
    return any(d.stat().st_mtime > t for d in deps)


def interpreter() -> str:
    """What the extension's ABI depends on: torch and Python."""
    import torch

    return f"torch {torch.__version__} at {torch.__file__}, Python {sys.version}"


def checks_stale() -> bool:
    """_tensors.so is older than its sources, or was compiled for another torch."""
    return (_stale(CHECKS, [CSRC / "tensors.cpp", INCLUDE / "specverify.h", Path(__file__)])
            or not CHECKS_FOR.exists() or CHECKS_FOR.read_text() != interpreter())


def build_checks() -> None:
    """The CPython extension of csrc/tensors.cpp."""
    import torch

    cuda = Path(nvcc()).resolve().parents[1]
    src = CSRC / "tensors.cpp"
    root = Path(torch.__file__).parent
    tmp = CHECKS.with_suffix(".so.tmp")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{root / 'include'}", f"-I{root / 'include/torch/csrc/api/include'}",
           "-I" + sysconfig.get_paths()["include"], f"-I{cuda / 'include'}", f"-I{INCLUDE}",
           str(src), "-o", str(tmp),
           f"-L{root / 'lib'}", f"-Wl,-rpath,{root / 'lib'}", "-ltorch_python", "-ltorch_cpu",
           "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src.name}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CHECKS)
    BUILD.mkdir(exist_ok=True)
    CHECKS_FOR.write_text(interpreter())


def build(force: bool = False, debug: bool = False, verbose: bool = False) -> Path:
    headers = list(CSRC.glob("*.h")) + list(CSRC.glob("*.cuh")) + list(INCLUDE.glob("*.h"))
    srcs = sources()
    checks = force or checks_stale()
    if not force and not _stale(LIB, srcs + headers + [Path(__file__)]):
        if checks:
            build_checks()
        return LIB
    BUILD.mkdir(exist_ok=True)
    flags = ARCH + ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
                    "-I", str(INCLUDE), "-I", str(CSRC), "--expt-relaxed-constexpr"]
    if debug:
        flags += ["-DSV_DEBUG"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    cc = nvcc()

    def compile_one(src: Path) -> Path:
        obj = BUILD / (src.stem + ".o")
        cmd = [cc, *flags, "-c", str(src), "-o", str(obj)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src.name}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        extension = ex.submit(build_checks) if checks else None
        objs = list(ex.map(compile_one, srcs))
        if extension:
            extension.result()
    tmp = LIB.with_suffix(".so.tmp")
    cmd = [cc, *ARCH, "-shared", "-o", str(tmp), *map(str, objs)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--debug", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, debug=a.debug, verbose=a.verbose))
