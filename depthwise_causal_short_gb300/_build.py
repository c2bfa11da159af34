"""Build the sm_103a CUDA libraries ``libcconv.so`` and ``libcattn.so`` in-tree (nvcc, no cmake).

    python -m depthwise_causal_short_gb300._build

Each translation unit is compiled in parallel for sm_103a only; ``csrc/*.cu`` are linked into
``libcconv.so`` (C ABI: ``include/cconv.h``), ``csrc/attn/*.cu`` into ``libcattn.so`` (C ABI:
``include/cattn.h``), with hidden visibility for everything else and the CUDA runtime linked
statically.
"""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
OBJ_DIR = PKG / "_build"
LIB_DIR = PKG / "_lib"
LIB = LIB_DIR / "libcconv.so"
ATTN_LIB = LIB_DIR / "libcattn.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", str(INCLUDE),
]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libcconv.so")
    return exe


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def attn_sources() -> list[Path]:
    return sorted((CSRC / "attn").glob("*.cu"))


def _inputs(lib: Path) -> list[Path]:
    """Everything `lib` is built from."""
    shared = sorted(CSRC.glob("*.cuh")) + [INCLUDE / "cconv.h", Path(__file__)]
    if lib == LIB:
        return sources() + shared
    return attn_sources() + sorted((CSRC / "attn").glob("*.cuh")) + [INCLUDE / "cattn.h"] + shared


def _newer(lib: Path) -> bool:
    if not lib.exists():
        return False
    t = lib.stat().st_mtime
    return all(p.stat().st_mtime <= t for p in _inputs(lib))


def up_to_date() -> bool:
    return _newer(LIB) and _newer(ATTN_LIB)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> Path:
    """Compile and link each library unless it is newer than every source of it."""
    todo = [(lib, srcs) for lib, srcs in ((LIB, sources()), (ATTN_LIB, attn_sources()))
            if force or extra_flags or not _newer(lib)]
    if not todo:
        return LIB
    OBJ_DIR.mkdir(parents=True, exist_ok=True)
    LIB_DIR.mkdir(parents=True, exist_ok=True)
    exe = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: Path) -> Path:
        obj = OBJ_DIR / (src.stem + ".o")
        cmd = [exe, *ARCH, *flags, "-c", str(src), "-o", str(obj)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src.name}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        built = {src: ex.submit(compile_one, src) for _, srcs in todo for src in srcs}
    for lib, srcs in todo:
        objs = [built[src].result() for src in srcs]
        tmp = lib.with_suffix(f".{os.getpid()}.tmp")
        cmd = [exe, *ARCH, "-shared", "-cudart", "static", "-o", str(tmp), *map(str, objs)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of {lib.name} failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None))
