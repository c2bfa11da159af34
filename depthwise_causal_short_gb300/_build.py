"""Build the sm_103a CUDA libraries ``libcconv.so`` and ``libcattn.so`` in-tree (nvcc, no cmake).

    python -m depthwise_causal_short_gb300._build

Each translation unit is compiled in parallel for sm_103a only; ``csrc/*.cu`` are linked into
``libcconv.so`` (C ABI: ``include/cconv.h``), ``csrc/attn/*.cu`` into ``libcattn.so`` (C ABI:
``include/cattn.h``), with hidden visibility for everything else and the CUDA runtime linked
statically.  ``csrc/attn/py/attn_py.cpp`` becomes ``_cattn.so``, libcattn's PyTorch binding (a
CPython extension, host compiler).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
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
ATTN_PY = LIB_DIR / "_cattn.so"

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


def attn_binding() -> Path:
    return CSRC / "attn" / "py" / "attn_py.cpp"


def _inputs(lib: Path) -> list[Path]:
    """Everything `lib` is built from."""
    shared = sorted(CSRC.glob("*.cuh")) + [INCLUDE / "cconv.h", Path(__file__)]
    if lib == ATTN_PY:
        return [attn_binding(), INCLUDE / "cattn.h", INCLUDE / "cconv.h", Path(__file__)]
    if lib == LIB:
        return sources() + shared
    headers = sorted((CSRC / "attn").glob("*.cuh")) + sorted((CSRC / "attn").glob("*.h"))
    return attn_sources() + headers + [INCLUDE / "cattn.h"] + shared


def _torch_stamp() -> Path:
    """Names the interpreter and the torch that _cattn.so was built against."""
    return OBJ_DIR / "attn_py.torch"


def _torch_version() -> str:
    import torch
    return f"{sys.version} / {torch.__version__} / {Path(torch.__file__).resolve().parent}"


def _newer(lib: Path) -> bool:
    if not lib.exists():
        return False
    if lib == ATTN_PY and (not _torch_stamp().exists() or _torch_stamp().read_text() != _torch_version()):
        return False
    t = lib.stat().st_mtime
    return all(p.stat().st_mtime <= t for p in _inputs(lib))


def up_to_date() -> bool:
    return _newer(LIB) and _newer(ATTN_LIB) and _newer(ATTN_PY)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> Path:
    """Compile and link each library unless it is newer than every source of it."""
    todo = [(lib, srcs) for lib, srcs in ((LIB, sources()), (ATTN_LIB, attn_sources()))
            if force or extra_flags or not _newer(lib)]
    binding = force or not _newer(ATTN_PY)
    if not todo and not binding:
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

    def compile_binding() -> Path:
        import sysconfig

        import torch
        root = Path(torch.__file__).resolve().parent
        obj = OBJ_DIR / "attn_py.o"
        cuda = Path(exe).resolve().parent.parent
        dirs = [root / "include", root / "include" / "torch" / "csrc" / "api" / "include",
                cuda / "include", sysconfig.get_paths()["include"]]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               *[a for d in dirs for a in ("-isystem", str(d))], "-c", str(attn_binding()), "-o", str(obj)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {attn_binding().name}:\n{r.stdout}\n{r.stderr}")
        return obj

    def link(lib: Path, cmd: list[str]):
        tmp = lib.with_suffix(f".{os.getpid()}.tmp")
        r = subprocess.run([*cmd, "-o", str(tmp)], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of {lib.name} failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        py_obj = ex.submit(compile_binding) if binding else None
        built = {src: ex.submit(compile_one, src) for _, srcs in todo for src in srcs}
    for lib, srcs in todo:
        link(lib, [exe, *ARCH, "-shared", "-cudart", "static", *[str(built[src].result()) for src in srcs]])
    if py_obj is not None:
        import torch
        libs = Path(torch.__file__).resolve().parent / "lib"
        _torch_stamp().unlink(missing_ok=True)
        link(ATTN_PY, ["g++", "-shared", str(py_obj.result()), f"-L{LIB_DIR}", "-lcattn",
                       "-Wl,-rpath,$ORIGIN", f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10",
                       "-lc10_cuda"])
        _torch_stamp().write_text(_torch_version())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None))
