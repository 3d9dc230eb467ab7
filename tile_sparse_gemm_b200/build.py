"""Build libpatch.so in-tree with nvcc for sm_100a (B200), and beside it, where
this torch has CUDA and its headers, the CPython extension of the decode step's
calls (without it they take their way through Python).

    python -m tile_sparse_gemm_b200.build          # compile if sources changed
    python -m tile_sparse_gemm_b200.build --force  # always recompile
    python -m tile_sparse_gemm_b200.build --debug  # libpatch_debug.so: every GEMM entry point
                                                   # first checks its weights on the device
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
LIB = PKG / "libpatch.so"
LIB_DEBUG = PKG / "libpatch_debug.so"
BINDING = PKG / "_decoder_binding.so"
SOURCES = ["capi.cu", "hard_mask.cu", "pack.cu", "gemm_decode.cu", "gemm_decode_tc.cu", "gemm_prefill.cu",
           "gemm_decode_noalloc.cu", "gated_mlp.cu", "gemm_decode_chain.cu", "mma_probe.cu", "validate.cu",
           "gemm64.cu", "capi_decoder.cu", "rope.cu", "kv8_append.cu", "attn_kv8.cu",
           "attn_kv8_rows.cu", "gemm4.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(lib: Path) -> bool:
    if not lib.exists():
        return True
    t = lib.stat().st_mtime
    deps = [CSRC / s for s in SOURCES] + list(CSRC.glob("*.cuh")) + [INCLUDE / "patch.h"]
    return any(d.stat().st_mtime > t for d in deps)


def no_binding() -> str | None:
    """Why the extension cannot be built here (the library needs nvcc alone), or None."""
    try:
        import torch
    except ImportError as e:
        return str(e)
    home = Path(torch.__file__).resolve().parent
    needed = [home / "lib" / "libtorch_cuda.so", home / "include" / "c10" / "cuda" / "CUDAStream.h",
              Path(sysconfig.get_paths()["include"]) / "Python.h"]
    missing = [str(p) for p in needed if not p.exists()] + ([] if shutil.which("g++") else ["g++"])
    return f"missing: {', '.join(missing)}" if missing else None


def build_binding(force: bool = False) -> Path:
    """_decoder_binding.so: against this interpreter's and this torch's headers."""
    import torch

    src, home = CSRC / "decoder_binding.cpp", Path(torch.__file__).resolve().parent
    if not force and BINDING.exists() and all(d.stat().st_mtime <= BINDING.stat().st_mtime
                                              for d in (src, INCLUDE / "patch.h", home / "version.py")):
        return BINDING
    cuda = Path(shutil.which(_nvcc()) or _nvcc()).parent.parent
    includes = [INCLUDE, home / "include", home / "include/torch/csrc/api/include", sysconfig.get_paths()["include"],
                cuda / "include"]
    tmp = BINDING.with_suffix(f".so.{os.getpid()}.tmp")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    *(f for i in includes for f in ("-isystem", str(i))), str(src), "-L", str(home / "lib"),
                    "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-o", str(tmp)],
                   check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> Path:
    lib = LIB_DEBUG if debug else LIB
    if force or _stale(lib):
        _build_library(lib, verbose, debug)
    if not debug:
        why = no_binding()
        if why:
            print(f"{BINDING.name} is left out: {why}", file=sys.stderr)
        else:
            build_binding(force)
    return lib


def _build_library(lib: Path, verbose: bool, debug: bool) -> None:
    build_dir = PKG / ("_build_debug" if debug else "_build")
    build_dir.mkdir(exist_ok=True)
    extra = ["-DPATCH_DEBUG"] if debug else []

    def compile_one(src):
        obj = build_dir / (src + ".o")
        cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-I", str(INCLUDE), "-c", str(CSRC / src), "-o", str(obj)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        return str(obj)

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib.with_suffix(f".so.{os.getpid()}.tmp")
    subprocess.run([_nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", str(tmp), *objs,
                    "-lcudart"], check=True)
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
