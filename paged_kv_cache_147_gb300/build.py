"""Builds libpkv.so (the CUDA kernels behind the C ABI in include/pkv.h) in-tree for sm_103a.

The translation units compile in parallel with nvcc, then link into one shared object with
the CUDA runtime linked statically, so the library needs only the driver at run time. Beside it
goes _pkv_torch.so, the part of the Python binding that is compiled (csrc/pkv_torch.cpp), against
the installed torch; without one the library is built alone.
"""
from __future__ import annotations

import os
import shutil
import signal
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
TORCH_LIB = os.path.join(HERE, "_pkv_torch.so")
TORCH_SOURCE = "pkv_torch.cpp"
TORCH_STAMP = os.path.join(BUILD, "pkv_torch.version")   # the torch and Python it was compiled for
SOURCES = ["pkv_decode.cu", "pkv_cache.cu", "pkv_host.cu", "pkv_blocks.cpp", "pkv_spec.cu",
           "pkv_prefill.cu", "pkv_cache_int4.cu", "pkv_decode_int4.cu", "pkv_norm_rope.cu",
           "pkv_tables.cu", "pkv_cache_int8.cu", "pkv_decode_int8.cu", "pkv_select.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "-diag-suppress", "177"]


def _nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")
    return path


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != TORCH_SOURCE]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "pkv.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _torch():
    """The installed torch, or None where there is none to bind to (or one without CUDA)."""
    try:
        import torch
    except ImportError:
        return None
    return torch if torch.version.cuda else None


def _torch_tag(torch) -> str:
    return f"{torch.__version__} {sys.implementation.cache_tag}"


def _torch_stale(torch) -> bool:
    try:
        with open(TORCH_STAMP) as f:
            if f.read() != _torch_tag(torch):
                return True
        t = os.path.getmtime(TORCH_LIB)
    except OSError:
        return True
    deps = [os.path.join(CSRC, TORCH_SOURCE),
            os.path.join(os.path.dirname(HERE), "include", "pkv.h")]
    return any(os.path.getmtime(d) > t for d in deps)


class _TorchBuild:
    """g++ on the compiled binding, beside the library's own build. Leaving the context before
    finish() (that build failed) ends it and takes its output away."""

    def __init__(self, torch):
        self.torch, self.tmp = torch, TORCH_LIB + f".tmp{os.getpid()}"
        root = os.path.dirname(torch.__file__)
        lib = os.path.join(root, "lib")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
        os.makedirs(BUILD, exist_ok=True)
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               "-isystem", os.path.join(root, "include"),
               "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
               os.path.join(CSRC, TORCH_SOURCE), "-o", self.tmp, f"-L{lib}", "-ltorch_python",
               "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]
        self.process = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                        text=True, start_new_session=True)

    def finish(self) -> None:
        text, _ = self.process.communicate()
        if self.process.returncode != 0:
            sys.stdout.write(text)
            raise RuntimeError(f"g++ failed on {TORCH_SOURCE}")
        os.replace(self.tmp, TORCH_LIB)
        with open(TORCH_STAMP, "w") as f:
            f.write(_torch_tag(self.torch))

    def __enter__(self):
        return self

    def __exit__(self, *exc) -> None:
        if self.process.poll() is None:
            os.killpg(self.process.pid, signal.SIGTERM)   # g++ and the compiler it started
            self.process.communicate()
        if os.path.exists(self.tmp):
            os.remove(self.tmp)


def build(force: bool = False, verbose: bool = False, defines=(), out: str | None = None) -> str:
    """Compiles libpkv.so. `defines` (e.g. ["PKV_DECODE_STAGES=10"]) and `out` build a
    variant elsewhere; the default library is rebuilt only when a source is newer."""
    if defines or out is not None:
        return _build_library(out or LIB, BUILD if out is None else out + ".build", verbose, defines)
    torch = _torch()
    stale = force or _stale()
    if torch is None or not (force or _torch_stale(torch)):
        return _build_library(LIB, BUILD, verbose) if stale else LIB
    with _TorchBuild(torch) as binding:
        if stale:
            _build_library(LIB, BUILD, verbose)
        binding.finish()
    return LIB


def _build_library(lib: str, bdir: str, verbose: bool, defines=()) -> str:
    nvcc = _nvcc()
    os.makedirs(bdir, exist_ok=True)
    procs = []
    for src in SOURCES:
        obj = os.path.join(bdir, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *[f"-D{d}" for d in defines], "-c",
               os.path.join(CSRC, src), "-o", obj]
        procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT, text=True)))
    objs = []
    for src, obj, p in procs:
        text, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stdout.write(text)
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
        objs.append(obj)
    tmp = lib + f".tmp{os.getpid()}"
    link = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        sys.stdout.write(r.stdout)
        raise RuntimeError("linking libpkv.so failed")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
