"""Compile the CUDA library in-tree for sm_103a (nvcc, no cmake)."""
from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libspecverify.so")
DEBUG_LIB_PATH = os.path.join(PKG, "libspecverify_debug.so")  # range-checked build (-DSV_DEBUG)
SOURCES = [os.path.join(CSRC, f) for f in ("spec_verify.cu", "sv_kv.cu", "sv_budget.cu", "sv_append.cu",
                                              "sv_attention.cu", "sv_logprobs.cu", "sv_cache.cu",
                                              "sv_attention_e4m3.cu", "sv_chunk.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("sv_device.cuh", "sv_draw.cuh", "sv_stream.cuh", "sv_rescan.cuh",
                                                  "sv_decide.cuh", "sv_topkp.cuh", "sv_topkp_ring.cuh",
                                                  "sv_check.cuh", "sv_ops.cuh", "sv_tc.cuh", "sv_e4m3.cuh", "sv_reference.cuh",
                                                  "sv_attention.cuh")] + [
    os.path.join(INCLUDE, "spec_verify.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def _nvcc() -> str:
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return nvcc if os.path.exists(nvcc) else "nvcc"


def compile_command(source: str, out: str, debug: bool = False) -> list[str]:
    return [_nvcc(), *NVCC_FLAGS, *(["-DSV_DEBUG"] if debug else []), "-I", INCLUDE, "-c", source, "-o", out]


def up_to_date(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in DEPS)


class _Build:
    """A compilation under way: one nvcc per source, linked when all have ended."""

    def __init__(self, path: str, debug: bool):
        self.path = path
        self.objects = [f"{path}.{os.path.basename(s)}.{os.getpid()}.o" for s in SOURCES]
        self.procs = [subprocess.Popen(compile_command(s, o, debug)) for s, o in zip(SOURCES, self.objects)]

    def finish(self) -> str:
        try:
            if any([p.wait() for p in self.procs]):
                raise RuntimeError(f"nvcc failed building {os.path.basename(self.path)}")
            tmp = f"{self.path}.tmp{os.getpid()}"
            subprocess.run([_nvcc(), "-shared", *self.objects, "-o", tmp], check=True)
            os.replace(tmp, self.path)
        finally:
            for o in self.objects:
                if os.path.exists(o):
                    os.remove(o)
        return self.path


def start_build(force: bool = False, debug: bool = False):
    """Start nvcc in the background; returns the build (or None when already built).  debug: the
    range-checked library (libspecverify_debug.so) instead of the release one."""
    path = DEBUG_LIB_PATH if debug else LIB_PATH
    if not force and up_to_date(path):
        return None
    return _Build(path, debug)


def finish_build(build) -> str:
    return LIB_PATH if build is None else build.finish()


def build(force: bool = False) -> str:
    finish_build(start_build(force))
    return LIB_PATH


def build_debug(force: bool = False) -> str:
    """The range-checked library: every global-memory access of every kernel checked (-DSV_DEBUG)."""
    finish_build(start_build(force, debug=True))
    return DEBUG_LIB_PATH
