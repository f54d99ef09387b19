"""Builds ``libmi355gemm.so`` and ``libmi355fused.so`` (the C-ABI libraries)
from ``csrc/`` and ``csrc/fused/`` with hipcc for gfx950.

Usage: ``python -m dense_gemm_sgemm_amd.build`` or ``build()`` from Python.
Each ``.hip`` file is compiled to an object in ``_build/`` (in parallel), then
linked in place next to this file so that the libraries travel with the tree.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libmi355gemm.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
FUSED_CSRC = os.path.join(CSRC, "fused")
FUSED_LIB_PATH = os.path.join(HERE, "libmi355fused.so")
ARCH = "gfx950"

# Packed fp32 VALU instructions are kept out of the generated code on purpose;
# hipcc's host pass warns that it does not know the feature, which is harmless.
HIPCC_FLAGS = [
    "-O3", "--offload-arch=" + ARCH, "-fPIC", "-std=c++17", "-fvisibility=hidden",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I" + INCLUDE, "-I" + CSRC,
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain (ROCm) is required to build")


# Per-source compiler flags.  The fp16 tile kernels (A * B^T and the in-place
# layouts) keep two register sets of
# operand fragments and 112-128 accumulator registers live in each of its
# waves; LLVM's register-minimising scheduler spills less there than the
# default one and measured about 1 % faster on 5376 x 5376 x 2048.
FILE_FLAGS = {
    "hgemm_mfma.hip": ["-mllvm", "--amdgpu-sched-strategy=iterative-minreg"],
    "hgemm_kmajor.hip": ["-mllvm", "--amdgpu-sched-strategy=iterative-minreg"],
    "tiles_gated.hip": ["-mllvm", "--amdgpu-sched-strategy=iterative-minreg"],
    "tiles_logits.hip": ["-mllvm", "--amdgpu-sched-strategy=iterative-minreg"],
    "tiles_grad.hip": ["-mllvm", "--amdgpu-sched-strategy=iterative-minreg"],
}


def sources(folder: str = CSRC) -> list[str]:
    return sorted(os.path.join(folder, f) for f in os.listdir(folder) if f.endswith(".hip"))


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, *FILE_FLAGS.get(os.path.basename(src), []), *extra, "-c", src,
           "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr))
    return obj


def _link(objs: list[str], lib_path: str) -> None:
    tmp = lib_path + ".tmp%d" % os.getpid()
    cmd = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
    os.replace(tmp, lib_path)


def build(extra_flags: list[str] | None = None, jobs: int | None = None) -> str:
    """Compile every kernel source for gfx950 and link the shared libraries."""
    extra = list(extra_flags or [])
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs, fused = sources(), sources(FUSED_CSRC)
    with ThreadPoolExecutor(max_workers=jobs or min(8, len(srcs) + len(fused))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), srcs + fused))
    _link(objs[:len(srcs)], LIB_PATH)
    _link(objs[len(srcs):], FUSED_LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(sys.argv[1:]))
