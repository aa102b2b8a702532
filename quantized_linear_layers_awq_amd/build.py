"""Compile the HIP library (libtilefuse.so) for gfx950, in-tree, and the host
module that marshals the attention and cache calls (_calls.so).

Every HIP source is compiled with hipcc for gfx950 only; packed-fp32 code
generation is switched off for all device code.  _calls.so is plain C++ against
torch's headers, by the same compiler; where torch is not installed, so that the
library serves C programs alone, it is left out.  The results land next to this
file, where the binding loads them.
"""

from __future__ import annotations

import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(HERE, "libtilefuse.so")
CALLS_PATH = os.path.join(HERE, "_calls.so")
SOURCES = ("api.hip", "repack.hip", "gemv.hip", "gemm.hip", "gemm256.hip", "probe.hip", "attn_api.hip",
           "attn_decode.hip", "attn_prefill.hip", "kv.hip")
ARCH = "gfx950"


def hipcc() -> str:
    return os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def compile_flags() -> list[str]:
    # -amdgpu-mfma-vgpr-form: MFMA accumulators in arch VGPRs, so the GEMM's
    # per-group rescale is one multiply per accumulator (no AGPR round trips)
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-mllvm", "-amdgpu-mfma-vgpr-form",
            "-I", INCLUDE, "-I", CSRC]


def _compile_calls() -> str | None:
    try:
        import torch
    except ModuleNotFoundError:
        return None
    from torch.utils.cpp_extension import include_paths

    obj = os.path.join(BUILD_DIR, "torch_calls.o")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    includes = [x for path in (*include_paths(), sysconfig.get_paths()["include"]) for x in ("-isystem", path)]
    cmd = [hipcc(), "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", INCLUDE,
           *includes, "-c", os.path.join(CSRC, "torch_calls.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError(f"hipcc failed on torch_calls.cpp:\n{r.stdout}{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    from torch.utils.cpp_extension import library_paths

    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = [hipcc(), "-no-hip-rt", "-shared", "-fPIC", obj, "-o", tmp, "-L", HERE, "-l:libtilefuse.so",
           *[f"-L{path}" for path in library_paths()], "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, CALLS_PATH)


def build(verbose: bool = False) -> str:
    """Compile every source, link libtilefuse.so and, where torch is, _calls.so; returns the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)

    def one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        cmd = [hipcc(), *compile_flags(), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        out = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
        if r.returncode:
            raise RuntimeError(f"hipcc failed on {src}:\n{out}")
        if verbose and out.strip():
            print(out)
        return obj

    jobs = min(len(SOURCES), int(os.environ.get("MAX_JOBS", "8")))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        calls = ex.submit(_compile_calls)
        objs = list(ex.map(one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if calls.result():
        _link_calls(calls.result())
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
