"""Build libtbe.so (HIP kernels for gfx950 + the C ABI) and _lmcall.so (Python
calls of the language-model operators) in-tree.

    python bwd_tbe_pooled_amd/build.py

Every HIP source is compiled for gfx950 only, with packed-fp32 instructions
disabled (the compiler would otherwise pair float operations into
v_pk_*_f32, which this library does not use).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtbe.so")
CALLS = os.path.join(HERE, "_lmcall.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-Wall",
          "-Wno-unused-function", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", INCLUDE, "-I", CSRC]

SOURCES = ["api.cpp", "util.hip", "forward.hip", "hot_rows.hip", "sort.hip", "rle_route.hip",
           "backward.hip", "hot_backward.hip", "probe.hip", "small_table.hip",
           "lm_api.cpp", "token.hip", "expert.hip", "distill.hip"]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {src}\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    # the host pass does not know the packed-fp32 target feature: drop that note
    noise = "'-packed-fp32-ops' is not a recognized feature"
    msgs = [l for l in (r.stderr or "").splitlines() if noise not in l and l.strip()]
    if msgs:
        print("\n".join(msgs), file=sys.stderr)
    return obj


def _hip_include() -> str:
    """The directory HIPCC has HIP's headers from. The compiler is asked, as it may
    be a name found on PATH or a wrapper outside the ROCm tree."""
    cmd = [HIPCC, "-x", "hip", "--offload-host-only", "-M", "-"]
    r = subprocess.run(cmd, input="#include <hip/hip_runtime_api.h>\n", capture_output=True, text=True)
    tail = os.path.join("hip", "hip_runtime_api.h")
    for path in r.stdout.split():
        if r.returncode == 0 and path.endswith(os.sep + tail):
            return os.path.abspath(path[:-len(tail)])
    raise RuntimeError(f"HIP's headers not found\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def _build_calls() -> None:
    """Host code only: it looks into torch's tensors and calls through addresses."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    tmp = CALLS + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"), "-isystem", _hip_include(),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "lm_call.cpp"), "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"build failed: lm_call.cpp\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        print(r.stderr, file=sys.stderr)
    os.replace(tmp, CALLS)


def build(jobs: int = 8) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        calls = ex.submit(_build_calls)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    calls.result()  # after the library, which the table calls need alone
    return LIB


def clean() -> None:
    shutil.rmtree(BUILD, ignore_errors=True)


if __name__ == "__main__":
    print(build())
