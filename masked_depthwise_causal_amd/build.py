"""Compile the HIP libraries (libmccb.so, libmccb_ssm.so) for gfx950, and the binding of the second
(_ssm.so), in-tree."""
from __future__ import annotations

import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "mccb.hip")
# MCCB_LIBRARY names another build of the library to load instead (the tests' host-sanitized
# build); it is loaded as given and never built.
LIB = os.environ.get("MCCB_LIBRARY") or os.path.join(PKG, "libmccb.so")
INCLUDE = os.path.join(ROOT, "include")
# the state space block's operators; MCCB_SSM_LIBRARY as above
SSM_SRCS = [os.path.join(PKG, "csrc", f) for f in ("ssm_conv.hip", "ssm_scan.hip", "ssm_linear.hip")]
SSM_LIB = os.environ.get("MCCB_SSM_LIBRARY") or os.path.join(PKG, "libmccb_ssm.so")
BINDING_SRC = os.path.join(PKG, "csrc", "ssm_binding.cpp")
BINDING = os.path.join(PKG, "_ssm.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-shared", "-fPIC",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def build_library(out: str = LIB, extra: list[str] | None = None, verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    cmd = [hipcc, *HIPCC_FLAGS, *(extra or []), "-I", INCLUDE, SRC, "-o", out + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stderr}")
    if verbose:
        print(res.stderr)
    os.replace(out + ".tmp", out)
    return out


def build_ssm_library(out: str = SSM_LIB, extra: list[str] | None = None,
                      verbose: bool = False) -> str:
    """One object a source, compiled side by side, then linked."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stderr}")
        if verbose:
            print(res.stderr)

    flags = [f for f in HIPCC_FLAGS if f != "-shared"] + (extra or [])
    objects = [f"{out}.{os.path.basename(src)}.o" for src in SSM_SRCS]
    try:
        with ThreadPoolExecutor(len(SSM_SRCS)) as pool:
            list(pool.map(lambda so: run([hipcc, *flags, "-I", INCLUDE, "-c", so[0], "-o", so[1]]),
                          zip(SSM_SRCS, objects)))
        run([hipcc, *HIPCC_FLAGS, *(extra or []), *objects, "-o", out + ".tmp"])
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    os.replace(out + ".tmp", out)
    return out


def build_binding(out: str = BINDING) -> str:
    """The tensor front end of libmccb_ssm.so, host code against torch's C++ interface."""
    import torch
    from torch.utils import cpp_extension

    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    cmd = [hipcc, "-x", "c++", "-O2", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__=1",
           "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"]]
    for path in cpp_extension.include_paths("cuda"):
        cmd += ["-isystem", path]
    cmd += [BINDING_SRC, "-o", out + ".tmp"]
    for path in cpp_extension.library_paths("cuda"):
        cmd += ["-L", path]
    cmd += ["-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stderr}")
    os.replace(out + ".tmp", out)
    return out


def build_all() -> list[str]:
    """Both libraries and the binding, side by side."""
    with ThreadPoolExecutor(3) as pool:
        return [f.result() for f in [pool.submit(b) for b in
                                     (build_library, build_ssm_library, build_binding)]]


if __name__ == "__main__":
    print(*build_all())
