"""Compile the HIP libraries (libmccb.so, libmccb_ssm.so, libmccb_delta.so) for gfx950, and the bindings
of the last two (_ssm.so, _delta.so), in-tree."""
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
# the gated delta rule and the norms; MCCB_DELTA_LIBRARY as above
DELTA_SRCS = [os.path.join(PKG, "csrc", f) for f in ("delta_norm.hip", "delta_rule.hip",
                                                    "delta_back.hip")]
DELTA_LIB = os.environ.get("MCCB_DELTA_LIBRARY") or os.path.join(PKG, "libmccb_delta.so")
DELTA_BINDING_SRC = os.path.join(PKG, "csrc", "delta_binding.cpp")
DELTA_BINDING = os.path.join(PKG, "_delta.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-shared", "-fPIC",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


# the delta rule's walks have a SIMD's registers to themselves, where the compiler would have the matrix
# instructions' results in accumulation registers and move each of them (674 vector instructions a chunk, 578 without)
DELTA_FLAGS = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]


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


def _build_objects(srcs: list[str], out: str, extra: list[str] | None, verbose: bool) -> str:
    """One object a source, compiled side by side, then linked."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stderr}")
        if verbose:
            print(res.stderr)

    flags = [f for f in HIPCC_FLAGS if f != "-shared"] + (extra or [])
    objects = [f"{out}.{os.path.basename(src)}.o" for src in srcs]
    try:
        with ThreadPoolExecutor(len(srcs)) as pool:
            list(pool.map(lambda so: run([hipcc, *flags, "-I", INCLUDE, "-c", so[0], "-o", so[1]]),
                          zip(srcs, objects)))
        run([hipcc, *HIPCC_FLAGS, *(extra or []), *objects, "-o", out + ".tmp"])
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    os.replace(out + ".tmp", out)
    return out


def build_ssm_library(out: str = SSM_LIB, extra: list[str] | None = None,
                      verbose: bool = False) -> str:
    return _build_objects(SSM_SRCS, out, extra, verbose)


def build_delta_library(out: str = DELTA_LIB, extra: list[str] | None = None,
                        verbose: bool = False) -> str:
    return _build_objects(DELTA_SRCS, out, DELTA_FLAGS + (extra or []), verbose)


def build_binding(out: str = BINDING, src: str = BINDING_SRC) -> str:
    """The tensor front end of a library, host code against torch's C++ interface."""
    import torch
    from torch.utils import cpp_extension

    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    cmd = [hipcc, "-x", "c++", "-O2", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__=1",
           "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"]]
    for path in cpp_extension.include_paths("cuda"):
        cmd += ["-isystem", path]
    cmd += [src, "-o", out + ".tmp"]
    for path in cpp_extension.library_paths("cuda"):
        cmd += ["-L", path]
    cmd += ["-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stderr}")
    os.replace(out + ".tmp", out)
    return out


def build_delta_binding(out: str = DELTA_BINDING) -> str:
    return build_binding(out, DELTA_BINDING_SRC)


def build_all() -> list[str]:
    """The libraries and the bindings, side by side."""
    with ThreadPoolExecutor(5) as pool:
        return [f.result() for f in [pool.submit(b) for b in
                                     (build_library, build_ssm_library, build_binding,
                                      build_delta_library, build_delta_binding)]]


if __name__ == "__main__":
    print(*build_all())
