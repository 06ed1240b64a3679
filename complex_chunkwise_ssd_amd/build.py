"""Compiles the gfx950 library (libssd.so, hipcc) and the compiled part of the Python
binding (_binding.so, the C++ compiler against torch's headers) in place.

    python -m complex_chunkwise_ssd_amd.build
"""

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libssd.so")
BINDING = os.path.join(PKG, "_binding.so")
ARCH = "gfx950"
SOURCES = ("ssd_api.hip", "ssd_ops_api.hip")


def hipcc_command(out: str, extra=()):
    return [
        "hipcc", "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-shared",
        # keep hipcc from forming packed fp32 instructions on its own
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I" + INCLUDE, "-I" + CSRC, *extra,
        *(os.path.join(CSRC, f) for f in SOURCES), "-o", out,
    ]


def binding_command(out: str):
    import sysconfig

    import torch
    torch_dir = os.path.dirname(torch.__file__)
    include = os.path.join(torch_dir, "include")
    return [
        "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1",
        "-DTORCH_API_INCLUDE_EXTENSION_H", "-DTORCH_EXTENSION_NAME=_binding", "-Wall", "-Wextra",
        "-I" + INCLUDE, "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
        "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"],
        os.path.join(CSRC, "ssd_ops_binding.cpp"), "-o", out,
        "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python",
    ]


def _compile(cmd, out: str, tmp: str, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("%s failed for %s" % (cmd[0], os.path.basename(out)))
    if verbose:
        sys.stderr.write(res.stderr)  # warnings
    os.replace(tmp, out)


def build(verbose: bool = False, extra=()) -> str:
    tmp = LIB + ".tmp%d" % os.getpid()
    _compile(hipcc_command(tmp, extra), LIB, tmp, verbose)
    tmp = BINDING + ".tmp%d" % os.getpid()
    _compile(binding_command(tmp), BINDING, tmp, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
