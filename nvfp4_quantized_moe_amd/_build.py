"""Build libnvfp4moe.so for gfx950 with hipcc and the native part of the Python
binding with the host compiler (in-tree, no JIT cache)."""
from __future__ import annotations

import glob
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libnvfp4moe.so")
NATIVE = os.path.join(PKG, "_native.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # packed fp32 VALU ops are kept out of generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


PROBE_LIB = os.path.join(PKG, "libnvfp4probe.so")


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.hip")))


def probe_sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "probe", "*.hip")))


def _run(cmd, out, verbose):
    tmp = out + ".tmp"
    res = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(os.path.basename(cmd[0]) + " failed:\n" + res.stdout + res.stderr)
    if verbose:
        msg = "\n".join(l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l)
        if msg.strip():
            print(msg)
    os.replace(tmp, out)


def _compile(srcs, out, verbose):
    jobs = f"-parallel-jobs={min(8, len(srcs), os.cpu_count() or 1)}"   # 80 s; one after the other 160
    _run([HIPCC, *FLAGS, jobs, "-I", os.path.join(ROOT, "include"), *srcs], out, verbose)


def _compile_native(verbose):
    """csrc/binding.cpp against torch's headers; it finds the library beside itself."""
    import torch
    th = os.path.dirname(torch.__file__)
    inc = os.path.join(th, "include")
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          os.path.join(PKG, "csrc", "binding.cpp"), "-L", PKG, "-lnvfp4moe", "-Wl,-rpath,$ORIGIN",
          "-L", os.path.join(th, "lib"), "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10"], NATIVE, verbose)


def build(verbose: bool = False) -> str:
    """Compile every HIP source of the layer into one shared library next to
    this file, the binding's native calls, and the benchmark's roofline probes."""
    _compile(sources(), LIB, verbose)
    _compile_native(verbose)
    _compile(probe_sources(), PROBE_LIB, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
