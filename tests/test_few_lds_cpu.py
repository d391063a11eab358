"""Shared memory of the few tokens' down kernel: what the host asks for at every number of tokens and choices, together
with what the compiler laid out for the kernel, fits a compute unit, and the faster variant is taken wherever it does.
few.hip is compiled for gfx950 and few_lds.h for the host; no kernel is launched."""
import importlib.util
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_quantized_moe_amd", "csrc")
LDS = 160 * 1024

WALK = r"""
#include <cstdio>
#include "few_lds.h"
int main() {
  for (int T = 1; T <= 64; ++T)
    for (int k = 1; k <= 64; ++k) {
      const nvfp4::FewDownLds d = nvfp4::few_down_lds(T, k);
      std::printf("%d %d %d %zu\n", T, k, (int)d.ring, d.bytes);
    }
}
"""


def build_script():
    spec = importlib.util.spec_from_file_location("_nvfp4_build", os.path.join(ROOT, "nvfp4_quantized_moe_amd", "_build.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def fixed(tmp_path_factory):
    """LDS bytes that the compiler gives each kernel of few.hip, by its name."""
    b = build_script()
    if not (os.path.exists(b.HIPCC) or shutil.which(b.HIPCC)):
        pytest.skip("hipcc not available")
    asm = str(tmp_path_factory.mktemp("few") / "few.s")
    flags = [f for f in b.FLAGS if f != "-shared"]
    run = subprocess.run([b.HIPCC, *flags, "-I", os.path.join(ROOT, "include"), "--offload-device-only", "-S",
                          os.path.join(CSRC, "few.hip"), "-o", asm], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
    with open(asm) as f:
        found = re.findall(r"\.amdhsa_kernel (\S+)\s+\.amdhsa_group_segment_fixed_size (\d+)", f.read())
    return {name: int(size) for name, size in found}


@pytest.fixture(scope="module")
def asked(tmp_path_factory):
    """{(T, k): (ring, bytes)}"""
    cxx = build_script().CXX
    if not shutil.which(cxx):
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("walk")
    src, exe = where / "walk.cpp", where / "walk"
    src.write_text(WALK)
    run = subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
    rows = [[int(v) for v in line.split()] for line in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines()]
    assert len(rows) == 64 * 64
    return {(T, k): (bool(ring), n) for T, k, ring, n in rows}


def of_down(fixed, ring):
    name, = [n for n in fixed if f"few_down_kernelILb{int(ring)}E" in n]
    return fixed[name]


def test_every_size_fits(fixed, asked):
    for (T, k), (ring, n) in asked.items():
        assert n >= 8 * T * 36 * 4 + T * k * 6
        assert of_down(fixed, ring) + n <= LDS, (T, k, ring)


def test_through_lds_wherever_it_fits(fixed, asked):
    for (T, k), (ring, n) in asked.items():
        assert ring == (of_down(fixed, True) + n <= LDS), (T, k)


def test_up_kernel_fits(fixed):
    """Its choices, 2 bytes each, are all that it is given at the launch."""
    name, = [n for n in fixed if "few_up_kernel" in n]
    assert fixed[name] + 64 * 64 * 2 <= LDS
