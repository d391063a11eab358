"""LDS that a kernel is given at its launch starts behind what the compiler laid out for it: on 16 bytes wherever it is
read and written 16 bytes at a time. Taken from the built library's own notes; no kernel is launched."""
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_quantized_moe_amd", "libnvfp4moe.so")
LLVM = os.environ.get("LLVM_BIN", "/opt/rocm/llvm/bin")


@pytest.fixture(scope="module")
def fixed(tmp_path_factory):
    """LDS bytes that the compiler gave each kernel, by its name."""
    if not os.path.exists(LIB):
        pytest.skip("library not built (run build())")
    if not all(os.path.exists(os.path.join(LLVM, tool)) for tool in ("llvm-objdump", "llvm-readelf")):
        pytest.skip("no LLVM tools")
    where = str(tmp_path_factory.mktemp("lib"))
    shutil.copy(LIB, where)
    name = os.path.basename(LIB)
    subprocess.run([os.path.join(LLVM, "llvm-objdump"), "--offloading", name], cwd=where, check=True, capture_output=True)
    sizes = {}
    for code in glob.glob(os.path.join(where, "*gfx950*")):
        notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", code], check=True, capture_output=True, text=True)
        for kernel in notes.stdout.split("- .agpr_count")[1:]:
            sizes[re.search(r"\.name:\s+(\S+)", kernel[kernel.index(".max_flat"):]).group(1)] = int(
                re.search(r"\.group_segment_fixed_size:\s+(\d+)", kernel).group(1))
    return sizes


@pytest.mark.parametrize("kernel", ["few_down_kernel", "layer_norm_backward_kernel", "block_norm_backward_kernel",
                                    "grouped_gemm_kernel"])
def test_starts_on_16_bytes(fixed, kernel):
    sizes = {n: v for n, v in fixed.items() if kernel in n}
    assert sizes
    assert not {n: v for n, v in sizes.items() if v % 16}
