"""The bound of the scale bytes that the FP8 products read (fp8_internal.h),
checked on the host over every load of the kernels' tiles."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "microscaling_fp4_quantized_block_amd", "csrc")
CXX = "/opt/rocm/lib/llvm/bin/clang++"


@pytest.mark.skipif(not os.path.exists(CXX), reason="needs ROCm clang")
def test_scale_reads_end_with_the_operands_rows(tmp_path):
    exe = str(tmp_path / "extent")
    r = subprocess.run([CXX, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", CSRC, "-I", "/opt/rocm/include",
                        os.path.join(ROOT, "tests", "helpers", "fp8_extent.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


def test_every_scale_resource_has_the_bound():
    """No product bounds a resource of scales by whole lines of the matrix around a view."""
    with open(os.path.join(CSRC, "fp8_gemm.hip")) as f:
        text = f.read()
    calls = [line for line in text.splitlines() if "resource(" in line and "scales" in line]
    assert len(calls) == 3 and all("fp8_scale_extent(" in line for line in calls)
