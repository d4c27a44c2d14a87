"""Address and undefined-behaviour sanitizer build of the expert-layer host
code (dense_ragged_grouped_amd/csrc/api_moe.cpp, its launchers replaced by
stubs), driven by tests/sanitize/moe_driver.cpp (CPU only; host code only,
built with g++)."""
import os
import shutil
import subprocess

import pytest

from tests.test_sanitize import HERE, ROCM, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="needs g++ and the HIP headers")
def test_moe_host_code_under_sanitizers(tmp_path):
    exe = str(tmp_path / "moe_driver")
    csrc = os.path.join(ROOT, "dense_ragged_grouped_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(HERE, "moe_driver.cpp"), os.path.join(csrc, "api_moe.cpp"), "-o", exe], check=True)
    _run(exe, tmp_path)
