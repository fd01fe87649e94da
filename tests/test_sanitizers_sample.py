"""The argument checks of sampling (kda_sample_api.cpp) built
with AddressSanitizer and UndefinedBehaviorSanitizer (host only) and swept
over extreme sizes by tests/sanitize/sample_driver.cpp: any report, undocumented
status or launch too large to be made fails."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import FLAGS, ROCM_INCLUDE, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE),
                    reason="g++ or the HIP headers not available")
def test_sample_validation_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "sample_driver")
    r = subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE,
                        "-I", os.path.join(ROOT, "include")] + FLAGS
                       + [os.path.join(SAN, "sample_driver.cpp"),
                          os.path.join(ROOT, "gated_delta_rule_27_amd", "csrc", "kda_sample_api.cpp"),
                          "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "all checks passed" in _run(exe)
