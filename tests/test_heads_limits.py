"""The largest sizes that the multi-head operators launch, and the next ones, which
they refuse (no GPU: the ABI layer with host stand-ins for the dispatchers)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or
                    not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="no host C++ compiler or HIP headers")
def test_a_launch_stays_below_2_to_32_threads(tmp_path):
    exe = str(tmp_path / "limits")
    csrc = os.path.join(ROOT, "scan_selective_fwd_amd", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                        f"-I{ROOT}/include", f"-I{csrc}",
                        os.path.join(ROOT, "tests", "sanitize", "heads_limits_driver.cpp"),
                        os.path.join(csrc, "heads_api.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "limits ok" in r.stdout, (r.stdout, r.stderr)
