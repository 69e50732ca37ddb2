"""The plan of the fp32 dk, dv kernel (csrc/cross_plan.h), checked on the CPU:
host_src/cross_f32_plan_check.cpp."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sub_quadratic_two_b200", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_blocks_that_share_an_sm_fit_there(tmp_path):
    exe = tmp_path / "cross_f32_plan_check"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I", CSRC,
                           os.path.join(HERE, "host_src", "cross_f32_plan_check.cpp"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout + out.stderr
