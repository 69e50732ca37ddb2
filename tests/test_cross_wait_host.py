"""How long a wait of the cross-attention kernels may last (csrc/cross_plan.h), checked on the CPU:
host_src/cross_wait_check.cpp."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sub_quadratic_two_b200", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_a_wait_may_last_as_long_as_the_work_of_its_cta(tmp_path):
    exe = tmp_path / "cross_wait_check"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I", CSRC,
                           os.path.join(HERE, "host_src", "cross_wait_check.cpp"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout + out.stderr
