"""The barriers of the cross-attention kernels in a host model that runs the roles in random order:
host_src/cross_protocol_check.cpp. A wait that is left out of the model has to be found."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sub_quadratic_two_b200", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path_factory.mktemp("model") / "cross_protocol_check"
    subprocess.check_call(["g++", "-O2", "-std=c++20", "-I", CSRC,
                           os.path.join(HERE, "host_src", "cross_protocol_check.cpp"), "-o", str(exe)])
    return lambda *args: subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, timeout=300)


@pytest.mark.parametrize("seed", range(5))
def test_every_role_finds_what_it_waits_for(model, seed):
    out = model(1200, seed)  # forward with no mask, lengths and key masks, whole and split keys; both backward kernels
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout + out.stderr


# forward, dQ, dK and dV (where 2 is not used: no mask passes through that kernel's barriers)
@pytest.mark.parametrize("plant", [*range(1, 9), *range(11, 19), 21, *range(23, 29)])
def test_a_wait_left_out_is_found(model, plant):
    out = model(600, 1, plant)
    assert out.returncode == 1 and out.stdout.startswith("FAIL"), out.stdout + out.stderr
