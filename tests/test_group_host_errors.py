"""CPU: the group entry points when a launch fails, and what they check of a
binding -- tests/native/group_host.cpp, the entry points' own source against
stand-ins for the HIP runtime and the launches, under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

from gradient_reduction_optimizer_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NATIVE = os.path.join(ROOT, "tests", "native", "group_host.cpp")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def client(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("group") / "group_host")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-D__HIP_PLATFORM_AMD__", f"-I{build.ROCM}/include",
                        f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", NATIVE, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def run(client, which):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:verify_asan_link_order=0")
    r = subprocess.run([client, which], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


def test_a_step_that_fails_midway_is_not_repeated(client):
    run(client, "step")


def test_a_norm_that_fails_midway_is_not_read(client):
    run(client, "norm")
