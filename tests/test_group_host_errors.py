"""CPU: the group entry points when a launch fails, and what they check of a
binding -- tests/native/group_host.cpp, the entry points' own source against
stand-ins for the HIP runtime and the launches, under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

from gradient_reduction_optimizer_amd import binding as B
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


def test_a_workspace_inside_an_array_is_refused():
    """The kernels would overwrite the table of array pointers that they
    follow.  Refused on the host: no pointer here is one of a device."""
    for bits8 in (False, True):
        h = B.gro_group_create([dict(numel=100_000, coded_moments=bits8)] * 2)
        need = B.gro_group_get_info(h)["workspace_bytes"]
        size = [400_000, 100_000, 100_000, 6252, 6252, 200_000] if bits8 else [400_000, 400_000, 400_000, 0, 0, 200_000]
        base = [[(1 + 6 * i + j) << 24 if size[j] else 0 for j in range(6)] for i in range(2)]
        for i in range(2):
            for j in range(6):
                if not size[j]:
                    continue
                at, last = base[i][j], (base[i][j] + size[j] - 1) // 256 * 256
                for ws in (at, last, at - need + 256):      # from its first byte, its last ones, up to its first ones
                    with pytest.raises(B.GroError) as e:
                        B.gro_group_bind(h, base, ws, need)
                    assert e.value.kind == "duplicate", (i, j, ws)
        B.gro_group_destroy(h)
