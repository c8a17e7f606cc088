"""CPU: the launch-shape knobs that lane.h and plan.h offer and the committed
launch-shape comparison builds with: every source of the library still compiles
with them (syntax and static assertions; nothing is linked or run)."""
import os
import subprocess

import pytest

from gradient_reduction_optimizer_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")

VARIANTS = {"block512": ["GRO_BLOCK=512", "GRO_UNROLL_ADAMW=2"], "chunk8k": ["GRO_CHUNK_ELEMS=8192"],
            "block128": ["GRO_BLOCK=128", "GRO_UNROLL_ADAMW=8"]}


@pytest.mark.parametrize("source", build.HIP_SOURCES)
@pytest.mark.parametrize("name", VARIANTS)
def test_sources_compile_with_the_knobs(name, source):
    cmd = [build.HIPCC, *build.COMMON, *build.HIP_FLAGS, *(f"-D{d}" for d in VARIANTS[name]), "-fsyntax-only",
           "--cuda-device-only", os.path.join(build.CSRC, f"{source}.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
