"""Bytes of the weight that a stage's loads may reach in the products with an activation:
from the stage to the weight's end, and none for a stage past the work unit's end, whose
loads are issued all the same and have to come back empty.  Checked by the compiler from
the kernels' own header; CPU only."""
import os
import shutil
import subprocess

import pytest

from w8a8_integer_linear_amd import build as hip_build

CHECKS = """
#include "gemm_kernel.hpp"
using namespace qlin;
static_assert(free_records(true, 4096) == 4096, "to the weight's end");
static_assert(free_records(true, kOob) == kOob && free_records(true, kOob + 4096) == kOob, "32-bit offsets");
static_assert(free_records(false, 4096) == 0 && free_records(false, 0xFFFFFF80u) == 0, "past the end");
"""


def test_extents(tmp_path):
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    src = tmp_path / "k.hip"
    src.write_text(CHECKS)
    r = subprocess.run([cc, *hip_build.FLAGS, f"-I{hip_build.CSRC}", "--cuda-device-only", "-fsyntax-only", str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    plan = open(os.path.join(hip_build.CSRC, "gemm_kernel.hpp")).read()
    assert "make_rsrc(bk, free_records(L.live, bleft - (uint32_t)k0))" in plan
