"""The products with an activation in their epilogues share the product kernels' main
loop with its inline-asm fragment reads: the same checks of the compiled code as for
the plain products, and no register spill.  CPU only."""
import os
import re
import shutil
import subprocess

import pytest

from tests.test_gemm_asm_hazard import _kernels, fragment_read_hazards, loop_exit_hazards
from w8a8_integer_linear_amd import build as hip_build

KERNELS = 5 * 2 * 2         # activations, with and without a gate, whole and split tiles


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "gemm_act.s"
    cmd = [cc, *hip_build.FLAGS, "--cuda-device-only", "-S",
           os.path.join(hip_build.CSRC, "gemm_act.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text()


@pytest.fixture(scope="module")
def kernels(asm):
    found = _kernels(asm)
    assert len(found) == KERNELS
    return found


def test_no_register_reuse_before_fragment_reads_land(kernels):
    found = {k: loop_exit_hazards(body) for k, body in kernels.items()}
    assert not any(found.values()), {k: v[:3] for k, v in found.items() if v}


def test_fragment_reads_are_waited_for_before_use(kernels):
    found = {k: fragment_read_hazards(body) for k, body in kernels.items()}
    assert not any(found.values()), {k: v[:3] for k, v in found.items() if v}


def test_nothing_is_spilled(asm):
    spills = re.findall(r"\.name:\s+(_Z\w*gemm_kernel\w*)(?:.|\n)*?\.vgpr_spill_count:\s+(\d+)", asm)
    assert len(spills) == KERNELS and all(n == "0" for _, n in spills), spills

