"""The products of few tokens with an activation reuse their stage buffers for the sums
after the contraction's loop.  The barrier between the two has no fence: a wave may
arrive there only when its own LDS reads are back, and that wait stands at each of the
kernel's barriers, whatever the compiler moves into or out of the loop before it.
Compiles the source for gfx950.  CPU only."""
import os
import re
import shutil
import subprocess

import pytest

from w8a8_integer_linear_amd import build as hip_build


def barriers_without_a_wait(body):
    """Barriers whose own straight run of code, back to the label or branch before it, has
    no wait for all LDS reads behind its last one."""
    bad, waited = [], False
    for n, l in enumerate(body):
        l = l.split(";")[0].strip()
        if l.endswith(":") or re.match(r"s_c?branch|ds_(read|load)", l):
            waited = False
        if l.startswith("s_waitcnt") and "lgkmcnt(0)" in l:
            waited = True
        if l.startswith("s_barrier") and not waited:
            bad.append(n)
    return bad


def test_the_check_itself():
    read, wait, bar = "ds_read_b128 v[0:3], v4", "s_waitcnt lgkmcnt(0)", "s_barrier"
    assert barriers_without_a_wait([read, wait, bar]) == []
    assert barriers_without_a_wait([read, wait, ".LBB0_1:", bar]) == [3]
    assert barriers_without_a_wait([wait, read, bar]) == [2]
    assert barriers_without_a_wait(["s_waitcnt vmcnt(0)", bar]) == [1]


def test_every_barrier_has_its_wait(tmp_path):
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    out = tmp_path / "k.s"
    r = subprocess.run([cc, *hip_build.FLAGS, "--cuda-device-only", "-S",
                        os.path.join(hip_build.CSRC, "gemm_act_few.hip"), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    asm = out.read_text()
    found = {}
    for m in re.finditer(r"^(_Z\w*few_act_kernel\w*):", asm, re.M):
        found[m.group(1)] = barriers_without_a_wait(asm[m.end():asm.index(".Lfunc_end", m.end())].split("\n"))
    assert found and not any(found.values()), {k: v[:3] for k, v in found.items() if v}
