"""The kernels that stream the weight through LDS with buffer-to-LDS loads refill a
buffer behind a barrier without a fence: a wave may arrive there only when its own LDS
reads are back.  (The compiler moves matrix instructions, and the waits of the reads
they use, past such a barrier.)  Compiles the sources for gfx950 and checks that no LDS
read is outstanding at a barrier.  CPU only."""
import os
import re
import shutil
import subprocess

import pytest

from w8a8_integer_linear_amd import build as hip_build


def reads_at_barriers(body):
    """Barriers at which an LDS read may be outstanding: (line, number of reads).  LDS
    operations complete in order, so lgkmcnt(n) leaves at most the last n."""
    out, bad = 0, []
    for l in body:
        l = l.split(";")[0].strip()
        if re.match(r"ds_(read|load)", l):
            out += 1
        w = re.search(r"lgkmcnt\((\d+)\)", l)
        if l.startswith("s_waitcnt") and w:
            out = min(out, int(w.group(1)))
        if l.startswith("s_barrier") and out:
            bad.append((l, out))
    return bad


def test_the_check_itself():
    read, wait, bar = "ds_read_b128 v[0:3], v4", "s_waitcnt vmcnt(3) lgkmcnt(%d)", "s_barrier"
    assert reads_at_barriers([read, bar]) and not reads_at_barriers([read, wait % 0, bar])
    assert reads_at_barriers([read, read, wait % 1, bar]) == [(bar, 1)]
    assert reads_at_barriers([read, "s_waitcnt vmcnt(0)", bar])


@pytest.mark.parametrize("source,kernel,count", [
    ("gemm_act.hip", "stream_act_kernel", 30), ("gemm_act_few.hip", "few_act_kernel", 9),
    ("gemm.hip", "skinny_fwd_kernel", 4), ("gemm_adapter.hip", "skinny_fwd_kernel", 4)])
def test_no_read_is_outstanding_at_a_barrier(tmp_path, source, kernel, count):
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    out = tmp_path / "k.s"
    r = subprocess.run([cc, *hip_build.FLAGS, "--cuda-device-only", "-S", os.path.join(hip_build.CSRC, source),
                        "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    asm = out.read_text()
    found = {}
    for m in re.finditer(r"^(_Z\w*%s\w*):" % kernel, asm, re.M):
        found[m.group(1)] = reads_at_barriers(asm[m.end():asm.index(".Lfunc_end", m.end())].split("\n"))
    assert len(found) == count
    assert not any(found.values()), {k: v[:3] for k, v in found.items() if v}
