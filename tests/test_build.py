"""The library's build where the binding's compiled half cannot be built."""
import subprocess

import pytest

from w8a8_integer_linear_amd import build as hip_build


def test_library_is_linked_without_the_bindings_headers(monkeypatch, tmp_path):
    """libqlin.so needs neither torch's nor Python's headers: it is there although the
    build then fails, and the failure names what is missing."""
    lib = tmp_path / "libqlin.so"
    linked = []

    def run(cmd, **kw):         # the linker
        linked.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def no_headers(verbose):
        raise RuntimeError("Python.h: no such file")

    monkeypatch.setattr(hip_build, "LIB", str(lib))
    monkeypatch.setattr(hip_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(hip_build, "_compile", lambda src, verbose: src + ".o")
    monkeypatch.setattr(hip_build, "_build_marshal", no_headers)
    monkeypatch.setattr(hip_build.subprocess, "run", run)
    monkeypatch.setattr(hip_build, "hipcc", lambda: "hipcc")
    with pytest.raises(RuntimeError, match="Python.h"):
        hip_build.build()
    assert lib.exists() and [s + ".o" for s in hip_build.SOURCES] == [a for a in linked[0] if a.endswith(".hip.o")]
