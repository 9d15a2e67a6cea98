"""What the build compiles anew: every object after a change to any header it
may include, and nothing otherwise.  The build's own code, on a small tree and
with a compiler that only writes its output."""
import os
import subprocess

import pytest

from pipeline_schedule_simulation_gb300 import build_lib as L

HEADERS = ("include/ppsched.h", "include/ppstage.h", "csrc/common.cuh", "csrc/host_only.h")
SOURCES = ("csrc/one.cu", "csrc/two.cu")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    for d in ("include", "csrc", "_build"):
        (tmp_path / d).mkdir()
    for f in HEADERS + SOURCES:
        (tmp_path / f).write_text("")
        os.utime(tmp_path / f, (1000, 1000))
    monkeypatch.setattr(L, "ROOT", str(tmp_path))
    monkeypatch.setattr(L, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(L, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(L, "LIB", str(tmp_path / "_build" / "lib.so"))
    monkeypatch.setattr(L, "_nvcc", lambda: "nvcc")
    compiled = []

    def run(cmd, **kw):
        if "-c" in cmd:
            compiled.append(os.path.basename(cmd[cmd.index("-c") + 1]))
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(L.subprocess, "run", run)

    def build():
        del compiled[:]
        L.build()
        return sorted(compiled)

    return tmp_path, build


def test_nothing_is_compiled_twice(tree):
    _, build = tree
    assert build() == ["one.cu", "two.cu"]
    assert build() == []


@pytest.mark.parametrize("header", HEADERS)
def test_a_changed_header_recompiles_everything(tree, header):
    root, build = tree
    build()
    later = os.path.getmtime(root / "_build" / "one.o") + 10
    os.utime(root / header, (later, later))
    assert build() == ["one.cu", "two.cu"]


def test_a_changed_source_recompiles_itself(tree):
    root, build = tree
    build()
    later = os.path.getmtime(root / "_build" / "one.o") + 10
    os.utime(root / "csrc/two.cu", (later, later))
    assert build() == ["two.cu"]
