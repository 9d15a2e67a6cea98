"""Records of waits that ran out, on the host: one that cannot be read is an
error, not "no failure".  The library's own collecting code
(csrc/stage_waits.h) with readers that fail in place of the CUDA calls."""
import os
import re
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "pipeline_schedule_simulation_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "stage_waits.h"
using namespace pps;
static int calls;
static int none(uint64_t *w) { ++calls, *w = 0; return 0; }
static int record(uint64_t *w) { ++calls, *w = (1ull << 63) | (5ull << 32) | 7; return 0; }
static int broken(uint64_t *) { ++calls; return 700; }
static void show(std::initializer_list<int (*)(uint64_t *)> takes) {
    WaitRecords records;
    WaitReader readers[4];
    int n = 0;
    for (auto t : takes) readers[n] = {t, nullptr}, records.add(&readers[n++]);
    uint64_t r = 42;
    calls = 0;
    const int rc = records.take(&r);
    std::printf("%d %llx %d\n", rc, (unsigned long long)r, calls);
}
int main() {
    show({});
    show({none, none});
    show({none, record, none});
    show({broken, none});
    show({none, broken});
    show({record, broken});
    show({broken, record, broken});
}
"""


def test_a_record_that_cannot_be_read_is_an_error(tmp_path):
    src, exe = tmp_path / "w.cpp", tmp_path / "w"
    src.write_text("#include <initializer_list>\n" + PROGRAM)
    subprocess.run(["g++", "-std=c++20", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    word = "8000000500000007"
    # status, record, readers asked: every reader is asked whatever the others say
    assert out[:-1] == ["0 0 0", "0 0 2", f"0 {word} 3", "700 0 2", "700 0 2", f"700 {word} 2", f"700 {word} 3"]


def test_without_a_gpu_the_answer_is_an_error():
    import torch

    from pipeline_schedule_simulation_gb300 import stage as S
    if torch.cuda.is_available():
        pytest.skip("there is a GPU")
    with pytest.raises(S.PPSchedError):
        S.wait_failure()


def test_every_waiting_role_is_documented():
    roles = set()
    for f in os.listdir(CSRC):
        if f.startswith("stage_"):
            src = open(os.path.join(CSRC, f)).read()
            roles |= {int(r) for r in re.findall(r"mbar_wait\([^;{]*?stop, (\d+)\)", src)}
    assert roles == {1, 2, 3, 4, 5, 6}
    text = open(os.path.join(ROOT, "include", "ppstage.h")).read()
    text = re.sub(r"\s*\n \*\s*", " ", text[text.index("---- waits"):])
    assert "1 loads, 2 and 3 matrix instructions, 4 results; of a ring: 5 forward, 6 backward" in text
