"""A wait of the join's ring that runs out: the block is told so, asks for no
more rows, lets the copies in flight land and ends, and the context stays
usable.  The ring is the library's own (csrc/stage_ring.cuh), in a kernel
of one block with a limit of some milliseconds in place of two seconds; the
wait runs out because its barrier expects 16 bytes that nothing copies."""
import ctypes
import os
import subprocess

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu
STAGES = 4


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    from pipeline_schedule_simulation_gb300 import build_lib as L
    so = str(tmp_path_factory.mktemp("probe") / "ring_probe.so")
    r = subprocess.run([L._nvcc(), *L.ARCH, *L.FLAGS, "-I", L.CSRC, "-shared", "-cudart", "static", "-o", so,
                        os.path.join(ROOT, "tests", "stage_ring_probe.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(so)
    lib.ring_probe.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 3 + [ctypes.c_ulonglong] + [ctypes.c_void_p] * 4

    def run(rows, words, held, limit_ms=5):
        x = torch.randint(0, 1 << 20, (rows, words), dtype=torch.int32, device="cuda")
        out = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        issued, landed = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(STAGES, dtype=torch.int32, device="cuda")
        record = ctypes.c_uint64()
        torch.cuda.synchronize()
        rc = lib.ring_probe(x.data_ptr(), rows, words, held, limit_ms * 1000000, out.data_ptr(), issued.data_ptr(),
                            landed.data_ptr(), ctypes.byref(record))
        assert rc == 0
        return x, out.tolist(), issued.item(), landed.tolist(), record.value

    return run


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 8, 9, 41])
def test_every_row_comes(probe, rows):
    x, out, issued, landed, record = probe(rows, 1024, -1, limit_ms=2000)
    assert out == x.sum(1).tolist() and issued == rows and record == 0
    assert landed == [int(i < rows) for i in range(STAGES)]


@pytest.mark.parametrize("held", [0, 2, 3, 5, 10, 37, 40])
def test_a_wait_that_runs_out(probe, held):
    rows = 41
    x, out, issued, landed, record = probe(rows, 1024, held)
    # the rows before it came; the first wait of the block is on record, as role 5 of block 0
    assert out == x.sum(1).tolist()[:held] + [0] * (rows - held)
    assert record == 1 << 63 | 5 << 32
    # rows were asked for up to the last one that every thread had read, and no further
    assert issued == min(rows, held + STAGES)
    # every copy has landed; only the barrier that was held up stays open
    assert landed == [int(i != held % STAGES) for i in range(STAGES)]
    # the next launch works as before
    x, out, issued, landed, record = probe(rows, 1024, -1, limit_ms=2000)
    assert out == x.sum(1).tolist() and issued == rows and record == 0
