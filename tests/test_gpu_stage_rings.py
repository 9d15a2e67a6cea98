"""The join of long runs of rows, whose rows come through a ring of bulk copies
(stage.join_forward, join_backward): every stage of the ring is filled several
times over, against the definitions in 64 bits, with stage_ref's bounds.

The number of rows follows from the GPU's SMs and from the most blocks that
share an SM, so that a block's rows go round the ring of at most four stages
more than twice."""
import math

import pytest
import torch

import stage_ref as R
from test_gpu_stage_join import EPS, S, _backward, _forward, _inputs  # noqa: F401

pytestmark = pytest.mark.gpu
ROUNDS = 9  # rows a block: two for each of four stages, and one


def _rows(H, threads_on_sm):
    """Rows that give every ring block more than ROUNDS: a block has a thread for every 16 columns (for 8 up to 1024),
    in whole warps, and an SM as many blocks as fit."""
    threads = -(-(-(-H // (8 if H <= 1024 else 16))) // 32) * 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return sms * (threads_on_sm // threads) * ROUNDS + 5


# one and two vectors a thread, each size of block, rows as wide as the block's vectors (multiples of 512) and narrower
WIDTHS = [520, 1000, 1024, 1360, 1536, 2048, 2504, 4096, 5128, 8192]


def _short_last_group(a, T):
    """Three gates, the last of them for fewer rows than the others: the runs that its rows are cut into end early,
    and some have no row."""
    a["rows"] = 5 * T // 12
    assert 2 * a["rows"] < T < 3 * a["rows"]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("groups", [0, 1, 3])
def test_forward(S, H, groups):  # noqa: F811
    T = _rows(H, 1024)
    a = _inputs(T, H, groups, T + H)
    if groups == 3:
        _short_last_group(a, T)
    want = R.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], a["gate"], a["rows"], 0.7, EPS)
    plain = _forward(S, a, 0.7)
    kept = _forward(S, a, 0.7, keep=True)
    for k in want:
        R.check(plain[k], want[k], k)
        assert torch.equal(plain[k], kept[k]), k
    for k, of in (("kept_y", kept["y"]), ("kept_f", a["f"])):
        q, e = R.pack(of)
        assert torch.equal(kept[k].q, q) and torch.equal(kept[k].e, e), k
    # a row does not depend on the kernel that takes it
    few = {k: (v[-7:] if k in ("x", "f") else v) for k, v in a.items()}
    if groups == 3:
        few["gate"], few["rows"] = a["gate"][2:], 0
    few = _forward(S, few, 0.7)
    for k in want:
        R.check(few[k], tuple(t[-7:] for t in want[k]), k)


@pytest.mark.parametrize("H", [528, *WIDTHS])  # 520, 1000, 2504 and 5128: checkpoint rows that bulk copies cannot take
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("groups", [1, 3])
def test_backward(S, H, packed, groups):  # noqa: F811
    T = _rows(H, 512)
    a = _inputs(T, H, groups, 2 * T + H)
    if groups == 3:
        _short_last_group(a, T)
    fw = _forward(S, a, 0.7, keep=packed)
    y, f = (fw["kept_y"], fw["kept_f"]) if packed else (fw["y"], a["f"])
    yv, fv = (R.value(y.q, y.e), R.value(f.q, f.e)) if packed else (y, f)
    for dy in (True, False):
        got = _backward(S, a, y, f, fw["rstd_post"], fw["rstd_pre"], 0.7, dy=dy)
        want = R.join_backward(a["dh"], a["dy"] if dy else None, yv, fv, fw["rstd_post"], fw["rstd_pre"], a["w_post"],
                               a["w_pre"], a["gate"], a["rows"], 0.7)
        assert set(got) == set(want)
        for k in want:
            R.check(got[k], want[k], k)


@pytest.mark.parametrize("packed", [False, True])
def test_backward_of_nonfinite_rows(S, packed):  # noqa: F811
    """A row with a NaN or an infinity leaves the results of other rows as they are, in whichever round it comes."""
    H = 1360
    T = _rows(H, 512)
    a = _inputs(T, H, 1, 5)
    fw = _forward(S, a, 1.0, keep=packed)
    y, f = (fw["kept_y"], fw["kept_f"]) if packed else (fw["y"], a["f"])
    good = _backward(S, a, y, f, fw["rstd_post"], fw["rstd_pre"], 1.0)
    bad = torch.tensor([0, 1, 4, 5, 9, T // 2, T - 1], device="cuda")
    a["dh"][bad, 3] = math.nan
    a["dy"][bad, H - 1] = math.inf
    got = _backward(S, a, y, f, fw["rstd_post"], fw["rstd_pre"], 1.0)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[bad] = False
    for k in ("dx", "df"):
        assert torch.equal(got[k][rest], good[k][rest]), k
        assert got[k][bad].isnan().all(), k


@pytest.mark.parametrize("H", [520, 1360, 2504, 5128])
@pytest.mark.parametrize("where", ["w_post", "gate"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_nonfinite_weight_of_the_first_column(S, H, where, value):  # noqa: F811
    """Rows that end before the block's last vector: what is past their end adds nothing to the norm, whatever the
    weights of a row's own columns are.  An infinite weight of column 0 gives an infinite y there, so rstd_pre is 0
    and h is 0 beside it."""
    T = _rows(H, 1024)
    a = _inputs(T, H, 1, 6)
    a["f"][:, 0] = 0.5
    a[where][..., 0] = value
    got = _forward(S, a, 0.7, keep=True)
    want = R.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], a["gate"], 0, 0.7, EPS)
    for k in want:
        R.check(got[k], want[k], k)
    if value == math.inf:
        assert (got["rstd_pre"] == 0).all() and (got["h"][:, 1:] == 0).all()
    q, e = R.pack(got["y"])
    assert torch.equal(got["kept_y"].q, q) and torch.equal(got["kept_y"].e, e)
    assert (got["kept_y"].e[:, 0] == -128).all() and (got["kept_y"].e[:, 1:] != -128).all()
