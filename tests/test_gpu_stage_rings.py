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
from test_gpu_stage_join import EPS, S, _forward, _inputs  # noqa: F401

pytestmark = pytest.mark.gpu
ROUNDS = 9  # rows a block: two for each of four stages, and one


def _rows(H, threads_on_sm):
    """Rows that give every ring block more than ROUNDS: a block has a thread for every 16 columns (for 8 up to 1024),
    in whole warps, and an SM as many blocks as fit."""
    threads = -(-(-(-H // (8 if H <= 1024 else 16))) // 32) * 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return sms * (threads_on_sm // threads) * ROUNDS + 5


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
