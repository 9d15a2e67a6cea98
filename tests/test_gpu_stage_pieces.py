"""Gradients of the loss over a vocabulary that is taken in several pieces
(stage.head_backward), against the definitions in 64 bits, with the bounds of
stage_ref: the sums of dx over the pieces, the places of the targets and of dw
in each, and a last piece that is shorter."""
import math

import pytest
import torch

import stage_ref as R
from test_gpu_stage_head import S, _inputs  # noqa: F401

pytestmark = pytest.mark.gpu


def _piece(T, V):
    """Columns of a piece: the gradient of its logits takes 2^29 bytes at most, in bf16 and pieces of one size."""
    most = min(max((1 << 28) // T // 256 * 256, 256), 1 << 18)
    n = -(-V // most)
    return -(-(-(-V // n)) // 256) * 256


# few tokens (K in parts, lone blocks) and many (pairs of blocks); widths of whole panels, of whole 16 bytes and odd
SHAPES = [(3, 300000, 64), (3, 300001, 531), (130, 530000, 72), (8192, 33000, 72), (8192, 33003, 531),
          (8192, 65791, 128)]


def _case(T, V, H, seed):
    x, w, target, weight = _inputs(T, V, H, seed)
    p = _piece(T, V)
    assert p < V
    # both sides of each piece's end, the first and the last column
    ends = [c + d for c in range(p, V, p) for d in (-1, 0)] + [0, V - 1]
    target[:len(ends)] = torch.tensor(ends[:T], device="cuda")
    return x, w, target, weight


@pytest.mark.parametrize("T,V,H", SHAPES)
def test_gradients(S, T, V, H):  # noqa: F811
    x, w, target, weight = _case(T, V, H, T + V + H)
    lse = S.head_forward(x, w, target)["lse"]
    want = R.head(x, w, target, 1 / T, weight)
    got = S.head_backward(x, w, target, lse, scale=1 / T, weight=weight)
    for k in ("dx", "dw"):
        R.check(got[k], want[k], k)
    assert (got["dx"][~R.left_in(target, V)] == 0).all()
    # B and W apart, results whose rows are not aligned, nothing written beside them
    bx = torch.full((T, H + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    bw = torch.full((V, H + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    S.head_backward(x, w, target, lse, scale=1 / T, weight=weight, outputs=("dx",), out={"dx": bx[:, 1:H + 1]})
    S.head_backward(x, w, target, lse, scale=1 / T, weight=weight, outputs=("dw",), out={"dw": bw[:, 1:H + 1]})
    assert torch.equal(bx[:, 1:H + 1], got["dx"]) and torch.equal(bw[:, 1:H + 1], got["dw"])
    for b in (bx, bw):
        assert (b[:, 0] == 7).all() and (b[:, H + 1:] == 7).all()


@pytest.mark.parametrize("T,V,H", [(3, 300001, 531), (8192, 33000, 72)])
def test_added_to_a_float_sum(S, T, V, H):  # noqa: F811
    x, w, target, weight = _case(T, V, H, 3 * T + V + H)
    lse = S.head_forward(x, w, target)["lse"]
    before = torch.randn(V, H, generator=R.generator(1), device="cuda") * 1e-3
    acc = before.clone()
    S.head_backward(x, w, target, lse, scale=1 / T, weight=weight, outputs=("dw",), add=True, out={"dw": acc})
    value, bound = R.head(x, w, target, 1 / T, weight)["dw"]
    total = value + before.double()
    R.check(acc, (total, bound + R.U32 * total.abs()), "dw")


def test_left_out_rows_are_not_read(S):  # noqa: F811
    """Nor are they with several pieces, and their dx is 0 after the last."""
    T, V, H = 130, 530000, 72
    x, w, target, _ = _case(T, V, H, 4)
    gone = torch.arange(7, T, 5, device="cuda")
    target[gone] = -100
    lse = S.head_forward(x, w, target)["lse"]
    clean = S.head_backward(x, w, target, lse)
    x[gone] = math.nan
    got = S.head_backward(x, w, target, lse)
    assert torch.equal(got["dx"], clean["dx"]) and torch.equal(got["dw"], clean["dw"])
    assert (got["dx"][gone] == 0).all()
