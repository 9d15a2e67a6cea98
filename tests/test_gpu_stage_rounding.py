"""What the rounding of d, the gradient of the logits, may cost the results.

d is an operand of 16 bits: every entry is off by up to 2^-8 of itself.  The
entry of a token at its target, weight (p - 1), is most of its gradient, and what
its rounding leaves over is added in 32 bits.  So of the relative error (in the
norm, over inputs with independent entries)

    sqrt(sum of (2^-8 d)^2 over the entries that are not targets / sum of d^2 over all)

is left, beside the rounding of a bf16 result, which is known exactly.  2^-12 of
a target's entry may be taken for nothing, and 2^-10 of the whole is allowed for
sums in 32 bits and for the inputs' own spread.  Without the addition the
targets' entries alone are off by about 1.6e-3 of the norm, several times what
is left at these shapes."""
import math

import pytest
import torch

import stage_ref as R

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


def _case(T, V, H, seed, spread=1.0):
    """Weighted tokens; spread > 1 makes low targets frequent."""
    g = R.generator(seed)
    x, w = R.normal(g, T, H), R.normal(g, V, H, scale=2 / math.sqrt(H))
    target = (torch.rand(T, generator=g, device="cuda") ** spread * V).long().clamp_(0, V - 1)
    return x, w, target, torch.rand(T, generator=g, device="cuda") + 0.5


def _exact(x, w, target, weight):
    x, w, c = x.to(F64), w.to(F64), weight.to(F64)
    d = torch.softmax(x @ w.t(), 1)
    rows = torch.arange(len(target), device="cuda")
    d[rows, target] -= 1
    d *= c[:, None]
    return d, d @ w, d.t() @ x


def _left(d, rows, at):
    """The error that is left: of every entry but the targets' (rows, at)."""
    rest = d.clone()
    rest[rows, at] *= 2.0 ** -4
    return 2.0 ** -8 * (rest.norm() / d.norm()).item()


def _off(got, want):
    return ((got.to(F64) - want).norm() / want.norm()).item()


SUMS = 2.0 ** -10


@pytest.mark.parametrize("T,V,H", [(777, 5000, 300), (300, 20000, 264), (64, 9000, 64), (1, 4000, 512), (3, 300000, 72),
                                   (2050, 6000, 512)])
def test_gradients_of_weighted_tokens(S, T, V, H):
    x, w, target, weight = _case(T, V, H, T + V)
    d, dx, dw = _exact(x, w, target, weight)
    lse = S.head_forward(x, w, target)["lse"]
    left = _left(d, torch.arange(T, device="cuda"), target)
    assert left < 0.5e-3  # so that the targets' own 1.6e-3 would show
    got = S.head_backward(x, w, target, lse, weight=weight)
    for k, want in (("dx", dx), ("dw", dw)):
        rounding = _off(want.to(torch.bfloat16), want)
        assert _off(got[k], want) <= math.hypot(rounding, left + SUMS / 2) + 1e-5, k
    acc = torch.zeros(V, H, device="cuda")
    S.head_backward(x, w, target, lse, weight=weight, outputs=("dw",), add=True, out={"dw": acc})
    assert _off(acc, dw) <= left + SUMS / 4


@pytest.mark.parametrize("T,V,H,spread", [(600, 3000, 128, 2.0), (900, 4000, 136, 3.0), (5000, 2000, 64, 1.0),
                                          (3000, 2500, 72, 4.0)])
def test_tokens_that_share_a_target(S, T, V, H, spread):
    """Up to eight tokens of one target are corrected, more average out; more and fewer tokens than columns."""
    x, w, target, weight = _case(T, V, H, T + V, spread)
    d, _, dw = _exact(x, w, target, weight)
    lse = S.head_forward(x, w, target)["lse"]
    count = torch.bincount(target, minlength=V)
    few = count[target] <= 8
    assert (count > 8).any() == (spread > 1 or T > 2 * V) and ((count > 1) & (count <= 8)).any()
    acc = torch.zeros(V, H, device="cuda")
    S.head_backward(x, w, target, lse, weight=weight, outputs=("dw",), out={"dw": acc})
    rows = ((count > 0) & (count <= 8)).nonzero()[:, 0]
    left = _left(d[:, rows], few.nonzero()[:, 0], torch.searchsorted(rows, target[few]))
    assert _off(acc[rows], dw[rows]) <= left + SUMS / 4
    bf = S.head_backward(x, w, target, lse, weight=weight, outputs=("dw",))["dw"]
    rounding = _off(dw[rows].to(torch.bfloat16), dw[rows])
    assert _off(bf[rows], dw[rows]) <= math.hypot(rounding, left + SUMS / 2) + 1e-5


def test_same_on_every_call_whatever_the_order_of_the_lists(S):
    x, w, target, weight = _case(3000, 1200, 136, 5, 1.5)
    lse = S.head_forward(x, w, target)["lse"]
    first = S.head_backward(x, w, target, lse, weight=weight)
    acc = torch.zeros(1200, 136, device="cuda")
    S.head_backward(x, w, target, lse, weight=weight, outputs=("dw",), out={"dw": acc})
    for _ in range(10):
        again = S.head_backward(x, w, target, lse, weight=weight)
        assert torch.equal(first["dx"], again["dx"]) and torch.equal(first["dw"], again["dw"])
        b = torch.zeros(1200, 136, device="cuda")
        S.head_backward(x, w, target, lse, weight=weight, outputs=("dw",), out={"dw": b})
        assert torch.equal(acc, b)


def test_extreme_weights(S):
    """Weights of zero, of an infinity and of NaN, and one whose rounding to bf16 is an infinity, stay with their
    tokens and add nothing but themselves."""
    T, V, H = 40, 500, 64
    x, w, _, weight = _case(T, V, H, 6)
    target = torch.arange(T, device="cuda") * 7
    lse = S.head_forward(x, w, target)["lse"]
    want = R.head(x, w, target, 1.0, weight.index_fill(0, torch.tensor([3], device="cuda"), 0.0))
    weight[3] = 0
    got = S.head_backward(x, w, target, lse, weight=weight)
    for k in ("dx", "dw"):
        R.check(got[k], want[k], k)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    for t, c in ((5, math.inf), (6, math.nan), (7, 3.4e38)):
        weight[t] = c
        rest[t] = False
    bad = S.head_backward(x, w, target, lse, weight=weight, outputs=("dx",))["dx"]
    assert torch.equal(bad[rest], got["dx"][rest])
    assert not torch.isfinite(bad[5]).any() and bad[6].isnan().all() and not torch.isfinite(bad[7]).all()
