"""Long sums lose no more of themselves than short ones.

The tensor cores cut a sum off at every step, so that a sum of terms of one
sign shrinks, in proportion to its length if nothing is done.  Sums are taken
in runs of 2048 terms that are added up with rounding: each run shrinks by the
same share whatever the number of runs, and r - 1 additions of r runs round by
2^-24 of the sum at most.  So for terms of one distribution

    mean |error / value| of 8192 terms  <=  that of 2048 terms + 3 * 2^-24

where a single run of 8192 would be off by four times the error of 2048.  Each
mean is over at least 2^19 sums; 1/64 of it is allowed for their spread."""
import pytest
import torch

import stage_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


def _positive(g, *shape, scale=1.0):
    """Uniform over the upper half of 0 .. scale: no number is far below the others."""
    return ((0.5 + 0.5 * torch.rand(*shape, generator=g, device="cuda")) * scale).to(torch.bfloat16)


def _off(got, want):
    return ((got.double() - want) / want).abs().mean().item()


def _no_longer_than(short, long, roundings):
    assert long <= short * (1 + 1 / 64) + roundings * 2.0 ** -24, (short, long)


def test_weight_gradient(S):
    # enough tiles for the SMs: K is not cut into parts, which would shorten the sums
    N, H = 2560, 2560
    off = []
    for T in (2048, 8192):
        g = R.generator(T)
        dy, p = _positive(g, T, N), S.pack(_positive(g, T, H))
        off.append(_off(S.weight_grad(dy, p), dy.double().t() @ R.value(p.q, p.e)))
    _no_longer_than(*off, 3)


def test_logits(S):
    """Logits of about 100, all alike, so that each log-sum-exp is off by what its 1024 logits are off by, and by the
    rounding of its own last steps: the logarithm, the sum with the largest logit and the sums of exponentials (2^-24
    each, of numbers no larger than the result)."""
    T, V = 512, 1024
    off = []
    for H in (2048, 8192):
        g = R.generator(H)
        # mean of a product (0.75 of each scale) squared times H is 100
        x, w = (_positive(g, n, H, scale=(100 / (0.5625 * H)) ** 0.5) for n in (T, V))
        got = S.head_forward(x, w, torch.zeros(T, dtype=torch.int64, device="cuda"))["lse"]
        off.append(_off(got, torch.logsumexp(x.double() @ w.double().t(), 1)))
    _no_longer_than(*off, 3 + 3)
