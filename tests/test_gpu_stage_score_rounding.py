"""What the rounding of d costs the gradients of scores on peaked rows.

d is an operand of 16 bits, and only the target's term keeps what its rounding leaves
over.  Behind a policy gradient the likeliest other column of a peaked row may be as
large as the target, and stays rounded.  So the gradients are those of a d whose
terms are rounded to bf16 but for the targets' (in dw: of targets that at most
eight tokens share), and of nothing less.

Tolerance.  A term of d is known to 2^-18 of itself before its rounding: its logit is
exact here, the argument of its exponential is below 32 and rounded to 2^-24 of that
three times, the exponential to 2 units, its factors and lse to less.  Numbers of 8
significant bits lie 2^-8 of themselves apart at least, so that at most one term in
2^8 2^-18 2 = 2^-9 is rounded to the other neighbour and off by 2^-7 at most:
sqrt(2^-9) 2^-7 = 3.4e-4 of the norm.  With the terms' own 2^-18 and sums in 32 bits
that is below 2^-11.  A target's term that was rounded would add 1.1e-3 (its share of
the norm is 0.7 at least) and rounded sums more."""
import math

import pytest
import torch

import score_ref as Q
import stage_ref as R

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


@pytest.mark.parametrize("T,V,H", [(256, 4096, 64), (77, 3001, 104), (3, 20000, 64), (1, 700, 64)])
@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("entropy", [False, True])
def test_peaked_rows(S, T, V, H, sampled, entropy):
    g = R.generator(T + V)
    x, w = Q.grid(g, T, H), Q.grid(g, V, H, scale=2.0 ** round(math.log2(6 / math.sqrt(H))))  # logits some six units wide
    xd, wd = x.to(F64), w.to(F64)
    lp = torch.log_softmax(xd @ wd.t(), 1)
    p = lp.exp()
    target = (torch.multinomial(p, 1, generator=g) if sampled else torch.randint(0, V, (T, 1), generator=g, device="cuda"))[:, 0]
    a = torch.randn(T, generator=g, device="cuda")
    b = torch.full((T,), -0.01, device="cuda") if entropy else None
    ent = -(p * lp).sum(1, keepdim=True)
    d = -p * a.to(F64)[:, None]
    if entropy:
        d -= b.to(F64)[:, None] * p * (lp + ent)
    rows = torch.arange(T, device="cuda")
    d[rows, target] += a.to(F64)
    kept = d.to(torch.bfloat16).to(F64)
    by_token = kept.clone()
    by_token[rows, target] = d[rows, target]
    few = torch.bincount(target, minlength=V)[target] <= 8
    kept[rows[few], target[few]] = d[rows[few], target[few]]
    f = S.score_forward(x, w, target)
    more = dict(entropy=f["entropy"], dentropy=b) if entropy else {}
    acc = torch.zeros(V, H, device="cuda")
    S.score_backward(x, w, target, f["lse"], a, outputs=("dw",), add=True, out={"dw": acc}, **more)
    got = S.score_backward(x, w, target, f["lse"], a, **more)
    dx, dw = d @ wd, d.t() @ xd

    def off(y, want, of):
        return ((y.to(F64) - want).norm() / of.norm()).item()

    assert off(acc, kept.t() @ xd, dw) <= 2.0 ** -11
    for name, want, of in (("dx", by_token @ wd, dx), ("dw", kept.t() @ xd, dw)):
        # the result's own rounding, and together no more than the 2^0.5 of it that a rounded d can make
        rounding = off(want.to(torch.bfloat16), want, of)
        assert off(got[name], want, of) <= rounding + 2.0 ** -10, name
        assert off(got[name], of, of) <= math.hypot(rounding, 2.0 ** -8) + 2.0 ** -11, name
