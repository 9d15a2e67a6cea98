"""Score, its gradients, their norm and the step as a last stage uses them
together, and the stage example's step."""
import importlib.util
import math
import os

import pytest
import torch

import score_ref as Q
import stage_ref as R
import step_ref as P
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


def _policy(S, bits, seed):
    """Three steps on two microbatches each: log probabilities weighted, an entropy term, gradients added up in 32 bits,
    clipped, a step on the 32-bit matrix whose 16-bit copy the next pass reads."""
    T, V, H = 90, 400, 64
    g = R.generator(21)
    w = R.normal(g, V, H, scale=2 / math.sqrt(H))
    master, dw = w.float(), torch.zeros(V, H, device="cuda")
    opt = S.AdamW([master], bits=bits, copies=[w], betas=(0.9, 0.95), eps=0.1, weight_decay=0.1, seed=seed)
    want = master.double()
    m = v = torch.zeros(V, H, dtype=R.F64, device="cuda")
    moved = 0.0
    for t in range(1, 4):
        dw.zero_()
        exact, norms = torch.zeros(V, H, dtype=R.F64, device="cuda"), []
        for _ in range(2):
            x = R.normal(g, T, H)
            target = torch.randint(-20, V, (T,), generator=g, device="cuda")
            a, b = torch.randn(T, generator=g, device="cuda"), torch.full((T,), -0.05, device="cuda")
            f = S.score_forward(x, w, target, top=4)
            S.score_backward(x, w, target, f["lse"], a, entropy=f["entropy"], dentropy=b, outputs=("dw",), add=True,
                             out={"dw": dw})
            ref = Q.score(x, w, target, 4, a, b)
            for k in ("logp", "entropy", "top_logp"):
                R.check(f[k], ref[k], k)
            exact += ref["dw"][0]
        norm = S.grad_norm([dw])
        opt.step([dw], 0.05, norm=norm, max_norm=5.0)
        true = exact.norm()
        assert abs(norm.double() - true) <= 2e-3 * true
        before = want
        r = P.step(want, exact, m, v, t, 0.05, (0.9, 0.95), 0.1, 0.1, min(1.0, 5.0 / float(true)))
        want, m, v = (r[k][0] for k in ("p", "m", "v"))
        moved += float((want - before).norm())
        torch.cuda.synchronize()
        assert torch.equal(w, master.to(torch.bfloat16))
    assert int(opt.state["step"]) == 3 and S.wait_failure() == 0
    return float((master.double() - want).norm()) / moved


def test_steps_on_a_policy_gradient(S):
    """The gradient's terms are rounded to bf16, half a step 2^-9 of each on average at most: their sum is off by some
    10^-3 of its norm; the step with eps well above most gradients passes that on as it is.  Moments in 8 bits are off
    by 2^-4 (to nearest) or 2^-3 of themselves at most, m at once and the root of v by half of that."""
    assert _policy(S, 32, None) <= 0.01
    assert _policy(S, 8, None) <= 0.01 + 2 ** -4 + 2 ** -5
    assert _policy(S, 8, 3) <= 0.01 + 2 ** -3 + 2 ** -4


def test_the_examples_step(capsys):
    """The stage's tensors after its step against the definition, from the sums that the microbatches left."""
    spec = importlib.util.spec_from_file_location("stage_costs", os.path.join(ROOT, "examples", "stage_costs.py"))
    E = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(E)
    T, H, V, M = 64, 128, 300, 4
    stage = E.LastStage(H, V, 2, seed=5)
    g = R.generator(22)
    inputs = [tuple(R.normal(g, T, H) for _ in range(2)) for _ in range(M)]
    targets = [torch.randint(0, V, (T,), generator=g, device="cuda") for _ in range(M)]
    E.run_1f1b(stage, inputs, targets, 2, 0, 1 / (T * M))
    old, sums = [p.clone() for p in stage.adamw.params], [s.clone() for s in stage.sums]
    assert len(old) == len(sums) == 9 and all(s.abs().max() > 0 for s in sums)
    norm = float(stage.step(1e-2, max_norm=0.1))
    total = math.sqrt(sum(float(s.double().square().sum()) for s in sums))
    assert abs(norm - total) <= 1e-6 * total
    for p, q, s, c in zip(stage.adamw.params, old, sums, stage.adamw.copies):
        z = torch.zeros_like(q)
        decay = 0.1 if q.dim() == 2 and q.shape[0] > 1 else 0.0
        R.check(p, P.step(q, s, z, z, 1, 1e-2, (0.9, 0.95), 1e-8, decay, min(1.0, 0.1 / total))["p"])
        assert torch.equal(c, p.to(torch.bfloat16))
    assert all((s == 0).all() for s in stage.sums) and stage.blocks[0].matrix is stage.adamw.copies[0]
    assert stage.blocks[1].sums["gate"] is stage.sums[7] and stage.out_sum is stage.sums[8]
    E.main(["--tokens", "64", "--width", "128", "--vocab", "300", "--blocks", "2", "--stages", "4", "--microbatches", "8"])
    assert "the step over" in capsys.readouterr().out
