"""The stage example: its gradients over several microbatches in 1F1B order
against the same stage written with autograd in 64 bits, and its command."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    spec = importlib.util.spec_from_file_location("stage_costs", os.path.join(ROOT, "examples", "stage_costs.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(stage, inputs, targets, scale):
    """Losses and gradients by autograd in 64 bits, from unrounded activations."""
    f64 = torch.float64
    par = {"out": stage.out.to(f64).requires_grad_()}
    for i, b in enumerate(stage.blocks):
        for k in ("matrix", "w_post", "w_pre", "gate"):
            par[i, k] = getattr(b, k).to(f64).requires_grad_()
    norm = lambda v: v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    losses, ins = [], []
    for (x, h), t in zip(inputs, targets):
        x, h = x.to(f64).requires_grad_(), h.to(f64).requires_grad_()
        ins.append((x, h))
        for i in range(len(stage.blocks)):
            x = stage.alpha * x + par[i, "gate"] * par[i, "w_post"] * norm(h @ par[i, "matrix"].t())
            h = norm(x) * par[i, "w_pre"]
        l = h @ par["out"].t()
        keep = t >= 0
        losses.append(torch.where(keep, torch.logsumexp(l, 1) - l.gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0))
    (torch.cat(losses).sum() * scale).backward()
    return losses, ins, par


def test_gradients_of_a_stage(E):
    """Activations are rounded to bf16 and kept in 8 bits (half a step of a block's largest magnitude: up to 1/128 of
    it, about 3/128 of a typical value), so the gradients agree to a few percent of their norm, not to the last
    bit; a wrong term or a lost microbatch is off by far more."""
    T, H, V, M = 96, 128, 500, 5
    stage = E.LastStage(H, V, 3, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    inputs = [tuple(torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)) for _ in range(M)]
    targets = [torch.randint(0, V, (T,), generator=gen, device="cuda") for _ in range(M)]
    targets[1][::3] = -100
    scale = 1 / (T * M)
    losses, grads, times = E.run_1f1b(stage, inputs, targets, 4, 0, scale)
    assert not stage.held and set(times) == {"F", "B", "W"}
    want, ins, par = _reference(stage, inputs, targets, scale)
    for a, b in zip(losses, want):
        assert (a - b).abs().max() < 0.1
        assert (a - b).abs().mean() < 0.02

    def near(a, b):
        return (a.double() - b).norm() / b.norm() < 0.04

    for (dx, dh), (x, h) in zip(grads, ins):
        assert near(dx, x.grad) and near(dh, h.grad)
    assert near(stage.out_sum, par["out"].grad)
    for i, b in enumerate(stage.blocks):
        for k, g in b.sums.items():
            assert near(g, par[i, k].grad), (i, k)


def test_command(E, capsys):
    E.main(["--tokens", "64", "--width", "128", "--vocab", "300", "--blocks", "2", "--stages", "4", "--microbatches", "8"])
    out = capsys.readouterr().out
    assert "zb2p" in out and "MB in 8 bits" in out
