"""score, the step and the gradients' norm without a GPU: argument errors are
answered on the host before any CUDA call."""
import ctypes

import pytest
import torch

from pipeline_schedule_simulation_gb300 import binding as B
from pipeline_schedule_simulation_gb300 import stage as S

L = B.LIB
P = 1 << 20  # stands for an aligned pointer; never followed


def score_f(T=4, V=10, H=8, x=P, sx=8, w=P, sw=8, t=P, top=3, logp=P, lse=P, ent=P, tl=P, ti=P, ws=P, n=1 << 40):
    return L.pp_stage_score_forward(x, sx, w, sw, t, T, V, H, top, logp, lse, ent, tl, ti, ws, n, None)


def score_b(T=4, V=10, H=8, x=P, sx=8, w=P, sw=8, t=P, lse=P, dl=P, ent=P, de=P, dx=P, sdx=8, dw=P, sdw=8, wide=0, add=0, ws=P,
            n=1 << 40):
    return L.pp_stage_score_backward(x, sx, w, sw, t, lse, dl, ent, de, T, V, H, dx, sdx, dw, sdw, wide, add, ws, n, None)


@pytest.mark.parametrize("call", [score_f, score_b])
def test_inputs(call):
    for bad in (dict(T=-1), dict(V=0), dict(H=0), dict(x=None), dict(w=None), dict(t=None), dict(x=P + 1), dict(w=P + 1),
                dict(t=P + 4), dict(sx=7), dict(sw=7), dict(ws=None), dict(ws=P + 16), dict(n=8)):
        assert call(**bad) == B.PP_ERR_ARG, bad
    for big in (dict(T=(1 << 24) + 1), dict(V=(1 << 24) + 1), dict(H=(1 << 16) + 1)):
        assert call(**big) == B.PP_ERR_SIZE, big


def test_score_outputs():
    for bad in (dict(top=-1), dict(top=11), dict(top=0, logp=None, lse=None, ent=None), dict(logp=P + 2), dict(lse=P + 1),
                dict(ent=P + 2), dict(tl=None), dict(ti=None), dict(ti=P + 4), dict(tl=P + 2)):
        assert score_f(**bad) == B.PP_ERR_ARG, bad
    assert score_f(V=100, top=33) == B.PP_ERR_SIZE
    assert score_f(T=0, x=None, t=None, ws=None, n=0) == B.PP_OK
    for bad in (dict(lse=None), dict(dl=None), dict(dl=P + 2), dict(ent=None), dict(ent=P + 2), dict(de=P + 2),
                dict(dx=None, dw=None), dict(sdx=7), dict(sdw=7), dict(add=1), dict(wide=1, dw=P + 2)):
        assert score_b(**bad) == B.PP_ERR_ARG, bad


def test_workspaces():
    f, b = L.pp_stage_score_forward_workspace, L.pp_stage_score_backward_workspace
    assert f(P, 8, P, 8, 0, 10, 8, 0) == 0 and b(P, 8, P, 8, 0, 10, 8) == 0
    assert f(P, 8, P, 8, 4, 10, 8, 33) == 0
    assert 0 < f(P, 4096, P, 4096, 4096, 131072, 4096, 0) < f(P, 4096, P, 4096, 4096, 131072, 4096, 20) < 2 << 30
    # what the pieces leave is bounded, however many tokens there are
    assert f(P, 64, P, 64, 1 << 20, 131072, 64, 32) < 2 << 30
    assert b(P, 8, P, 8, 4, 10, 8) == L.pp_stage_head_backward_workspace(P, 8, P, 8, 4, 10, 8)


def _list(*entries):
    t = (S._Tensors * len(entries))()
    for e, given in zip(t, entries):
        for k, v in {**dict(p=P, g=P, copy=None, n=64, at=0, decay=0.0, p_float=1, g_float=1), **given}.items():
            setattr(e, k, v)
    return t


def adamw(*entries, count=None, lst=True, m=P, v=P, me=None, ve=None, held=128, step=P, lr_at=None, lr=1e-3, b1=0.9, b2=0.99,
          eps=1e-8, norm=None, wide=None, most=1.0, ws=P, n=256):
    t = _list(*(entries or ({}, {"at": 64})))
    return L.pp_stage_adamw(ctypes.addressof(t) if lst else None, len(t) if count is None else count, m, v, me, ve, held, step,
                            lr_at, lr, b1, b2, eps, norm, wide, most, 0, 0, ws, n, None)


def test_step():
    nan = float("nan")
    for bad in (dict(lst=False), dict(count=-1), dict(m=None), dict(v=None), dict(me=P), dict(ve=P), dict(held=-64), dict(held=100),
                dict(held=64), dict(m=P + 16), dict(v=P + 4), dict(step=None), dict(step=P + 4), dict(lr_at=P + 2), dict(lr=nan),
                dict(lr=float("inf")), dict(b1=1.0), dict(b1=-0.1), dict(b2=nan), dict(eps=-1.0), dict(eps=nan), dict(norm=P + 1),
                dict(norm=P, most=0.0), dict(norm=P, wide=P + 4), dict(norm=P, most=nan), dict(ws=None), dict(ws=P + 16), dict(n=8)):
        assert adamw(**bad) == B.PP_ERR_ARG, bad
    for bad in (dict(n=-1), dict(p=None), dict(g=None), dict(p=P + 2), dict(g=P + 2), dict(p_float=0, p=P + 1), dict(g_float=2),
                dict(p_float=255), dict(copy=P + 1), dict(copy=P, p_float=0), dict(at=-64), dict(at=32), dict(at=128), dict(n=129),
                dict(decay=nan)):
        assert adamw(bad) == B.PP_ERR_ARG, bad
    assert adamw({"n": (1 << 38) + 1}, held=1 << 38) == B.PP_ERR_SIZE
    assert adamw(held=(1 << 38) + 64) == B.PP_ERR_SIZE


@pytest.mark.parametrize("eps", [1e-300, 1e-46, 1e-40, 2.0 ** -126 * (1 - 2 ** -53), 3.1e38])
def test_an_eps_that_is_no_normal_number(eps):
    """The step's reciprocal takes what is below 2^-126 as 0: with both moments 0 it would make NaN of 0 / eps."""
    assert adamw(eps=eps) == B.PP_ERR_ARG


def test_norm_and_moments():
    def norm(*entries, count=None, out=P, wide=None, ws=P, n=1 << 20):
        t = _list(*entries)
        return L.pp_stage_grad_norm(ctypes.addressof(t), len(t) if count is None else count, out, wide, ws, n, None)
    for bad in (dict(out=None), dict(out=P + 2), dict(wide=P + 4), dict(count=-1), dict(ws=None), dict(ws=P + 8), dict(n=4)):
        assert norm({}, **bad) == B.PP_ERR_ARG, bad
    for bad in (dict(n=-1), dict(g=None), dict(g=P + 2), dict(g_float=7)):
        assert norm(bad) == B.PP_ERR_ARG, bad
    assert norm({"n": (1 << 38) + 1}) == B.PP_ERR_SIZE
    t = _list({}, {"n": 1 << 30}, {"n": 0, "g": None})
    assert 0 < L.pp_stage_grad_norm_workspace(ctypes.addressof(t), 3) < 1 << 16

    def moments(m=P, v=P, me=P, ve=P, held=64, mv=P, vv=P):
        return L.pp_stage_adamw_moments(m, v, me, ve, held, mv, vv, None)
    for bad in (dict(m=None), dict(v=None), dict(me=None), dict(ve=None), dict(mv=None), dict(vv=P + 8), dict(m=P + 4),
                dict(held=63), dict(held=-64)):
        assert moments(**bad) == B.PP_ERR_ARG, bad
    assert moments(held=0, m=None) == B.PP_OK


def test_host_tensors_are_refused():
    x, t, f = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        S.score_forward(x, x, t)
    with pytest.raises(ValueError, match="CUDA"):
        S.score_backward(x, x, t, f, f)
    with pytest.raises(ValueError, match="CUDA"):
        S.grad_norm([f])
    with pytest.raises(ValueError, match="CUDA"):
        S.AdamW([f])
    with pytest.raises(TypeError, match="list"):
        S.AdamW(f)
    with pytest.raises(ValueError, match="at least one"):
        S.AdamW([])
