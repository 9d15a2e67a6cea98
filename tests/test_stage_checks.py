"""The pipeline-stage operators without a GPU: every declared entry point is
exported and bound, and argument errors are answered on the host before any
CUDA call."""
import ctypes
import os
import re

import pytest
import torch

from conftest import ROOT
from pipeline_schedule_simulation_gb300 import binding as B
from pipeline_schedule_simulation_gb300 import stage as S

L = B.LIB
P = 1 << 20  # stands for an aligned pointer; never followed


def _declared():
    src = open(os.path.join(ROOT, "include", "ppstage.h")).read()
    return sorted(set(re.findall(r"\b(pp_stage_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S))))


def test_every_entry_point_is_declared_exported_and_bound():
    assert sorted(S.EXPORTS) == _declared()
    for name in S.EXPORTS:
        f = getattr(L, name)
        assert f.argtypes is not None and f.restype in (ctypes.c_int, ctypes.c_size_t), name


def head_f(T=4, V=10, H=8, x=P, sx=8, w=P, sw=8, t=P, loss=P, lse=P, ws=P, n=1 << 40):
    return L.pp_stage_head_forward(x, sx, w, sw, t, T, V, H, loss, lse, ws, n, None)


def head_b(T=4, V=10, H=8, x=P, sx=8, w=P, sw=8, t=P, lse=P, dx=P, sdx=8, dw=P, sdw=8, wide=0, add=0, ws=P, n=1 << 40):
    return L.pp_stage_head_backward(x, sx, w, sw, t, lse, None, 1.0, T, V, H, dx, sdx, dw, sdw, wide, add, ws, n, None)


@pytest.mark.parametrize("call", [head_f, head_b])
def test_head_refusals(call):
    for bad in (dict(T=-1), dict(V=0), dict(H=0), dict(x=None), dict(w=None), dict(t=None), dict(x=P + 1), dict(w=P + 1),
                dict(t=P + 4), dict(sx=7), dict(sw=7), dict(ws=None), dict(ws=P + 16), dict(n=8)):
        assert call(**bad) == B.PP_ERR_ARG, bad
    for big in (dict(T=(1 << 24) + 1), dict(V=(1 << 24) + 1), dict(H=(1 << 16) + 1)):
        assert call(**big) == B.PP_ERR_SIZE, big


def test_head_output_refusals():
    assert head_f(loss=None, lse=None) == B.PP_ERR_ARG
    assert head_f(loss=P + 2) == B.PP_ERR_ARG
    assert head_b(dx=None, dw=None) == B.PP_ERR_ARG
    assert head_b(sdx=7) == B.PP_ERR_ARG
    assert head_b(sdw=7) == B.PP_ERR_ARG
    assert head_b(add=1) == B.PP_ERR_ARG            # a sum is held in 32 bits
    assert head_b(wide=1, dw=P + 2) == B.PP_ERR_ARG
    assert head_b(lse=None) == B.PP_ERR_ARG
    assert head_f(T=0, x=None, t=None, ws=None, n=0) == B.PP_OK  # nothing to do


def test_kept_refusals():
    def pack(T=4, H=100, x=P, sx=100, q=P, sq=100, e=P, se=2):
        return L.pp_stage_pack(x, sx, T, H, q, sq, e, se, None)

    def unpack(T=4, H=100, x=P, sx=100, q=P, sq=100, e=P, se=2):
        return L.pp_stage_unpack(q, sq, e, se, T, H, x, sx, None)

    for call in (pack, unpack):
        for bad in (dict(T=-1), dict(H=0), dict(x=None), dict(x=P + 1), dict(q=None), dict(e=None), dict(sx=99),
                    dict(sq=99), dict(se=1)):
            assert call(**bad) == B.PP_ERR_ARG, bad
        assert call(H=(1 << 16) + 1) == B.PP_ERR_SIZE
        assert call(T=(1 << 24) + 1) == B.PP_ERR_SIZE
        assert call(T=0, x=None, q=None, e=None) == B.PP_OK

    def wgrad(T=4, N=6, H=100, dy=P, sdy=6, q=P, sq=100, e=P, se=2, add=None, sadd=0, dw=P, sdw=100, ws=P, n=1 << 40):
        return L.pp_stage_weight_grad(dy, sdy, q, sq, e, se, T, N, H, add, sadd, dw, sdw, ws, n, None)
    for bad in (dict(T=-1), dict(N=0), dict(H=0), dict(dy=None), dict(sdy=5), dict(q=None), dict(se=1), dict(dw=None),
                dict(dw=P + 2), dict(sdw=99), dict(add=P, sadd=99), dict(add=P + 2, sadd=100), dict(add=P, sadd=104),
                dict(ws=None), dict(ws=P + 16), dict(n=8)):
        assert wgrad(**bad) == B.PP_ERR_ARG, bad
    assert wgrad(N=(1 << 24) + 1) == B.PP_ERR_SIZE


def test_join_refusals():
    def fw(T=4, H=100, x=P, sx=100, f=P, w1=P, w2=P, g=P, sg=100, rows=2, eps=0.0, y=P, h=P, sh=100, r1=P, r2=P,
           yq=None, syq=0, ye=None, sye=0, fq=None, sfq=0, fe=None, sfe=0):
        return L.pp_stage_join_forward(x, sx, f, 100, w1, w2, g, sg, rows, 1.0, eps, T, H, y, 100, h, sh, r1, r2,
                                       yq, syq, ye, sye, fq, sfq, fe, sfe, None)
    kept = dict(yq=P, syq=100, ye=P, sye=2, fq=P, sfq=100, fe=P, sfe=2)
    for bad in (dict(T=-1), dict(H=0), dict(x=None), dict(x=P + 1), dict(sx=99), dict(f=None), dict(w1=None),
                dict(w2=P + 1), dict(sg=99), dict(eps=-1.0), dict(eps=float("nan")), dict(y=None), dict(sh=99),
                dict(r1=None), dict(r2=P + 2), dict(yq=P), {**kept, "fe": None}, {**kept, "sye": 1}):
        assert fw(**bad) == B.PP_ERR_ARG, bad
    assert fw(H=16385, sx=20000) == B.PP_ERR_SIZE

    def bw(T=4, H=100, dh=P, y=P, f=P, yq=None, r1=P, w1=P, g=P, dg=P, sdg=100, dx=P, df=P, d1=P, d2=P, ws=P, n=1 << 40,
           **k):
        return L.pp_stage_join_backward(dh, 100, None, 0, y, 100, f, 100, yq, 100, k.get("ye"), 2, k.get("fq"), 100,
                                        k.get("fe"), 2, r1, P, w1, P, g, 100, 2, 1.0, T, H, dx, 100, df, 100, d1, d2, dg,
                                        sdg, ws, n, None)
    for bad in (dict(T=-1), dict(H=0), dict(dh=None), dict(y=None), dict(f=None), dict(yq=P),
                dict(y=None, f=None, yq=P, ye=P, fq=P), dict(r1=None), dict(w1=None), dict(dg=None), dict(g=None),
                dict(sdg=99), dict(dx=None), dict(df=P + 1), dict(d1=None), dict(d2=P + 2), dict(ws=None), dict(n=8),
                dict(ws=P + 8)):
        assert bw(**bad) == B.PP_ERR_ARG, bad
    assert bw(H=16385) == B.PP_ERR_SIZE


def test_workspaces_of_nothing():
    assert L.pp_stage_head_forward_workspace(None, 0, P, 8, 0, 10, 8) == 0
    assert L.pp_stage_weight_grad_workspace(None, 0, 0, 4, 4) == 0
    assert L.pp_stage_join_backward_workspace(0, 100, 0) == 0
    assert L.pp_stage_join_backward_workspace(100, 100, 0) > 0


def test_host_tensors_are_refused():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="x: expected a tensor on a CUDA device"):
        S.head_forward(x, x, t)
    with pytest.raises(ValueError, match="CUDA"):
        S.pack(x)
    with pytest.raises(ValueError, match="CUDA"):
        S.Packed(x.to(torch.int8), x.to(torch.int8))
    with pytest.raises(ValueError, match="CUDA"):
        S.join_forward(x, x, x[0], x[0])
    with pytest.raises(TypeError, match="torch.Tensor"):
        S.pack([1, 2])
    with pytest.raises(ValueError, match="matrix"):
        S.pack(x[0])
