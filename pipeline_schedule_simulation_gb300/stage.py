"""The operators of one pipeline stage (include/ppstage.h): argument checks
and marshalling only, every step of the computation runs in the library.

    head_forward, head_backward   the last stage's loss over a large vocabulary
                                  and its gradients, without kept logits
    pack, unpack, weight_grad     activation checkpoints in 8 bits and the
                                  weight gradient (the W op) taken from them
    join_forward, join_backward   the norm after a block, its gate, the residual
                                  scale and sum, the norm before the next block

All tensors are CUDA tensors on one device; matrices have contiguous rows and
any row stride.  Calls are asynchronous on ``stream`` (default: the current
stream of the tensors' device).  Outputs and scratch memory that are not given
are allocated for that stream, so nothing else may reuse them before the call
has run; a caller that passes ``stream`` still orders its inputs before it.
``workspace`` may be any CUDA uint8 tensor that starts on 256 bytes, of at least
the bytes that the matching *_workspace function gives.  The forward and the
backward pass are calls of their own: nothing is recorded for autograd, and
results carry no gradient, whatever the inputs say.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import LIB, PP_OK, PPSchedError, _arg, _check, _reach

EXPORTS = ("pp_stage_head_forward_workspace", "pp_stage_head_forward", "pp_stage_head_backward_workspace",
           "pp_stage_head_backward", "pp_stage_pack", "pp_stage_unpack", "pp_stage_weight_grad_workspace",
           "pp_stage_weight_grad", "pp_stage_join_forward", "pp_stage_join_backward_workspace",
           "pp_stage_join_backward", "pp_stage_wait_failure")

#: Columns of a checkpoint that share one exponent.
BLOCK = 64
#: Exponent of a checkpoint's block that holds an infinity or a NaN.
NONFINITE = -128


def _declare(lib):
    vp, i32, i64, f32, size = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    m = [vp, i64]  # a matrix: pointer and row stride
    lib.pp_stage_head_forward_workspace.argtypes = [*m, *m, i64, i64, i64]
    lib.pp_stage_head_forward.argtypes = [*m, *m, vp, i64, i64, i64, vp, vp, vp, size, vp]
    lib.pp_stage_head_backward_workspace.argtypes = [*m, *m, i64, i64, i64]
    lib.pp_stage_head_backward.argtypes = [*m, *m, vp, vp, vp, f32, i64, i64, i64, *m, *m, i32, i32, vp, size, vp]
    lib.pp_stage_pack.argtypes = [*m, i64, i64, *m, *m, vp]
    lib.pp_stage_unpack.argtypes = [*m, *m, i64, i64, *m, vp]
    lib.pp_stage_weight_grad_workspace.argtypes = [*m, i64, i64, i64]
    lib.pp_stage_weight_grad.argtypes = [*m, *m, *m, i64, i64, i64, *m, *m, vp, size, vp]
    lib.pp_stage_join_forward.argtypes = [*m, *m, vp, vp, *m, i64, f32, f32, i64, i64, *m, *m, vp, vp,
                                          *m, *m, *m, *m, vp]
    lib.pp_stage_join_backward_workspace.argtypes = [i64, i64, i64]
    lib.pp_stage_join_backward.argtypes = [*m, *m, *m, *m, *m, *m, *m, *m, vp, vp, vp, vp, *m, i64, f32, i64, i64,
                                           *m, *m, vp, vp, *m, vp, size, vp]
    lib.pp_stage_wait_failure.argtypes = [vp]
    for name in EXPORTS:
        getattr(lib, name).restype = size if name.endswith("_workspace") else i32


_declare(LIB)


_BF16, _F32, _I64, _I8, _U8 = torch.bfloat16, torch.float32, torch.int64, torch.int8, torch.uint8
_Tensor, _empty = torch.Tensor, torch.empty
# the handle of a device's current stream and the current device, without the objects around them: a small call
# is mostly its host path
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


class Packed:
    """An activation checkpoint: ``q`` int8 [T, H] and ``e`` int8 [T, ceil(H / 64)]; an element stands for
    q * 2**e of its row and block of 64 columns (NaN where e is NONFINITE)."""

    __slots__ = ("q", "e")

    def __init__(self, q, e):
        dev = _device(q)
        _, _, T, H = _matrix(q, "q", _I8, dev)
        _matrix(e, "e", _I8, dev, T, (H + BLOCK - 1) // BLOCK)
        self.q, self.e = q, e

    @property
    def shape(self):
        return self.q.shape

    @property
    def nbytes(self):
        """Bytes that a held microbatch takes, padding between rows included."""
        return sum(_reach(t.shape, t.stride()) for t in (self.q, self.e))


def _device(t):
    """CUDA device index of the call's first tensor, -1 if it has none (its check then says what is wrong)."""
    return t.get_device() if isinstance(t, _Tensor) else -1


def _matrix(t, name, dtype, dev, rows=None, cols=None):
    """(pointer, row stride, rows, columns) of a matrix with contiguous rows on CUDA device `dev`; anything else is
    refused.  A single row's stride is its length, whatever the tensor says."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev >= 0 and t.dim() == 2:
        (r, c), (sr, sc) = t.shape, t.stride()
        if (r == rows or rows is None) and (c == cols or cols is None):
            if r <= 1:
                sr = c
            if (sc == 1 or c <= 1) and sr >= c:
                return t.data_ptr(), sr, r, c
    _refuse(t, name, dtype, dev, rows, cols)


def _refuse(t, name, dtype, dev, rows, cols):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix, got {t.dim()} dimensions")
    r, c = t.shape
    want = (r if rows is None else rows, c if cols is None else cols)
    if (r, c) != want:
        raise ValueError(f"{name}: expected shape {want}, got {(r, c)}")
    _arg(t, name, dtype, torch.device("cuda", dev) if dev >= 0 else None, 0)
    if c > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: expected contiguous rows, got a column stride of {t.stride(1)}")
    raise ValueError(f"{name}: rows overlap (stride {t.stride(0)}, {c} columns)")


def _vector(t, name, dtype, dev, n):
    """Pointer of a contiguous vector of n elements on CUDA device `dev`."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == 1 and t.shape[0] == n:
        if n <= 1 or t.stride(0) == 1:
            return t.data_ptr()
        raise ValueError(f"{name}: expected a contiguous vector")
    _arg(t, name, dtype, torch.device("cuda", dev), 0)
    raise ValueError(f"{name}: expected shape ({n},), got {tuple(t.shape)}")


def _elsewhere(dev, stream):
    """None where the call can be made as it stands: on the current stream of the current device.  Otherwise the
    context to make it in, so that what it allocates belongs to its stream."""
    if dev < 0:
        return None
    if stream is None:
        return None if _current_device() == dev else torch.cuda.device(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream: on {stream.device}, the tensors are on cuda:{dev}")
    return torch.cuda.stream(stream)


def _scratch(workspace, need, device, dev):
    """(tensor, pointer, bytes) of the scratch memory: the caller's, or new memory of the current stream."""
    if workspace is None:
        workspace = _empty(need or 1, dtype=_U8, device=device)
    else:
        _arg(workspace, "workspace", _U8, device, need)
        if not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError(f"workspace: needs {need} contiguous bytes, got {workspace.numel()}")
    return workspace, workspace.data_ptr(), workspace.numel()


def _out_matrix(out, name, rows, cols, dtype, device, dev):
    t = out.get(name)
    if t is None:
        t = out[name] = _empty((rows, cols), dtype=dtype, device=device)
        return t.data_ptr(), cols
    return _matrix(t, name, dtype, dev, rows, cols)[:2]


def _out_vector(out, name, n, dtype, device, dev):
    t = out.get(name)
    if t is None:
        t = out[name] = _empty(n, dtype=dtype, device=device)
        return t.data_ptr()
    return _vector(t, name, dtype, dev, n)


def _head_inputs(x, w, target, dev):
    px, sx, T, H = _matrix(x, "x", _BF16, dev)
    pw, sw, V, _ = _matrix(w, "w", _BF16, dev, None, H)
    return px, sx, pw, sw, T, V, H, _vector(target, "target", _I64, dev, T)


def head_forward_workspace(x, w):
    """Bytes of scratch memory that head_forward needs for these matrices."""
    px, sx, T, H = _matrix(x, "x", _BF16, _device(x))
    pw, sw, V, _ = _matrix(w, "w", _BF16, _device(x), None, H)
    return LIB.pp_stage_head_forward_workspace(px, sx, pw, sw, T, V, H)


def head_backward_workspace(x, w):
    """Bytes of scratch memory that head_backward needs for these matrices."""
    px, sx, T, H = _matrix(x, "x", _BF16, _device(x))
    pw, sw, V, _ = _matrix(w, "w", _BF16, _device(x), None, H)
    return LIB.pp_stage_head_backward_workspace(px, sx, pw, sw, T, V, H)


def head_forward(x, w, target, *, out=None, workspace=None, stream=None):
    """Softmax cross entropy of the logits x w^T without keeping them (the last stage's F).

    x [T, H], w [V, H] bf16; target [T] int64, a token whose target is outside 0..V-1 is left out.
    Returns loss [T] (0 where left out) and lse [T], the log-sum-exp that head_backward takes; float."""
    dev = _device(x)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return head_forward(x, w, target, out=out, workspace=workspace)
    px, sx, pw, sw, T, V, H, pt = _head_inputs(x, w, target, dev)
    out, device = dict(out) if out else {}, x.device
    loss = _out_vector(out, "loss", T, _F32, device, dev)
    lse = _out_vector(out, "lse", T, _F32, device, dev)
    need = LIB.pp_stage_head_forward_workspace(px, sx, pw, sw, T, V, H)
    _keep, ws, n = _scratch(workspace, need, device, dev)
    rc = LIB.pp_stage_head_forward(px, sx, pw, sw, pt, T, V, H, loss, lse, ws, n, _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_head_forward")
    return out


def head_backward(x, w, target, lse, *, scale=1.0, weight=None, outputs=("dx", "dw"), add=False, out=None,
                  workspace=None, stream=None):
    """Gradients of sum_t scale * weight[t] * loss[t] (weight: float [T], default 1).

    Returns dx [T, H] bf16 (the B op) and dw [V, H] (the W op), or the one named in `outputs`.  dw is bf16 unless
    out["dw"] is a float matrix; add=True then adds to what that holds (the microbatches' running sum)."""
    dev = _device(x)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return head_backward(x, w, target, lse, scale=scale, weight=weight, outputs=outputs, add=add, out=out,
                                 workspace=workspace)
    px, sx, pw, sw, T, V, H, pt = _head_inputs(x, w, target, dev)
    pl = _vector(lse, "lse", _F32, dev, T)
    pg = None if weight is None else _vector(weight, "weight", _F32, dev, T)
    if not outputs or any(o not in ("dx", "dw") for o in outputs):
        raise ValueError(f"outputs: expected some of 'dx' and 'dw', got {outputs!r}")
    out, device = dict(out) if out else {}, x.device
    dx = _out_matrix(out, "dx", T, H, _BF16, device, dev) if "dx" in outputs else (None, 0)
    dw, wide = (None, 0), False
    if "dw" in outputs:
        wide = isinstance(out.get("dw"), _Tensor) and out["dw"].dtype is _F32
        if add and not wide:
            raise ValueError("add: needs a float out['dw'] to add to")
        dw = _out_matrix(out, "dw", V, H, _F32 if wide else _BF16, device, dev)
    need = LIB.pp_stage_head_backward_workspace(px, sx, pw, sw, T, V, H)
    _keep, ws, n = _scratch(workspace, need, device, dev)
    rc = LIB.pp_stage_head_backward(px, sx, pw, sw, pt, pl, pg, scale, T, V, H, *dx, *dw, wide, bool(add) and wide, ws, n,
                                    _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_head_backward")
    return out


def _packed(p, name, dev, rows=None, cols=None):
    """(q, stride, e, stride, rows, columns) of a checkpoint on CUDA device `dev`."""
    if not isinstance(p, Packed):
        raise TypeError(f"{name}: expected a Packed checkpoint, got {type(p).__name__}")
    q, sq, T, H = _matrix(p.q, name, _I8, dev, rows, cols)
    return q, sq, *_matrix(p.e, name + ".e", _I8, dev, T)[:2], T, H


def _new_packed(T, H, device):
    # rows padded to 16 bytes, so that every reader takes its wide path
    p = Packed.__new__(Packed)
    ld = (H + 15) // 16 * 16
    q = _empty((T, ld), dtype=_I8, device=device)
    p.q = q if ld == H else q[:, :H]
    p.e = _empty((T, (H + BLOCK - 1) // BLOCK), dtype=_I8, device=device)
    return p


def pack(x, *, out=None, stream=None):
    """The 8-bit checkpoint (a Packed) of an activation x [T, H] bf16."""
    dev = _device(x)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return pack(x, out=out)
    px, sx, T, H = _matrix(x, "x", _BF16, dev)
    p = _new_packed(T, H, x.device) if out is None else out
    rc = LIB.pp_stage_pack(px, sx, T, H, *_packed(p, "out", dev, T, H)[:4], _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_pack")
    return p


def unpack(packed, *, out=None, stream=None):
    """What a checkpoint stands for, bf16 [T, H] (exactly: the steps are powers of two)."""
    dev = _device(packed.q if isinstance(packed, Packed) else None)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return unpack(packed, out=out)
    q, sq, e, se, T, H = _packed(packed, "packed", dev)
    if out is None:
        out = _empty((T, H), dtype=_BF16, device=packed.q.device)
        px, sx = out.data_ptr(), H
    else:
        px, sx, _, _ = _matrix(out, "out", _BF16, dev, T, H)
    rc = LIB.pp_stage_unpack(q, sq, e, se, T, H, px, sx, _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_unpack")
    return out


def weight_grad_workspace(dy, packed):
    """Bytes of scratch memory that weight_grad needs."""
    dev = _device(dy)
    pd, sd, T, N = _matrix(dy, "dy", _BF16, dev)
    return LIB.pp_stage_weight_grad_workspace(pd, sd, T, N, _packed(packed, "packed", dev, T)[5])


def weight_grad(dy, packed, *, add=None, out=None, workspace=None, stream=None):
    """The W op of a linear layer whose input [T, H] was kept: float [N, H] = add + dy^T value(packed).

    dy [T, N] bf16.  `add` (float [N, H]) is the running sum of the microbatches; out=add adds in place."""
    dev = _device(dy)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return weight_grad(dy, packed, add=add, out=out, workspace=workspace)
    pd, sd, T, N = _matrix(dy, "dy", _BF16, dev)
    if isinstance(packed, Packed) and packed.q.shape[0] != T:
        raise ValueError(f"packed: expected {T} rows, got {packed.q.shape[0]}")
    q, sq, e, se, _, H = _packed(packed, "packed", dev)
    pa, sa = (None, 0) if add is None else _matrix(add, "add", _F32, dev, N, H)[:2]
    device = dy.device
    if out is None:
        out = _empty((N, H), dtype=_F32, device=device)
        po, so = out.data_ptr(), H
    else:
        po, so, _, _ = _matrix(out, "out", _F32, dev, N, H)
    need = LIB.pp_stage_weight_grad_workspace(pd, sd, T, N, H)
    _keep, ws, n = _scratch(workspace, need, device, dev)
    rc = LIB.pp_stage_weight_grad(pd, sd, q, sq, e, se, T, N, H, pa, sa, po, so, ws, n, _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_weight_grad")
    return out


def _gate(gate, rows_per_gate, T, H, dev):
    """(pointer, stride, tokens to a gate row or 0) of the gate."""
    rows = int(rows_per_gate or 0)
    if gate is None:
        if rows:
            raise ValueError("rows_per_gate: given without a gate")
        return None, 0, 0
    if rows < 0:
        raise ValueError("rows_per_gate must not be negative")
    p, s, have, _ = _matrix(gate, "gate", _BF16, dev, None, H)
    need = (T + rows - 1) // rows if rows else 1
    if have < need or have < 1 or (rows == 0 and have != 1):
        raise ValueError(f"gate: {T} tokens with {rows or T} to a gate take {need} rows, got {have}")
    return p, s, rows


def join_forward(x, f, w_post, w_pre, gate=None, *, rows_per_gate=0, alpha=1.0, eps=1e-6, keep=False, out=None,
                 stream=None):
    """A block's output f joins the residual stream x: y = alpha x + gate * w_post * f / rms(f), and the next
    block's input h = w_pre * y / rms(y).

    x, f [T, H], w_post, w_pre [H], gate [G, H] bf16; row t uses gate[t // rows_per_gate] (0: one gate).
    Returns y, h (bf16), rstd_post, rstd_pre (float [T]); keep=True adds kept_y and kept_f, the checkpoints that
    join_backward reads."""
    dev = _device(x)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return join_forward(x, f, w_post, w_pre, gate, rows_per_gate=rows_per_gate, alpha=alpha, eps=eps, keep=keep,
                                out=out)
    px, sx, T, H = _matrix(x, "x", _BF16, dev)
    pf, sf, _, _ = _matrix(f, "f", _BF16, dev, T, H)
    w1, w2 = _vector(w_post, "w_post", _BF16, dev, H), _vector(w_pre, "w_pre", _BF16, dev, H)
    pg, sg, rows = _gate(gate, rows_per_gate, T, H, dev)
    out, device = dict(out) if out else {}, x.device
    py, sy = _out_matrix(out, "y", T, H, _BF16, device, dev)
    ph, sh = _out_matrix(out, "h", T, H, _BF16, device, dev)
    r1 = _out_vector(out, "rstd_post", T, _F32, device, dev)
    r2 = _out_vector(out, "rstd_pre", T, _F32, device, dev)
    kept = (None, 0, None, 0) * 2
    if keep:
        for k in ("kept_y", "kept_f"):
            if out.get(k) is None:
                out[k] = _new_packed(T, H, device)
        kept = (*_packed(out["kept_y"], "kept_y", dev, T, H)[:4], *_packed(out["kept_f"], "kept_f", dev, T, H)[:4])
    rc = LIB.pp_stage_join_forward(px, sx, pf, sf, w1, w2, pg, sg, rows, alpha, eps, T, H, py, sy, ph, sh, r1, r2, *kept,
                                   _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_join_forward")
    return out


def join_backward_workspace(T, H, rows_per_gate=0):
    """Bytes of scratch memory that join_backward needs."""
    return LIB.pp_stage_join_backward_workspace(T, H, rows_per_gate)


def join_backward(dh, dy, y, f, rstd_post, rstd_pre, w_post, w_pre, gate=None, *, rows_per_gate=0, alpha=1.0,
                  out=None, workspace=None, stream=None):
    """Gradients of the join, from dh (of h) and dy (what reaches y by other paths; None: nothing does).

    y and f are both bf16 [T, H] or both Packed checkpoints.  Returns dx, df (bf16), dw_post, dw_pre (float [H])
    and, with a gate, dgate (float [G, H])."""
    dev = _device(dh)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return join_backward(dh, dy, y, f, rstd_post, rstd_pre, w_post, w_pre, gate, rows_per_gate=rows_per_gate,
                                 alpha=alpha, out=out, workspace=workspace)
    ph, sh, T, H = _matrix(dh, "dh", _BF16, dev)
    pd, sd = (None, 0) if dy is None else _matrix(dy, "dy", _BF16, dev, T, H)[:2]
    if isinstance(y, Packed) != isinstance(f, Packed):
        raise TypeError("y and f: expected two checkpoints or two tensors")
    if isinstance(y, Packed):
        saved = (None, 0, None, 0, *_packed(y, "y", dev, T, H)[:4], *_packed(f, "f", dev, T, H)[:4])
    else:
        saved = (*_matrix(y, "y", _BF16, dev, T, H)[:2], *_matrix(f, "f", _BF16, dev, T, H)[:2],
                 None, 0, None, 0, None, 0, None, 0)
    r1, r2 = _vector(rstd_post, "rstd_post", _F32, dev, T), _vector(rstd_pre, "rstd_pre", _F32, dev, T)
    w1, w2 = _vector(w_post, "w_post", _BF16, dev, H), _vector(w_pre, "w_pre", _BF16, dev, H)
    pg, sg, rows = _gate(gate, rows_per_gate, T, H, dev)
    out, device = dict(out) if out else {}, dh.device
    dx, sdx = _out_matrix(out, "dx", T, H, _BF16, device, dev)
    df, sdf = _out_matrix(out, "df", T, H, _BF16, device, dev)
    d1 = _out_vector(out, "dw_post", H, _F32, device, dev)
    d2 = _out_vector(out, "dw_pre", H, _F32, device, dev)
    dg, sdg = None, 0
    if gate is not None:
        G = gate.shape[0]
        dg, sdg = _out_matrix(out, "dgate", G, H, _F32, device, dev)
        used = (T + rows - 1) // rows if rows else min(T, 1)
        if used < G:  # gates that no token uses
            out["dgate"][used:].zero_()
    need = LIB.pp_stage_join_backward_workspace(T, H, rows)
    _keep, ws, n = _scratch(workspace, need, device, dev)
    rc = LIB.pp_stage_join_backward(ph, sh, pd, sd, *saved, r1, r2, w1, w2, pg, sg, rows, alpha, T, H, dx, sdx, df, sdf,
                                    d1, d2, dg, sdg, ws, n, _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_join_backward")
    return out


def wait_failure():
    """A record of a wait that ran out on the current device since the previous call (0: none); synchronizes the device.

    Calls return before their kernels have run, so they cannot tell: a block whose wait for its own copies or matrix
    instructions runs out gives up, and the call's outputs are wrong.  Ask after a step, before its results are used."""
    word = ctypes.c_uint64()
    _check(LIB.pp_stage_wait_failure(ctypes.byref(word)), "pp_stage_wait_failure")
    return word.value
