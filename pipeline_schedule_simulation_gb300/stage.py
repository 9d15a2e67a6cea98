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
``workspace`` may be any CUDA uint8 tensor of at least the bytes that the
matching *_workspace function gives.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import LIB, PPSchedError, _arg, _check, _ptr, _reach, _stream  # noqa: F401

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


class Packed:
    """An activation checkpoint: ``q`` int8 [T, H] and ``e`` int8 [T, ceil(H / 64)]; an element stands for
    q * 2**e of its row and block of 64 columns (NaN where e is NONFINITE)."""

    __slots__ = ("q", "e")

    def __init__(self, q, e):
        T, H = _matrix(q, "q", torch.int8, None)
        _matrix(e, "e", torch.int8, q.device, (T, -(-H // BLOCK)))
        self.q, self.e = q, e

    @property
    def shape(self):
        return self.q.shape

    @property
    def nbytes(self):
        """Bytes that a held microbatch takes, padding between rows included."""
        return sum(_reach(t.shape, t.stride()) for t in (self.q, self.e))


def _matrix(t, name, dtype, device, shape=None):
    """Refuse anything but a CUDA matrix of this dtype with contiguous rows; returns its shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix, got {t.dim()} dimensions")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    _arg(t, name, dtype, device, 0)
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: expected contiguous rows, got a column stride of {t.stride(1)}")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name}: rows overlap (stride {t.stride(0)}, {cols} columns)")
    return rows, cols


def _vector(t, name, dtype, device, n):
    _arg(t, name, dtype, device, 0)
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name}: expected shape ({n},), got {tuple(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name}: expected a contiguous vector")
    return t


def _m(t):
    """Pointer and row stride of a matrix (a single row's stride is its length, whatever the tensor says)."""
    if t is None:
        return None, 0
    return _ptr(t), (t.stride(0) if t.shape[0] > 1 else t.shape[1])


class _On:
    """The stream of a call: allocations made through it belong to it."""

    def __init__(self, device, stream):
        self.device = device
        self.stream = torch.cuda.current_stream(device) if stream is None else stream
        if self.stream.device != device:
            raise ValueError(f"stream: on {self.stream.device}, the tensors are on {device}")

    def __enter__(self):
        self._ctx = torch.cuda.stream(self.stream)
        self._ctx.__enter__()
        return self

    def __exit__(self, *a):
        return self._ctx.__exit__(*a)

    @property
    def handle(self):
        return ctypes.c_void_p(self.stream.cuda_stream)

    def scratch(self, workspace, need):
        if workspace is None:
            return torch.empty(max(need, 1), dtype=torch.uint8, device=self.device)
        _arg(workspace, "workspace", torch.uint8, self.device, need)
        if not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError(f"workspace: needs {need} contiguous bytes, got {workspace.numel()}")
        return workspace


def _out(out, name, shape, dtype, device):
    t = out.get(name)
    if t is None:
        t = out[name] = torch.empty(shape, dtype=dtype, device=device)
    elif len(shape) == 2:
        _matrix(t, name, dtype, device, shape)
    else:
        _vector(t, name, dtype, device, shape[0])
    return t


_BF16, _F32, _I64 = torch.bfloat16, torch.float32, torch.int64


def _head_inputs(x, w, target):
    T, H = _matrix(x, "x", _BF16, None)
    V, _ = _matrix(w, "w", _BF16, x.device, (w.shape[0] if isinstance(w, torch.Tensor) and w.dim() == 2 else 0, H))
    _vector(target, "target", _I64, x.device, T)
    return T, V, H


def head_forward_workspace(x, w):
    """Bytes of scratch memory that head_forward needs for these matrices."""
    return LIB.pp_stage_head_forward_workspace(*_m(x), *_m(w), x.shape[0], w.shape[0], x.shape[1])


def head_backward_workspace(x, w):
    """Bytes of scratch memory that head_backward needs for these matrices."""
    return LIB.pp_stage_head_backward_workspace(*_m(x), *_m(w), x.shape[0], w.shape[0], x.shape[1])


def head_forward(x, w, target, *, out=None, workspace=None, stream=None):
    """Softmax cross entropy of the logits x w^T without keeping them (the last stage's F).

    x [T, H], w [V, H] bf16; target [T] int64, a token whose target is outside 0..V-1 is left out.
    Returns loss [T] (0 where left out) and lse [T], the log-sum-exp that head_backward takes; float."""
    T, V, H = _head_inputs(x, w, target)
    with _On(x.device, stream) as on:
        out = dict(out or {})
        loss = _out(out, "loss", (T,), _F32, x.device)
        lse = _out(out, "lse", (T,), _F32, x.device)
        ws = on.scratch(workspace, head_forward_workspace(x, w))
        _check(LIB.pp_stage_head_forward(*_m(x), *_m(w), _ptr(target), T, V, H, _ptr(loss), _ptr(lse), _ptr(ws),
                                         ws.numel(), on.handle), "pp_stage_head_forward")
    return out


def head_backward(x, w, target, lse, *, scale=1.0, weight=None, outputs=("dx", "dw"), add=False, out=None,
                  workspace=None, stream=None):
    """Gradients of sum_t scale * weight[t] * loss[t] (weight: float [T], default 1).

    Returns dx [T, H] bf16 (the B op) and dw [V, H] (the W op), or the one named in `outputs`.  dw is bf16 unless
    out["dw"] is a float matrix; add=True then adds to what that holds (the microbatches' running sum)."""
    T, V, H = _head_inputs(x, w, target)
    _vector(lse, "lse", _F32, x.device, T)
    if weight is not None:
        _vector(weight, "weight", _F32, x.device, T)
    if not outputs or any(o not in ("dx", "dw") for o in outputs):
        raise ValueError(f"outputs: expected some of 'dx' and 'dw', got {outputs!r}")
    with _On(x.device, stream) as on:
        out = dict(out or {})
        dx = _out(out, "dx", (T, H), _BF16, x.device) if "dx" in outputs else None
        dw, wide = None, False
        if "dw" in outputs:
            wide = isinstance(out.get("dw"), torch.Tensor) and out["dw"].dtype == _F32
            dw = _out(out, "dw", (V, H), _F32 if wide else _BF16, x.device)
        if add and not wide:
            raise ValueError("add: needs a float out['dw'] to add to")
        ws = on.scratch(workspace, head_backward_workspace(x, w))
        _check(LIB.pp_stage_head_backward(*_m(x), *_m(w), _ptr(target), _ptr(lse), _ptr(weight), float(scale), T, V, H,
                                          *_m(dx), *_m(dw), int(wide), int(bool(add)), _ptr(ws), ws.numel(),
                                          on.handle), "pp_stage_head_backward")
    return out


def _new_packed(T, H, device):
    # rows padded to 16 bytes, so that every reader takes its wide path
    ld = -(-H // 16) * 16
    return Packed(torch.empty((T, ld), dtype=torch.int8, device=device)[:, :H],
                  torch.empty((T, -(-H // BLOCK)), dtype=torch.int8, device=device))


def pack(x, *, out=None, stream=None):
    """The 8-bit checkpoint (a Packed) of an activation x [T, H] bf16."""
    T, H = _matrix(x, "x", _BF16, None)
    with _On(x.device, stream) as on:
        p = _new_packed(T, H, x.device) if out is None else _packed(out, "out", x.device, (T, H))
        _check(LIB.pp_stage_pack(*_m(x), T, H, *_m(p.q), *_m(p.e), on.handle), "pp_stage_pack")
    return p


def unpack(packed, *, out=None, stream=None):
    """What a checkpoint stands for, bf16 [T, H] (exactly: the steps are powers of two)."""
    _packed(packed, "packed", None)
    T, H = packed.q.shape
    with _On(packed.q.device, stream) as on:
        x = _out({} if out is None else {"out": out}, "out", (T, H), _BF16, packed.q.device)
        _check(LIB.pp_stage_unpack(*_m(packed.q), *_m(packed.e), T, H, *_m(x), on.handle), "pp_stage_unpack")
    return x


def _packed(p, name, device, shape=None):
    if not isinstance(p, Packed):
        raise TypeError(f"{name}: expected a Packed checkpoint, got {type(p).__name__}")
    if device is not None and p.q.device != device:
        raise ValueError(f"{name}: expected a checkpoint on {device}, got one on {p.q.device}")
    if shape is not None and tuple(p.q.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(p.q.shape)}")
    return p


def weight_grad_workspace(dy, packed):
    """Bytes of scratch memory that weight_grad needs."""
    return LIB.pp_stage_weight_grad_workspace(*_m(dy), dy.shape[0], dy.shape[1], packed.q.shape[1])


def weight_grad(dy, packed, *, add=None, out=None, workspace=None, stream=None):
    """The W op of a linear layer whose input [T, H] was kept: float [N, H] = add + dy^T value(packed).

    dy [T, N] bf16.  `add` (float [N, H]) is the running sum of the microbatches; out=add adds in place."""
    T, N = _matrix(dy, "dy", _BF16, None)
    _packed(packed, "packed", dy.device)
    if packed.q.shape[0] != T:
        raise ValueError(f"packed: expected {T} rows, got {packed.q.shape[0]}")
    H = packed.q.shape[1]
    if add is not None:
        _matrix(add, "add", _F32, dy.device, (N, H))
    with _On(dy.device, stream) as on:
        dw = _out({} if out is None else {"out": out}, "out", (N, H), _F32, dy.device)
        ws = on.scratch(workspace, weight_grad_workspace(dy, packed))
        _check(LIB.pp_stage_weight_grad(*_m(dy), *_m(packed.q), *_m(packed.e), T, N, H, *_m(add), *_m(dw), _ptr(ws),
                                        ws.numel(), on.handle), "pp_stage_weight_grad")
    return dw


def _gate(gate, rows_per_gate, T, H, device):
    if gate is None:
        if rows_per_gate:
            raise ValueError("rows_per_gate: given without a gate")
        return 0
    rows = int(rows_per_gate or 0)
    if rows < 0:
        raise ValueError("rows_per_gate must not be negative")
    G = 1 if rows == 0 else -(-T // rows)
    have, _ = _matrix(gate, "gate", _BF16, device, (gate.shape[0], H))
    if have < max(G, 1) or (rows == 0 and have != 1):
        raise ValueError(f"gate: {T} tokens with {rows or T} to a gate take {G} rows, got {have}")
    return rows


def join_forward(x, f, w_post, w_pre, gate=None, *, rows_per_gate=0, alpha=1.0, eps=1e-6, keep=False, out=None,
                 stream=None):
    """A block's output f joins the residual stream x: y = alpha x + gate * w_post * f / rms(f), and the next
    block's input h = w_pre * y / rms(y).

    x, f [T, H], w_post, w_pre [H], gate [G, H] bf16; row t uses gate[t // rows_per_gate] (0: one gate).
    Returns y, h (bf16), rstd_post, rstd_pre (float [T]); keep=True adds kept_y and kept_f, the checkpoints that
    join_backward reads."""
    T, H = _matrix(x, "x", _BF16, None)
    _matrix(f, "f", _BF16, x.device, (T, H))
    _vector(w_post, "w_post", _BF16, x.device, H)
    _vector(w_pre, "w_pre", _BF16, x.device, H)
    rows = _gate(gate, rows_per_gate, T, H, x.device)
    with _On(x.device, stream) as on:
        out = dict(out or {})
        y, h = (_out(out, k, (T, H), _BF16, x.device) for k in ("y", "h"))
        r1, r2 = (_out(out, k, (T,), _F32, x.device) for k in ("rstd_post", "rstd_pre"))
        kept = [None] * 4
        if keep:
            for i, k in enumerate(("kept_y", "kept_f")):
                if out.get(k) is None:
                    out[k] = _new_packed(T, H, x.device)
                kept[2 * i], kept[2 * i + 1] = _packed(out[k], k, x.device, (T, H)).q, out[k].e
        _check(LIB.pp_stage_join_forward(*_m(x), *_m(f), _ptr(w_post), _ptr(w_pre), *_m(gate), rows, float(alpha),
                                         float(eps), T, H, *_m(y), *_m(h), _ptr(r1), _ptr(r2),
                                         *(a for t in kept for a in _m(t)), on.handle), "pp_stage_join_forward")
    return out


def join_backward_workspace(T, H, rows_per_gate=0):
    """Bytes of scratch memory that join_backward needs."""
    return LIB.pp_stage_join_backward_workspace(T, H, rows_per_gate)


def join_backward(dh, dy, y, f, rstd_post, rstd_pre, w_post, w_pre, gate=None, *, rows_per_gate=0, alpha=1.0,
                  out=None, workspace=None, stream=None):
    """Gradients of the join, from dh (of h) and dy (what reaches y by other paths; None: nothing does).

    y and f are both bf16 [T, H] or both Packed checkpoints.  Returns dx, df (bf16), dw_post, dw_pre (float [H])
    and, with a gate, dgate (float [G, H])."""
    T, H = _matrix(dh, "dh", _BF16, None)
    dev = dh.device
    if dy is not None:
        _matrix(dy, "dy", _BF16, dev, (T, H))
    packed = isinstance(y, Packed)
    if packed != isinstance(f, Packed):
        raise TypeError("y and f: expected two checkpoints or two tensors")
    for name, t in (("y", y), ("f", f)):
        if packed:
            _packed(t, name, dev, (T, H))
        else:
            _matrix(t, name, _BF16, dev, (T, H))
    _vector(rstd_post, "rstd_post", _F32, dev, T)
    _vector(rstd_pre, "rstd_pre", _F32, dev, T)
    _vector(w_post, "w_post", _BF16, dev, H)
    _vector(w_pre, "w_pre", _BF16, dev, H)
    rows = _gate(gate, rows_per_gate, T, H, dev)
    with _On(dev, stream) as on:
        out = dict(out or {})
        dx, df = (_out(out, k, (T, H), _BF16, dev) for k in ("dx", "df"))
        dw1, dw2 = (_out(out, k, (H,), _F32, dev) for k in ("dw_post", "dw_pre"))
        dg = None
        if gate is not None:
            dg = _out(out, "dgate", tuple(gate.shape), _F32, dev)
            used = 1 if rows == 0 else -(-T // rows)
            if T == 0 or used < gate.shape[0]:  # gates that no token uses
                dg[used if T else 0:].zero_()
        ws = on.scratch(workspace, join_backward_workspace(T, H, rows))
        saved = [None if packed else y, None if packed else f,
                 *((y.q, y.e, f.q, f.e) if packed else (None,) * 4)]
        _check(LIB.pp_stage_join_backward(*_m(dh), *_m(dy), *(a for t in saved for a in _m(t)), _ptr(rstd_post),
                                          _ptr(rstd_pre), _ptr(w_post), _ptr(w_pre), *_m(gate), rows, float(alpha),
                                          T, H, *_m(dx), *_m(df), _ptr(dw1), _ptr(dw2), *_m(dg), _ptr(ws), ws.numel(),
                                          on.handle), "pp_stage_join_backward")
    return out


def wait_failure():
    """The first wait inside a product that ran out since the previous call (0: none); synchronizes the device."""
    word = ctypes.c_uint64()
    _check(LIB.pp_stage_wait_failure(ctypes.byref(word)), "pp_stage_wait_failure")
    return word.value
