"""The operators of one pipeline stage (include/ppstage.h): argument checks
and marshalling only, every step of the computation runs in the library.

    head_forward, head_backward   the last stage's loss over a large vocabulary
                                  and its gradients, without kept logits
    score_forward, score_backward log probabilities of given tokens, entropy and
                                  likeliest alternatives, and their gradients
    pack, unpack, weight_grad     activation checkpoints in 8 bits and the
                                  weight gradient (the W op) taken from them
    join_forward, join_backward   the norm after a block, its gate, the residual
                                  scale and sum, the norm before the next block
    grad_norm, AdamW              after the flush: the norm of the gradients and
                                  the step over all tensors of the stage

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

import array
import ctypes
import math
import operator
import struct

import torch

from .binding import LIB, PP_OK, PPSchedError, _arg, _check, _reach

EXPORTS = ("pp_stage_head_forward_workspace", "pp_stage_head_forward", "pp_stage_head_backward_workspace",
           "pp_stage_head_backward", "pp_stage_score_forward_workspace", "pp_stage_score_forward",
           "pp_stage_score_backward_workspace", "pp_stage_score_backward", "pp_stage_pack", "pp_stage_unpack",
           "pp_stage_weight_grad_workspace", "pp_stage_weight_grad", "pp_stage_join_forward", "pp_stage_join_backward_workspace",
           "pp_stage_join_backward", "pp_stage_grad_norm_workspace", "pp_stage_grad_norm", "pp_stage_adamw_workspace",
           "pp_stage_adamw", "pp_stage_adamw_moments", "pp_stage_wait_failure")

#: Columns of a checkpoint, and elements of a moment in 8 bits, that share one exponent.
BLOCK = 64
#: Most alternatives of a token.
MAX_TOP = 32
#: Exponent of a checkpoint's block that holds an infinity or a NaN.
NONFINITE = -128


class _Tensors(ctypes.Structure):
    """pp_stage_tensor.  Lists of them are built as 64-bit words, six to an entry: setting fields one by one is most of
    the time that a call over a few hundred tensors takes."""
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("at", ctypes.c_int64), ("decay", ctypes.c_float), ("p_float", ctypes.c_uint8), ("g_float", ctypes.c_uint8)]


_WORDS, _P_FLOAT, _G_FLOAT = 6, 1 << 32, 1 << 40  # words of an entry; bits of its last
assert ctypes.sizeof(_Tensors) == 8 * _WORDS and _Tensors.g_float.offset == 8 * _WORDS - 3


def _declare(lib):
    vp, i32, i64, f32, size = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    f64, u64 = ctypes.c_double, ctypes.c_uint64
    m = [vp, i64]  # a matrix: pointer and row stride
    lib.pp_stage_head_forward_workspace.argtypes = [*m, *m, i64, i64, i64]
    lib.pp_stage_head_forward.argtypes = [*m, *m, vp, i64, i64, i64, vp, vp, vp, size, vp]
    lib.pp_stage_head_backward_workspace.argtypes = [*m, *m, i64, i64, i64]
    lib.pp_stage_head_backward.argtypes = [*m, *m, vp, vp, vp, f32, i64, i64, i64, *m, *m, i32, i32, vp, size, vp]
    lib.pp_stage_score_forward_workspace.argtypes = [*m, *m, i64, i64, i64, i64]
    lib.pp_stage_score_forward.argtypes = [*m, *m, vp, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, size, vp]
    lib.pp_stage_score_backward_workspace.argtypes = [*m, *m, i64, i64, i64]
    lib.pp_stage_score_backward.argtypes = [*m, *m, vp, vp, vp, vp, vp, i64, i64, i64, *m, *m, i32, i32, vp, size, vp]
    lib.pp_stage_grad_norm_workspace.argtypes = [vp, i64]
    lib.pp_stage_grad_norm.argtypes = [vp, i64, vp, vp, vp, size, vp]
    lib.pp_stage_adamw_workspace.argtypes = []
    lib.pp_stage_adamw.argtypes = [vp, i64, vp, vp, vp, vp, i64, vp, vp, f64, f64, f64, f64, vp, vp, f64, i32, u64, vp, size, vp]
    lib.pp_stage_adamw_moments.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp]
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
_STEP_BYTES = LIB.pp_stage_adamw_workspace()


_BF16, _F32, _I64, _I8, _U8 = torch.bfloat16, torch.float32, torch.int64, torch.int8, torch.uint8
_Tensor, _empty = torch.Tensor, torch.empty
_data_ptr, _get_device, _is_contiguous, _numel = _Tensor.data_ptr, _Tensor.get_device, _Tensor.is_contiguous, _Tensor.numel
_dtype, _shape = operator.attrgetter("dtype"), operator.attrgetter("shape")
# the handle of a device's current stream and the current device, without the objects around them: a small call
# is mostly its host path
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_capturing = torch._C._cuda_isCurrentStreamCapturing


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


def _gradients(out, outputs, add, T, V, H, device, dev):
    """(pointer, stride) of dx and of dw, and whether dw is float."""
    if not outputs or any(o not in ("dx", "dw") for o in outputs):
        raise ValueError(f"outputs: expected some of 'dx' and 'dw', got {outputs!r}")
    dx = _out_matrix(out, "dx", T, H, _BF16, device, dev) if "dx" in outputs else (None, 0)
    dw, wide = (None, 0), False
    if "dw" in outputs:
        wide = isinstance(out.get("dw"), _Tensor) and out["dw"].dtype is _F32
        if add and not wide:
            raise ValueError("add: needs a float out['dw'] to add to")
        dw = _out_matrix(out, "dw", V, H, _F32 if wide else _BF16, device, dev)
    return dx, dw, wide


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
    out, device = dict(out) if out else {}, x.device
    dx, dw, wide = _gradients(out, outputs, add, T, V, H, device, dev)
    need = LIB.pp_stage_head_backward_workspace(px, sx, pw, sw, T, V, H)
    _keep, ws, n = _scratch(workspace, need, device, dev)
    rc = LIB.pp_stage_head_backward(px, sx, pw, sw, pt, pl, pg, scale, T, V, H, *dx, *dw, wide, bool(add) and wide, ws, n,
                                    _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_head_backward")
    return out


def _top(top, V):
    if isinstance(top, bool) or not isinstance(top, int) or not 0 <= top <= min(MAX_TOP, V):
        raise ValueError(f"top: expected a whole number from 0 to {min(MAX_TOP, V)}, got {top!r}")
    return top


def score_forward_workspace(x, w, top=0):
    """Bytes of scratch memory that score_forward needs for these matrices."""
    px, sx, T, H = _matrix(x, "x", _BF16, _device(x))
    pw, sw, V, _ = _matrix(w, "w", _BF16, _device(x), None, H)
    return LIB.pp_stage_score_forward_workspace(px, sx, pw, sw, T, V, H, _top(top, V))


def score_backward_workspace(x, w):
    """Bytes of scratch memory that score_backward needs for these matrices."""
    px, sx, T, H = _matrix(x, "x", _BF16, _device(x))
    pw, sw, V, _ = _matrix(w, "w", _BF16, _device(x), None, H)
    return LIB.pp_stage_score_backward_workspace(px, sx, pw, sw, T, V, H)


def score_forward(x, w, target, *, top=0, out=None, workspace=None, stream=None):
    """Log probabilities of the given tokens under the softmax of the logits x w^T, without keeping those.

    x [T, H], w [V, H] bf16; target [T] int64, a token whose target is outside 0..V-1 is left out.  Returns logp [T]
    (0 where left out), entropy [T] and lse [T]; float.  With `top` (up to 32) also top_index int64 [T, top], the
    columns of the largest logits in falling order (the lower one first among equals), and top_logp float [T, top]."""
    dev = _device(x)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return score_forward(x, w, target, top=top, out=out, workspace=workspace)
    px, sx, pw, sw, T, V, H, pt = _head_inputs(x, w, target, dev)
    k = _top(top, V)
    out, device = dict(out) if out else {}, x.device
    logp = _out_vector(out, "logp", T, _F32, device, dev)
    lse = _out_vector(out, "lse", T, _F32, device, dev)
    entropy = _out_vector(out, "entropy", T, _F32, device, dev)
    tops = [None, None]
    if k:
        for i, (name, dtype) in enumerate((("top_logp", _F32), ("top_index", _I64))):
            tops[i], stride = _out_matrix(out, name, T, k, dtype, device, dev)
            if stride != k:
                raise ValueError(f"{name}: expected contiguous memory, got a row stride of {stride}")
    need = LIB.pp_stage_score_forward_workspace(px, sx, pw, sw, T, V, H, k)
    _keep, ws, n = _scratch(workspace, need, device, dev)
    rc = LIB.pp_stage_score_forward(px, sx, pw, sw, pt, T, V, H, k, logp, lse, entropy, *tops, ws, n, _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_score_forward")
    return out


def score_backward(x, w, target, lse, dlogp, *, entropy=None, dentropy=None, outputs=("dx", "dw"), add=False, out=None,
                   workspace=None, stream=None):
    """Gradients of a loss that depends on score_forward's logp and entropy, from dlogp = dL/dlogp and, if given,
    dentropy = dL/dentropy (float [T]; with it the entropy that score_forward returned).

    Returns dx [T, H] bf16 and dw [V, H], or the one named in `outputs`; dw and `add` as in head_backward.  A token
    that is left out has no gradient, through its entropy neither.  The logits' gradient is held in bf16 between the
    products, each term off by up to 2^-8 of itself, but for the target's, whose rest is added in 32 bits: a float dw
    has 32 bits of the sums, not of the terms."""
    dev = _device(x)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return score_backward(x, w, target, lse, dlogp, entropy=entropy, dentropy=dentropy, outputs=outputs, add=add,
                                  out=out, workspace=workspace)
    px, sx, pw, sw, T, V, H, pt = _head_inputs(x, w, target, dev)
    pl, pg = _vector(lse, "lse", _F32, dev, T), _vector(dlogp, "dlogp", _F32, dev, T)
    if (entropy is None) != (dentropy is None):
        raise ValueError("entropy and dentropy: expected both or neither")
    pe, pd = (None, None) if entropy is None else (_vector(entropy, "entropy", _F32, dev, T),
                                                   _vector(dentropy, "dentropy", _F32, dev, T))
    out, device = dict(out) if out else {}, x.device
    dx, dw, wide = _gradients(out, outputs, add, T, V, H, device, dev)
    need = LIB.pp_stage_score_backward_workspace(px, sx, pw, sw, T, V, H)
    _keep, ws, n = _scratch(workspace, need, device, dev)
    rc = LIB.pp_stage_score_backward(px, sx, pw, sw, pt, pl, pg, pe, pd, T, V, H, *dx, *dw, wide, bool(add) and wide, ws, n,
                                     _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_score_backward")
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


def _flat(t, name, dev, dtypes):
    """Checks a tensor that is taken as one run of elements on CUDA device `dev`."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name}: expected a tensor on {f'cuda:{dev}' if dev >= 0 else 'a CUDA device'}, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous memory, got strides {t.stride()} for shape {tuple(t.shape)}")


def _listed(tensors, name):
    if isinstance(tensors, _Tensor) or not hasattr(tensors, "__iter__"):
        raise TypeError(f"{name}: expected a list of tensors, got {type(tensors).__name__}")
    return list(tensors)


def _accessors(tensors, name, dev):
    """(pointers, types) of tensors that are float or bf16, contiguous and on CUDA device `dev`.  Attribute by attribute:
    PyTorch's accessors are most of what a call over hundreds of tensors costs, and the loops around them are not."""
    if not tensors:
        return [], []
    try:
        ptrs, types = list(map(_data_ptr, tensors)), list(map(_dtype, tensors))
        fine = (dev >= 0 and types.count(_F32) + types.count(_BF16) == len(ptrs) and all(map(_is_contiguous, tensors))
                and list(map(_get_device, tensors)).count(dev) == len(ptrs))
    except (TypeError, AttributeError, RuntimeError):
        fine = False
    if not fine:
        for i, t in enumerate(tensors):
            _flat(t, f"{name}[{i}]", dev, (_F32, _BF16))
        raise ValueError(f"{name}: tensors without plain memory")
    return ptrs, types


def _wide_at(norm, dev):
    """Pointer of what a norm was before its rounding, None where the tensor has none.  Who records the norm on another
    stream does not know of it, so every stream that uses it is recorded here."""
    wide = getattr(norm, "_wide", None)
    if wide is None or wide.get_device() != dev:
        return None
    if wide._made_on != _raw_stream(dev):
        wide.record_stream(torch.cuda.current_stream(dev))
    return wide.data_ptr()


def grad_norm(grads, *, out=None, workspace=None, stream=None):
    """The 2-norm of all gradients together, float [1] on their device: what AdamW.step clips by.

    grads: float or bf16 tensors, contiguous, of any shapes.  A gradient above 1.8e19 makes it infinite.  The tensor
    also carries the norm before its rounding, which the step clips by as long as it rounds to what the tensor holds.
    An `out` keeps the one that it was given first, so that a captured step goes on reading what a later call writes."""
    grads = _listed(grads, "grads")
    dev = _device(grads[0]) if grads else _device(out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return grad_norm(grads, out=out, workspace=workspace)
    ptrs, types = _accessors(grads, "grads", dev)
    table = array.array("Q", bytes(8 * _WORDS * len(ptrs)))
    table[1::_WORDS] = array.array("Q", ptrs)
    table[3::_WORDS] = array.array("Q", map(_numel, grads))
    table[5::_WORDS] = array.array("Q", (_G_FLOAT if t is _F32 else 0 for t in types))
    at = table.buffer_info()[0]
    if out is None:
        if dev < 0:
            raise ValueError("grads: expected at least one tensor, or an `out` on a CUDA device")
        out = _empty(1, dtype=_F32, device=grads[0].device)
    po = _vector(out, "out", _F32, dev, 1)
    wide = _wide_at(out, dev)
    if wide is None:
        out._wide = t = _empty(1, dtype=torch.float64, device=out.device)
        t._made_on = _raw_stream(dev)
        wide = t.data_ptr()
    need = LIB.pp_stage_grad_norm_workspace(at, len(grads))
    _keep, ws, n = _scratch(workspace, need, out.device, dev)
    rc = LIB.pp_stage_grad_norm(at, len(grads), po, wide, ws, n, _raw_stream(dev))
    if rc != PP_OK:
        raise PPSchedError(rc, "pp_stage_grad_norm")
    return out


class AdamW:
    """The AdamW step over the tensors of a stage, in a few launches whatever their number.

        m = beta1 m + (1 - beta1) g      v = beta2 v + (1 - beta2) g^2
        p = p (1 - lr decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)

    params: contiguous float or bf16 tensors of any shapes, updated in place, none overlapping another, nor a gradient.
    copies: for float parameters, a list of bf16 tensors of the same shapes (or None for one that has none) that receive
    the new values.  weight_decay: a number, or one for each parameter.  eps: 0 (an element whose moments are both 0 is
    then 0 / 0), or 2**-126 and more.  All these keep the memory that they have here: a step refuses others.

    The moments are held in 32 bits or (bits=8) in 8: 64 consecutive elements share an exponent, each keeps 4 significant
    bits; 2.03 bytes an element for both.  A block of a moment that is not finite any more (a gradient whose square is
    beyond 32 bits) is NaN from then on; clip by a norm, which such a gradient makes infinite.  With a `seed` moments in
    8 bits and bf16 parameters are rounded up with the probability of what is cut off, by random bits that depend on the
    seed, the step and the element's place alone; without one to nearest, which an average that changes by 1 - beta2 a
    step does not survive in 4 bits for long.

    ``state`` has the flat tensors that a checkpoint keeps: "m", "v" (bits=8: and "m_exp", "v_exp"), each parameter's from
    a multiple of 64 elements on, and "step", int64 [1], the steps taken.  Pass such a dict as ``state`` to go on from it
    (the tensors are used, not copied).  The step's number is counted on the device: a captured step counts on at every
    replay.  One step at a time: calls on several streams are the caller's to order, and so are the tensors (``state``
    among them) that a step on another stream still works on when they are let go."""

    def __init__(self, params, *, bits=32, copies=None, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, seed=None,
                 state=None):
        params = _listed(params, "params")
        if not params:
            raise ValueError("params: expected at least one tensor")
        if bits not in (8, 32):
            raise ValueError(f"bits: expected 8 or 32, got {bits!r}")
        b1, b2 = (float(b) for b in betas)
        if not (0 <= b1 < 1 and 0 <= b2 < 1):
            raise ValueError(f"betas: expected two numbers from 0 to below 1, got {betas!r}")
        if float(eps) != 0 and not 2.0 ** -126 <= float(eps) <= 3e38:
            raise ValueError(f"eps: expected 0 or a normal number of 32 bits above it, got {eps!r}")
        if seed is not None and (isinstance(seed, bool) or not isinstance(seed, int) or not 0 <= seed < 1 << 64):
            raise ValueError(f"seed: expected a whole number of 64 bits or None, got {seed!r}")
        dev = _device(params[0])
        copies = [None] * len(params) if copies is None else _listed(copies, "copies")
        decay = [weight_decay] * len(params) if isinstance(weight_decay, (int, float)) else list(weight_decay)
        for name, given in (("copies", copies), ("weight_decay", decay)):
            if len(given) != len(params):
                raise ValueError(f"{name}: expected {len(params)}, one for each parameter, got {len(given)}")
        self.bits, self.betas, self.eps, self.seed = bits, (b1, b2), float(eps), seed
        self.params, self.copies = tuple(params), tuple(copies)
        self._dev = dev
        words = []
        held = 0
        for i, (p, c, d) in enumerate(zip(params, copies, decay)):
            _flat(p, f"params[{i}]", dev, (_F32, _BF16))
            if c is not None:
                _flat(c, f"copies[{i}]", dev, (_BF16,))
                if p.dtype is not _F32:
                    raise TypeError(f"copies[{i}]: params[{i}] is bf16 itself")
                if c.shape != p.shape:
                    raise ValueError(f"copies[{i}]: expected shape {tuple(p.shape)}, got {tuple(c.shape)}")
            if not abs(d) <= 3e38:
                raise ValueError(f"weight_decay: expected a finite number for params[{i}], got {d!r}")
            bits_of_d = int.from_bytes(struct.pack("<f", d), "little")
            words += (p.data_ptr(), 0, 0 if c is None else c.data_ptr(), p.numel(), held,
                      bits_of_d + (_P_FLOAT if p.dtype is _F32 else 0))
            held += (p.numel() + BLOCK - 1) // BLOCK * BLOCK
        self._table = array.array("Q", words)
        self._shapes = [p.shape for p in params]
        self._flags, self._types = self._table[5::_WORDS], None  # of the gradients that the table was filled with last
        self._held, self._device = held, params[0].device
        self._state = self._new_state() if state is None else self._given_state(state)
        # a step goes by the pointers and lengths that these had here
        self._written = [t for t in (*params, *copies, *self._state.values()) if t is not None]
        self._ptrs = list(map(_data_ptr, self._written))
        self._updated = [t for t in (*params, *copies) if t is not None]
        with torch.cuda.device(dev):
            self._work, self._work_on = _empty(_STEP_BYTES, dtype=_U8, device=self._device), _raw_stream(dev)
        named = ([("params", p) for p in params] + [("copies", c) for c in copies]
                 + [("state", t) for t in self._state.values()])
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name) for name, t in named
                       if t is not None and t.numel())
        for (_, end, one), (start, _, other) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError(f"{one} and {other}: two of their tensors overlap")

    @property
    def state(self):
        """The tensors that a checkpoint keeps, by name."""
        return dict(self._state)

    def _layout(self):
        small = self.bits == 8
        names = {"m": (_U8 if small else _F32, self._held), "v": (_U8 if small else _F32, self._held),
                 "step": (_I64, 1)}
        if small:
            names["m_exp"] = names["v_exp"] = (_U8, self._held // BLOCK)
        return names

    def _new_state(self):
        return {k: torch.zeros(n, dtype=dtype, device=self._device) for k, (dtype, n) in self._layout().items()}

    def _given_state(self, state):
        layout = self._layout()
        if set(state) != set(layout):
            raise ValueError(f"state: expected {sorted(layout)}, got {sorted(state)}")
        for k, (dtype, n) in layout.items():
            _vector(state[k], f"state[{k!r}]", dtype, self._dev, n)
            if k in "mv" and state[k].data_ptr() % 32:
                raise ValueError(f"state[{k!r}]: expected memory that starts on 32 bytes")
        return dict(state)

    def _check_memory(self):
        if list(map(_data_ptr, self._written)) != self._ptrs:
            raise ValueError("params, copies, state: their memory is not that which this step was made for")

    def step(self, grads, lr, *, norm=None, max_norm=None, stream=None):
        """One step.  grads: float or bf16, of the parameters' shapes.  lr: a number, or a float [1] tensor on the device
        that is read when the step runs.  With `norm` (of grad_norm) and `max_norm` the gradients are scaled by
        max_norm / norm where the norm is larger; where it is not a finite number nothing changes, the step's number
        neither."""
        dev = self._dev
        ctx = _elsewhere(dev, stream)
        if ctx is not None:
            with ctx:
                return self.step(grads, lr, norm=norm, max_norm=max_norm)
        if len(grads) != len(self.params):
            raise ValueError(f"grads: expected {len(self.params)}, one for each parameter, got {len(grads)}")
        grads = list(grads)
        ptrs, types = _accessors(grads, "grads", dev)
        if list(map(_shape, grads)) != self._shapes:
            i = next(i for i, (g, s) in enumerate(zip(grads, self._shapes)) if g.shape != s)
            raise ValueError(f"grads[{i}]: expected shape {tuple(self._shapes[i])}, got {tuple(grads[i].shape)}")
        self._check_memory()
        table = self._table
        table[1::_WORDS] = array.array("Q", ptrs)
        if types != self._types:
            self._types = types
            table[5::_WORDS] = array.array("Q", (f | _G_FLOAT if t is _F32 else f for f, t in zip(self._flags, types)))
        lr_at = _vector(lr, "lr", _F32, dev, 1) if isinstance(lr, _Tensor) else None
        rate = 0.0 if lr_at is not None else float(lr)
        if not math.isfinite(rate):
            raise ValueError(f"lr: expected a finite number, got {lr!r}")
        if (norm is None) != (max_norm is None):
            raise ValueError("norm and max_norm: expected both or neither")
        if max_norm is not None and not 0 < max_norm < math.inf:
            raise ValueError(f"max_norm: expected a number above 0, got {max_norm!r}")
        pn = None if norm is None else _vector(norm, "norm", _F32, dev, 1)
        wide = None if norm is None else _wide_at(norm, dev)
        s = self._state
        small = self.bits == 8
        # its own scratch memory only where that was allocated: another stream's step has its own, and a captured one
        # the graph's (allocating at every step takes 5 us of a small one's 20)
        ws = self._work
        if _raw_stream(dev) != self._work_on or _capturing():
            ws = _empty(_STEP_BYTES, dtype=_U8, device=self._device)
        rc = LIB.pp_stage_adamw(table.buffer_info()[0], len(self.params), s["m"].data_ptr(), s["v"].data_ptr(),
                                s["m_exp"].data_ptr() if small else None, s["v_exp"].data_ptr() if small else None,
                                self._held, s["step"].data_ptr(), lr_at, rate, *self.betas, self.eps, pn, wide,
                                max_norm or 1.0, self.seed is not None, self.seed or 0, ws.data_ptr(), _STEP_BYTES,
                                _raw_stream(dev))
        if rc != PP_OK:
            raise PPSchedError(rc, "pp_stage_adamw")
        # what autograd saved of them before is not what a backward pass would find now
        torch.autograd.graph.increment_version(self._updated)

    def moments(self, *, stream=None):
        """(m, v) as numbers, flat as in ``state``: its float tensors themselves, or what the 8 bits stand for, as bf16."""
        s, dev = self._state, self._dev
        if self.bits == 32:
            return s["m"], s["v"]
        ctx = _elsewhere(dev, stream)
        if ctx is not None:
            with ctx:
                return self.moments()
        self._check_memory()
        m, v = (torch.empty(self._held, dtype=_BF16, device=self._device) for _ in range(2))
        rc = LIB.pp_stage_adamw_moments(s["m"].data_ptr(), s["v"].data_ptr(), s["m_exp"].data_ptr(), s["v_exp"].data_ptr(),
                                        self._held, m.data_ptr(), v.data_ptr(), _raw_stream(dev))
        if rc != PP_OK:
            raise PPSchedError(rc, "pp_stage_adamw_moments")
        return m, v


def wait_failure():
    """A record of a wait that ran out on the current device since the previous call (0: none); synchronizes the device.

    Calls return before their kernels have run, so they cannot tell: a block whose wait for its own copies or matrix
    instructions runs out gives up, and the call's outputs are wrong.  Ask after a step, before its results are used."""
    word = ctypes.c_uint64()
    _check(LIB.pp_stage_wait_failure(ctypes.byref(word)), "pp_stage_wait_failure")
    return word.value
