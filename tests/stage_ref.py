"""The pipeline-stage operators' definitions in 64 bits, and for each output
the error that its computation in 32 bits with bf16 results may have.

Bounds: a sum of n products taken in 32 bits, in any order and with truncating
adders, is off by at most n * 2^-23 times the sum of the magnitudes (U32 per
step); a result rounded to bf16 by 2^-8 of itself (U16: the type has 8
significant bits, so 1 + 2^-8 lies halfway between two of its numbers), or by
the smallest bf16 step near 0."""
import torch

F64 = torch.float64
U32, U16, TINY = 2.0 ** -23, 2.0 ** -8, 2.0 ** -130
BLOCK = 64


def left_in(target, V):
    return (target >= 0) & (target < V)


def head(x, w, target, scale=1.0, weight=None):
    """{name: (value, bound)} of loss, lse, dx, dw."""
    V, H = w.shape
    T = x.shape[0]
    keep = left_in(target, V)
    x = torch.where(keep[:, None], x.to(F64), 0.0) if x.isnan().any() or x.isinf().any() else x.to(F64)
    w = w.to(F64)
    l = x @ w.t()
    lse = torch.logsumexp(l, 1)
    at = torch.where(keep, target, 0)
    loss = torch.where(keep, lse - l.gather(1, at[:, None])[:, 0], 0.0)
    # a logit's error; then the exponentials' own: their argument is at most some 200 wide, and the sum's
    dl = H * U32 * (x.abs() @ w.abs().t()).amax(1)
    eps = 2 * dl + 2.0 ** -16 + (256 + V / 64) * U32
    c = torch.where(keep, torch.ones(T, dtype=F64, device=x.device) if weight is None else weight.to(F64), 0.0)
    p = torch.exp(l - lse[:, None])
    d = p.clone()
    d[torch.arange(T, device=x.device), at] -= 1
    d *= c[:, None]
    err = U16 * d.abs() + (c.abs() * eps)[:, None] * p + TINY
    dx, dw = scale * (d @ w), scale * (d.t() @ x)
    s = abs(scale)
    b_dx = s * ((err + V * U32 * d.abs()) @ w.abs()) + U16 * dx.abs() + TINY
    b_dw = s * ((err + T * U32 * d.abs()).t() @ x.abs()) + U16 * dw.abs() + TINY
    return {"loss": (loss, eps + U32 * loss), "lse": (lse, eps + U32 * lse.abs()), "dx": (dx, b_dx), "dw": (dw, b_dw)}


def pack(x):
    """The checkpoint of x: whole numbers, exact."""
    T, H = x.shape
    v = torch.nn.functional.pad(x.to(F64), (0, -H % BLOCK)).reshape(T, -1, BLOCK)
    a = v.abs().amax(2)
    fine = torch.isfinite(v).all(2)
    k = torch.frexp(torch.where(fine & (a > 0), a, 1.0))[1] - 1
    e = torch.where(a > 0, k - 6, -126).clamp_min(-126)
    step = torch.ldexp(torch.ones((), dtype=F64), e.cpu()).to(x.device)
    q = torch.where(fine[:, :, None], (v / step[:, :, None]).round().clamp(-127, 127), 0.0)
    return q.reshape(T, -1)[:, :H].to(torch.int8), torch.where(fine, e, -128).to(torch.int8)


def value(q, e):
    """What a checkpoint stands for, in 64 bits."""
    step = torch.ldexp(torch.ones((), dtype=F64), e.cpu().int()).to(q.device)
    step = torch.where(e == -128, torch.nan, step)
    return q.to(F64) * step.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def weight_grad(dy, v, add=None):
    dy = dy.to(F64)
    r = dy.t() @ v
    b = (dy.shape[0] + 1) * U32 * (dy.abs().t() @ v.abs()) + TINY
    if add is not None:
        r = r + add.to(F64)
        b = b + U32 * r.abs()
    return r, b


def _gate_rows(gate, rows, T, H, device):
    if gate is None:
        return torch.ones(T, H, dtype=F64, device=device)
    at = torch.zeros(T, dtype=torch.int64, device=device) if not rows else torch.arange(T, device=device) // rows
    return gate.to(F64)[at]


def join_forward(x, f, w_post, w_pre, gate, rows, alpha, eps):
    T, H = x.shape
    x, f, w1, w2 = (t.to(F64) for t in (x, f, w_post, w_pre))
    g = _gate_rows(gate, rows, T, H, x.device)
    r1 = (f.square().mean(1) + eps).rsqrt()
    b = g * w1 * f * r1[:, None]
    y = alpha * x + b
    r2 = (y.square().mean(1) + eps).rsqrt()
    h = y * r2[:, None] * w2
    # a norm's sum: at most 16 + 5 + 32 adders in a row; with the rsqrt and the products fewer than 64 steps of 2^-24
    rel = 32 * U32
    ey = rel * ((alpha * x).abs() + b.abs())
    # y's own error moves r2 by at most its share of the row's norm
    er2 = rel + (ey.square().mean(1) / (y.square().mean(1) + eps)).sqrt()
    eh = (ey * r2[:, None] + y.abs() * (r2 * (er2 + rel))[:, None]) * w2.abs()
    return {"y": (y, ey + U16 * y.abs() + TINY), "h": (h, eh + U16 * h.abs() + TINY), "rstd_post": (r1, rel * r1),
            "rstd_pre": (r2, er2 * r2)}


def join_backward(dh, dy, y, f, r1, r2, w_post, w_pre, gate, rows, alpha):
    T, H = dh.shape
    dh, y, f, w1, w2 = (t.to(F64) for t in (dh, y, f, w_post, w_pre))
    dy = torch.zeros_like(dh) if dy is None else dy.to(F64)
    r1, r2 = r1.to(F64)[:, None], r2.to(F64)[:, None]
    g = _gate_rows(gate, rows, T, H, dh.device)
    rel = 64 * U32

    def norm_back(up, n, r, e_up):
        """Gradient through n = v r and its error, given the upstream gradient's error."""
        m, M = (up * n).mean(1, keepdim=True), (up * n).abs().mean(1, keepdim=True)
        v = r * (up - n * m)
        e = r * (e_up + rel * (up.abs() + n.abs() * M) + n.abs() * (e_up * n.abs()).mean(1, keepdim=True))
        return v, e

    n2, n1 = y * r2, f * r1
    back, e_d = norm_back(dh * w2, n2, r2, rel * (dh * w2).abs())
    d = dy + back
    e_d = e_d + rel * (dy.abs() + back.abs())
    s = d * g * w1
    df, e_df = norm_back(s, n1, r1, (e_d * (g * w1).abs()) + rel * s.abs())
    out = {"dx": (alpha * d, abs(alpha) * e_d + U16 * (alpha * d).abs() + TINY),
           "df": (df, e_df + U16 * df.abs() + TINY),
           "dw_pre": ((dh * n2).sum(0), (rel + T * U32) * (dh * n2).abs().sum(0) + TINY),
           "dw_post": ((d * g * n1).sum(0),
                       ((e_d * g.abs() + (rel + T * U32) * (d * g).abs()) * n1.abs()).sum(0) + TINY)}
    if gate is not None:
        at = torch.zeros(T, dtype=torch.int64, device=dh.device) if not rows else torch.arange(T, device=dh.device) // rows
        zero = torch.zeros(gate.shape, dtype=F64, device=dh.device)
        out["dgate"] = (zero.index_add(0, at, d * n1) * w1,
                        zero.index_add(0, at, (e_d + (rel + T * U32) * d.abs()) * n1.abs()) * w1.abs() + TINY)
    return out


def check(got, want, what=""):
    """Every element within its bound; non-finite ones equal."""
    value_, bound = want
    got = got.to(F64)
    assert got.shape == value_.shape, what
    fine = torch.isfinite(value_)
    assert torch.equal(torch.isnan(got), torch.isnan(value_)), f"{what}: NaN in other places"
    rest = ~fine & ~torch.isnan(value_)
    assert torch.equal(got[rest], value_[rest]), f"{what}: infinities differ"
    over = (got[fine] - value_[fine]).abs() - bound.expand_as(value_)[fine]
    assert not (over > 0).any(), f"{what}: {int((over > 0).sum())} of {over.numel()} over the bound, worst by {over.max()}"


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0, stride=None, offset=0):
    """A bf16 matrix, as a view with this row stride and offset (elements) of a larger buffer filled with NaN."""
    v = (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)
    if stride is None:
        return v
    buf = torch.full((offset + shape[0] * stride,), torch.nan, dtype=torch.bfloat16, device="cuda")
    view = buf[offset:offset + shape[0] * stride].view(shape[0], stride)[:, :shape[1]]
    view.copy_(v)
    return view
