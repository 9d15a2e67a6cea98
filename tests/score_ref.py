"""What score_forward and score_backward compute, in 64 bits, with the error that
each output may have; the bounds' steps are those of stage_ref.

A logit's error dl moves lse by dl at most, and the entropy by
sum_v p |log p + H| 2 dl <= 4 H dl.  With every exponential off by a share eps
(its argument's rounding, the sum's steps), log s is off by eps and the mean of
-log p by 2 eps of itself.  What is summed up for d is off by p times the error of
its factor, plus the rounding to bf16."""
import torch

import stage_ref as R

F64, U32, U16, TINY = R.F64, R.U32, R.U16, R.TINY


def grid(g, *shape, scale=1.0):
    """Whole numbers up to 31 times scale / 8, a power of two: sums of up to 16,384 products of two such are exact in 32
    bits, whatever their order."""
    return ((torch.randn(*shape, generator=g, device="cuda") * 8).round().clamp(-31, 31) * (scale / 8)).to(torch.bfloat16)


def top(l, k):
    """Columns of the k largest of each row in falling order, the lower first among equals, NaN behind all."""
    order = torch.sort(torch.where(l.isnan(), -torch.inf, l), dim=1, descending=True, stable=True).indices[:, :k]
    return order


def score(x, w, target, k=0, dlogp=None, dentropy=None, exact=False):
    """{name: (value, bound)}; exact: the logits are (see grid)."""
    V, H = w.shape
    T = x.shape[0]
    keep = R.left_in(target, V)
    xd, wd = x.to(F64), w.to(F64)
    l = xd @ wd.t()
    lse = torch.logsumexp(l, 1)
    at = torch.where(keep, target, 0)
    lp = l - lse[:, None]
    logp = torch.where(keep, lp.gather(1, at[:, None])[:, 0], 0.0)
    dl = torch.zeros(T, dtype=F64, device=x.device) if exact else H * U32 * (xd.abs() @ wd.abs().t()).amax(1)
    share = 2.0 ** -16 + (256 + V / 64) * U32
    eps = 2 * dl + share
    p = torch.exp(lp)
    ent = -(p * lp.clamp_min(-1e30)).sum(1)
    e_ent = 4 * ent * dl + share * (1 + 2 * ent) + U32 * ent
    out = {"logp": (logp, eps + U32 * logp.abs()), "lse": (lse, eps + U32 * lse.abs()), "entropy": (ent, e_ent)}
    if k:
        i = top(l, k)
        t = lp.gather(1, i)
        out["top_logp"] = (t, (eps[:, None] + U32 * t.abs()))
        out["top_index"] = i
    if dlogp is not None:
        a = torch.where(keep, dlogp.to(F64), 0.0)
        b = torch.zeros_like(a) if dentropy is None else torch.where(keep, dentropy.to(F64), 0.0)
        inner = a[:, None] + b[:, None] * (lp + ent[:, None])
        d = -p * inner
        d[torch.arange(T, device=x.device), at] += a
        err = U16 * d.abs() + p * (inner.abs() * eps[:, None] + (b.abs() * (eps + e_ent + 4 * U32 * (ent + 1)))[:, None]
                                   + 4 * U32 * (a.abs()[:, None] + b.abs()[:, None] * lp.abs())) + TINY
        xk = torch.where(keep[:, None], xd, 0.0)
        dx, dw = d @ wd, d.t() @ xk
        out["dx"] = (dx, (err + V * U32 * d.abs()) @ wd.abs() + U16 * dx.abs() + TINY)
        out["dw"] = (dw, (err + T * U32 * d.abs()).t() @ xk.abs() + U16 * dw.abs() + TINY)
    return out
