"""The AdamW step and its 8-bit moments from their definitions in 64 bits, on
whatever device the inputs are on.

E = 2^-24: a 32-bit rounding.  m and v are two products (v: three, with the
square) and a sum, of constants that are rounded themselves, and g may carry a
rounded factor (v: twice): 4 E and 8 E of the terms' magnitudes.  The step
m / (sqrt(v) r + eps) has a root and a quotient to 2 units each, four more
roundings, and m's and v's own errors."""
import torch

F64 = torch.float64
E, U16, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -126
BLOCK = 64


def two_to(e):
    """2 to whole numbers (-1022..1023) in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def step(p, g, m, v, t, lr, betas, eps, decay, clip=1.0):
    """{name: (value, bound)} of p, m, v; inputs in any type, p's rounding to bf16 not counted."""
    b1, b2 = betas
    p, g, m, v = (x.to(F64) for x in (p, g, m, v))
    g = g * clip
    mm, em = b1 * m + (1 - b1) * g, 4 * E * ((b1 * m).abs() + ((1 - b1) * g).abs()) + TINY
    vv, ev = b2 * v + (1 - b2) * g * g, 8 * E * (b2 * v + (1 - b2) * g * g) + TINY
    size, root = lr / (1 - b1 ** t), (1 - b2 ** t) ** -0.5
    den = vv.sqrt() * root + eps
    up = size * mm / den
    # the root's own share of v's error is at most half of it
    e_up = size * em / den + up.abs() * (16 * E + (0.5 * ev / vv.clamp_min(TINY)).clamp_max(1.0))
    out = p * (1 - lr * decay) - up
    return {"p": (out, e_up + 4 * E * (p.abs() + up.abs()) + TINY), "m": (mm, em), "v": (vv, ev)}


def decode(codes, exps, window):
    """What moments in 8 bits stand for."""
    c = codes.to(torch.int64).view(-1, BLOCK)
    size = c if window == 31 else c % 128
    place = size + 8 * (exps.to(torch.int64)[:, None] - window)
    # a float's bits from the 20th on: eight fractions to a binade, subnormal numbers below the first
    value = torch.where(place < 8, place.clamp_min(0).to(F64) * 2.0 ** -129,
                        (8 + (place % 8).to(F64)) * two_to(place // 8 - 130))
    value = torch.where(size == 0, 0.0, value)
    value = torch.where(exps[:, None] == 255, torch.nan, value)
    return (value if window == 31 else torch.where(c >= 128, -value, value)).view(-1)


def steps_of(x, window):
    """(unit, least) of each element of x (64 bits): the distance of numbers of 4 significant bits at x, and the least
    number of its block's window."""
    x = x.abs().view(-1, BLOCK)
    unit = two_to(torch.frexp(x)[1] - 4)
    top = x.amax(1, keepdim=True)
    at = two_to(torch.frexp(top)[1] - 4)
    top = torch.ceil(top / at) * at
    least = 1.125 * two_to(torch.frexp(top)[1] - 1 - window)
    return unit.view(-1), least.expand_as(x).reshape(-1)


def check_small(codes, exps, want, window, what, nearest):
    """Codes of a moment of this value and bound: the number of 4 significant bits next to it (nearest: within half a
    step; else either neighbour), within the block's window."""
    value, bound = want
    got = decode(codes, exps, window)
    unit, least = steps_of(value, window)
    off = (got - value).abs()
    allowed = unit * (0.5 if nearest else 1.0) * (1 + 1e-9) + bound
    inside = value.abs() >= least
    assert (off <= allowed)[inside].all(), f"{what}: {int((off > allowed)[inside].sum())} elements off"
    out = ~inside & (value != 0)
    if window == 31:
        assert (got[out] <= least[out] * 1.125).all() and (got[out] > 0).all(), what
    else:
        assert (got[out].abs() <= least[out] * 1.125).all(), what
    assert (got[value == 0].abs() <= bound.expand_as(value)[value == 0]).all(), what
