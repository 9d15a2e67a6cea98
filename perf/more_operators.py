"""Operators of a stage that learns from the log probabilities of given tokens, as
cases that can be timed and compared.

score  log probabilities of given tokens over a large vocabulary, with the
       entropy and the likeliest alternatives.  ``score_forward``; ``score_step``:
       the same, then the gradients of the activations and of the output matrix.
step   an AdamW step over all tensors of a stage, its moments in 32 or in 8
       bits, with the norm of the gradients and the clip where a case asks.

``run`` computes a case either in plain torch operations in 32 bits or, where
``own`` is true, with the package's ``stage`` calls.
"""
import itertools
import math

import torch

own = False

#: Elements that share one exponent in an 8-bit moment; each tensor's moments start on a multiple of it.
BLOCK = 64
BETAS, EPS, DECAY, LR, CLIP = (0.9, 0.95), 1e-8, 0.1, 3e-4, 1.0


def listed():
    return [
        # one token just sampled: its log probability and what else was likely; serving, one read of the matrix
        {"name": "score_one_token", "op": "score_forward", "T": 1, "V": 32000, "H": 2048, "top": 8, "left_out": 0.0},
        # a short ragged prompt scored against an odd vocabulary
        {"name": "score_ragged", "op": "score_forward", "T": 333, "V": 50257, "H": 1000, "top": 5, "left_out": 0.1},
        # a microbatch of rollouts scored by the reference policy: no alternatives
        {"name": "score_2048", "op": "score_forward", "T": 2048, "V": 131072, "H": 4096, "top": 0, "left_out": 0.05},
        # a full microbatch with as many alternatives as a serving interface gives
        {"name": "score_4096_top", "op": "score_forward", "T": 4096, "V": 131072, "H": 4096, "top": 20, "left_out": 0.05},
        # a policy gradient with an entropy term on a ragged microbatch, a fifth of its tokens the prompt's
        {"name": "score_step_ragged", "op": "score_step", "T": 777, "V": 50257, "H": 1000, "top": 0, "left_out": 0.2},
        # the same on a full training microbatch
        {"name": "score_step_8192", "op": "score_step", "T": 8192, "V": 131072, "H": 4096, "top": 0, "left_out": 0.05},
        # a toy stage: nothing but latency, clip included
        {"name": "step_toy", "op": "step", "blocks": 2, "H": 128, "V": 300, "par": "copied", "grad": "float", "bits": 32,
         "clip": True, "random": False},
        # many odd tensors of a deep narrow stage, all in 16 bits, moments in 8, rounded at random
        {"name": "step_odd_8", "op": "step", "blocks": 40, "H": 1001, "V": 50257, "par": "bf16", "grad": "bf16", "bits": 8,
         "clip": False, "random": True},
        # a stage without an output matrix: 32-bit parameters alone, gradients as an all-reduce in 16 bits leaves them
        {"name": "step_blocks_32", "op": "step", "blocks": 12, "H": 2048, "V": 0, "par": "float", "grad": "bf16", "bits": 32,
         "clip": False, "random": False},
        # the last stage after its flush: 32-bit parameters with the 16-bit copies that the next batch runs on
        {"name": "step_stage_32", "op": "step", "blocks": 2, "H": 4096, "V": 131072, "par": "copied", "grad": "float", "bits": 32,
         "clip": True, "random": False},
        # the same with the moments in 8 bits
        {"name": "step_stage_8", "op": "step", "blocks": 2, "H": 4096, "V": 131072, "par": "copied", "grad": "float", "bits": 8,
         "clip": True, "random": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 64, sometimes of 8, sometimes odd."""
    n, to = _spread(rng, lo, hi), rng.choice((64, 64, 64, 8, 1))
    return max(to, n // to * to)


def draw(rng):
    op = rng.choice(("score_forward", "score_step", "step", "step"))
    if op == "step":
        H = _width(rng, 64, 4096)
        V = rng.choice((0, _spread(rng, 100, 131072)))
        # as many blocks as leave the whole no larger than the largest listed stage
        most = (570_000_000 - V * H) // (H * (H + 3))
        return {"op": op, "blocks": _spread(rng, 1, max(1, min(60, most))), "H": H, "V": V,
                "par": rng.choice(("float", "copied", "bf16")), "grad": rng.choice(("float", "bf16")), "bits": rng.choice((8, 32)),
                "clip": rng.random() < 0.5, "random": rng.random() < 0.5}
    c = {"op": op, "T": _spread(rng, 1, 8192), "V": _spread(rng, 100, 131072), "H": _width(rng, 64, 4096),
         "top": rng.choice((0, 1, 5, 8, 20)), "left_out": rng.choice((0.0, 0.05, 0.5))}
    if c["T"] * c["V"] * c["H"] > 4096 * 131072 * 4096:
        c["top"] = 0
    return c


# ---------------------------------------------------------------- inputs

def _sizes(c):
    """Elements of each tensor of a stage: its blocks' matrix, two norms and gate, then the output matrix."""
    return [c["H"] * c["H"], c["H"], c["H"], c["H"]] * c["blocks"] + ([c["V"] * c["H"]] if c["V"] else [])


def _starts(sizes):
    """Where each tensor starts, on multiples of a block, and where all of them end."""
    at = list(itertools.accumulate((-(-n // BLOCK) * BLOCK for n in sizes), initial=0))
    return at[:-1], at[-1]


def _grid(x):
    """Whole numbers within +-31, in the distribution of 8 times x."""
    return (x * 8).round().clamp(-31, 31)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": dict(case)}
    if case["op"] != "step":
        T, V, H = case["T"], case["V"], case["H"]
        # A normalised activation against rows whose logits are a few units wide, as late in training, both on a grid of
        # powers of two: a logit is then the same whichever way it is summed up, and which alternative comes first is the
        # operator's affair and not that of a rounding.
        s["x"] = (_grid(normal(T, H)) / 8).to(torch.bfloat16)
        s["w"] = (_grid(normal(V, H)) * 2.0 ** round(math.log2(0.25 / math.sqrt(H)))).to(torch.bfloat16)
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        s["target"] = torch.where(torch.rand(T, generator=g, device="cuda") < case["left_out"], -100, target)
        if case["op"] == "score_step":
            s["dlogp"] = -normal(T) / T           # a policy gradient: minus the advantage
            s["dentropy"] = torch.full((T,), -0.01 / T, device="cuda")
        return s
    sizes = _sizes(case)
    at, total = _starts(sizes)
    ends = torch.tensor(at, device="cuda") + torch.tensor(sizes, device="cuda")
    s["tensor"] = torch.repeat_interleave(torch.tensor([b - a for a, b in zip(at, at[1:] + [total])], device="cuda"))
    flat = torch.arange(total, device="cuda") < ends[s["tensor"]]  # what is not padding

    def buffer(scale, dtype=torch.float32):
        return (normal(total) * scale * flat).to(dtype)

    wide = case["par"] != "bf16"
    s["p"] = buffer(0.02, torch.float32 if wide else torch.bfloat16)
    s["copy"] = s["p"].to(torch.bfloat16) if case["par"] == "copied" else None
    # gradients of channels of different width, the norm a few units
    width = torch.exp(1.5 * normal(-(-total // 1024))).repeat_interleave(1024)[:total]
    s["g"] = (buffer(2.0 / math.sqrt(total)) * width).to(torch.float32 if case["grad"] == "float" else torch.bfloat16)
    m = buffer(0.5 / math.sqrt(total)) * width
    v = (buffer(1.0 / math.sqrt(total)) * width).square() + (1e-2 / math.sqrt(total) * width).square() * flat
    s["m"], s["v"] = (m, v) if case["bits"] == 32 else (_encode(m, 15, None), _encode(v, 31, None))
    s["step"] = torch.full((1,), 100, dtype=torch.int64, device="cuda")
    # matrices decay, vectors do not
    s["decay"] = [DECAY if n > case["H"] else 0.0 for n in sizes]
    s["decays"] = torch.tensor(s["decay"], device="cuda")
    s["seed"] = seed + 1 if case["random"] else None
    if own:
        from pipeline_schedule_simulation_gb300 import stage

        def views(t):
            return [t[a:a + n] for a, n in zip(at, sizes)]

        state = {"m": s["m"], "v": s["v"]} if case["bits"] == 32 else {
            "m": s["m"][0], "m_exp": s["m"][1], "v": s["v"][0], "v_exp": s["v"][1]}
        s["grads"] = views(s["g"])
        s["opt"] = stage.AdamW(views(s["p"]), bits=case["bits"], copies=None if s["copy"] is None else views(s["copy"]),
                               betas=BETAS, eps=EPS, weight_decay=s["decay"], seed=s["seed"],
                               state={**state, "step": s["step"]})
    return s


# ---------------------------------------------------------------- moments in 8 bits

def _decode(codes, exps, window):
    """What codes stand for, in 32 bits: the float whose bits from the 20th on are the code, counted from the block's window."""
    c = codes.view(-1, BLOCK).int()
    size = c if window == 31 else c & 127
    bits = (size + (exps.int()[:, None] - window) * 8).clamp_min(0) << 20
    value = torch.where(size > 0, bits, 0).view(torch.float32)
    value = torch.where(exps[:, None] == 255, torch.nan, value)
    return (value if window == 31 else torch.where(c > 127, -value, value)).view(-1)


def _encode(x, window, draws):
    """(codes, one exponent for each block) of a moment: 3 bits of the fraction are kept, the exponent is held relative to the
    block's.  draws: 16 random bits for each element, None to round to nearest."""
    bits = x.abs().view(torch.int32).view(-1, BLOCK)
    top = bits.amax(1)
    exps = torch.where(top >= 0x7F800000, 255, ((top + 0xFFFFF) >> 23).clamp_max(254))
    r = 0x80000 if draws is None else (draws.view(-1, BLOCK).int() << 4) + 8
    size = ((bits + r) >> 20) - (exps[:, None] - window) * 8
    if window == 31:  # a second moment that is not 0 is never held as 0
        size = torch.where(bits > 0, size.clamp(1, 255), 0)
    else:
        size = size.clamp(0, 127) + torch.where(x.view(-1, BLOCK) < 0, 128, 0)
    return torch.where(exps[:, None] == 255, 0, size).to(torch.uint8).view(-1), exps.to(torch.uint8)


def _mix(x):
    """32 bits mixed: multiplications and shifts."""
    x = ((x ^ (x >> 16)) * 0x243F6A89) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x85A308D3) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _draws(total, seed, step):
    """32 random bits for each element, and 16 more."""
    at = torch.arange(total // BLOCK, device="cuda")
    key = _mix((at & 0xFFFFFFFF) ^ _mix((step & 0xFFFFFFFF) ^ _mix((seed & 0xFFFFFFFF) ^ _mix(torch.full_like(step, seed >> 32)))))
    x = (key[:, None] + torch.arange(BLOCK, device="cuda") * 0x9E3779B1) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x13198A2F) & 0xFFFFFFFF
    x = ((x ^ (x >> 12)) * 0xA4093823) & 0xFFFFFFFF
    x = (x ^ (x >> 15)).view(-1)
    return x, (x * 0x299F31D1 & 0xFFFFFFFF) >> 16


# ---------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from pipeline_schedule_simulation_gb300 import stage

    c = s["case"]
    if c["op"] == "step":
        norm = stage.grad_norm(s["grads"]) if c["clip"] else None
        s["opt"].step(s["grads"], LR, norm=norm, max_norm=CLIP if c["clip"] else None)
        m, v = s["opt"].moments()
        return {"p": s["p"], "copy": s["copy"], "m": m, "v": v, "norm": norm}
    r = stage.score_forward(s["x"], s["w"], s["target"], top=c["top"])
    if c["op"] == "score_step":
        r.update(stage.score_backward(s["x"], s["w"], s["target"], r["lse"], s["dlogp"], entropy=r["entropy"],
                                      dentropy=s["dentropy"]))
    return r


def _run_plain(s):
    c = s["case"]
    if c["op"] == "step":
        return _step_plain(s)
    x, w, target = s["x"].float(), s["w"].float(), s["target"]
    keep = (target >= 0) & (target < c["V"])
    at = torch.where(keep, target, 0)[:, None]
    logits = x @ w.t()
    largest = logits.amax(1, keepdim=True)
    lse = (logits - largest).exp().sum(1, keepdim=True).log() + largest
    r = {"logp": torch.where(keep, (logits.gather(1, at) - lse)[:, 0], 0.0), "lse": lse[:, 0]}
    if c["top"]:
        # sorted in a stable way, so that of equal logits the lowest index comes first
        found = torch.sort(logits, dim=1, descending=True, stable=True)
        r["top_logp"], r["top_index"] = found.values[:, :c["top"]] - lse, found.indices[:, :c["top"]].contiguous()
        del found
    logits.sub_(lse)
    p = logits.exp()
    r["entropy"] = -(p * logits).sum(1)
    if c["op"] == "score_step":
        a = torch.where(keep, s["dlogp"], 0.0)[:, None]
        b = torch.where(keep, s["dentropy"], 0.0)[:, None]
        d = logits.add_(r["entropy"][:, None]).mul_(-b).sub_(a).mul_(p)
        del p
        d.scatter_add_(1, at, a)
        r["dx"] = (d @ w).to(torch.bfloat16)
        r["dw"] = (d.t() @ x).to(torch.bfloat16)
    return r


def _step_plain(s):
    c = s["case"]
    small, (b1, b2) = c["bits"] == 8, BETAS
    s["step"] += 1
    t = s["step"].double()
    g, norm = s["g"].float(), None
    if c["clip"]:
        norm = g.double().square().sum().sqrt().view(1)  # a long sum
        g = g * torch.where(norm > CLIP, CLIP / norm, 1.0).float()
        norm = norm.float()
    m, v = (_decode(*s["m"], 15), _decode(*s["v"], 31)) if small else (s["m"], s["v"])
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * (g * g)
    size = (LR / (1 - b1 ** t)).float()
    p = s["p"].float() * (1 - LR * s["decays"])[s["tensor"]]
    p = p - size * m / (v.sqrt() / (1 - b2 ** t).sqrt().float() + EPS)
    draws, more = _draws(p.numel(), s["seed"], s["step"]) if c["random"] else (None, None)
    if c["par"] == "bf16" and c["random"]:
        # the magnitude's bits beyond bf16 become a carry at random
        s["p"].copy_(((p.view(torch.int32) + more.int()) & -65536).view(torch.float32))
    else:
        s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if small:
        # held as the next pass finds them
        s["m"] = _encode(m, 15, None if draws is None else draws & 0xFFFF)
        s["v"] = _encode(v, 31, None if draws is None else draws >> 16)
        m, v = _decode(*s["m"], 15).to(torch.bfloat16), _decode(*s["v"], 31).to(torch.bfloat16)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
        m, v = s["m"], s["v"]
    return {"p": s["p"], "copy": s["copy"], "m": m, "v": v, "norm": norm}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "step":
        n = sum(_sizes(case))
        wide, grad, small = case["par"] != "bf16", 4 if case["grad"] == "float" else 2, case["bits"] == 8
        b = (8 if wide else 4) + grad * (2 if case["clip"] else 1) + (2 if case["par"] == "copied" else 0)
        # moments read and written; those in 8 bits also returned as 16-bit values
        b += 4 + 4 / BLOCK + 4 if small else 16
        return {"bytes": b * n, "flops": (16 + (2 if case["clip"] else 0)) * n}
    T, V, H = case["T"], case["V"], case["H"]
    if case["op"] == "score_forward":
        return {"bytes": 2 * T * H + 2 * V * H + 8 * T + 12 * T + 12 * T * case["top"], "flops": 2 * T * V * H}
    # three products; both inputs read and both gradients written
    return {"bytes": 4 * T * H + 4 * V * H + 28 * T + 12 * T * case["top"], "flops": 6 * T * V * H}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """The outputs from the definitions in 64 bits; None for a case that would take too long."""
    s = prepare(case, seed)
    return _exact_step(s) if case["op"] == "step" else _exact_score(s)


def _exact_score(s):
    c, f64 = s["case"], torch.float64
    T, V, H, k = c["T"], c["V"], c["H"], c["top"]
    if (2 if c["op"] == "score_forward" else 8) * T * V * H > 1.5e13:
        return None
    x, target = s["x"].to(f64), s["target"]
    cut = [(a, min(V, a + 8192)) for a in range(0, V, 8192)]
    inside = target.ge(0) & target.lt(V)
    rows = torch.arange(T, device="cuda")
    picked = torch.zeros(T, dtype=f64, device="cuda")
    lses, best, which = [], None, None
    for a, b in cut:
        l = x @ s["w"][a:b].to(f64).t()
        lses.append(torch.logsumexp(l, 1))
        here = inside & (target >= a) & (target < b)
        picked[here] = l[rows[here], target[here] - a]
        if k:
            # those found so far stand first: equal logits keep the order of their indices
            index = torch.arange(a, b, device="cuda").expand(T, b - a)
            both, index = (l, index) if best is None else (torch.cat([best, l], 1), torch.cat([which, index], 1))
            order = torch.argsort(both, dim=1, descending=True, stable=True)[:, :k]
            best, which = both.gather(1, order), index.gather(1, order)
    lse = torch.logsumexp(torch.stack(lses), 0)
    out = {"logp": (picked - lse) * inside, "lse": lse}
    if k:
        out["top_logp"], out["top_index"] = best - lse[:, None], which
    ent = torch.zeros(T, dtype=f64, device="cuda")
    for a, b in cut:
        q = x @ s["w"][a:b].to(f64).t() - lse[:, None]
        ent -= (q.exp() * q).sum(1)
    out["entropy"] = ent
    if c["op"] == "score_step":
        gl, ge = s["dlogp"].to(f64) * inside, s["dentropy"].to(f64) * inside
        dx, dw = torch.zeros(T, H, dtype=f64, device="cuda"), []
        for a, b in cut:
            w = s["w"][a:b].to(f64)
            q = x @ w.t() - lse[:, None]
            d = -q.exp() * (gl[:, None] + ge[:, None] * (q + ent[:, None]))
            here = inside & (target >= a) & (target < b)
            d[rows[here], target[here] - a] += gl[here]
            dx += d @ w
            dw.append(d.t() @ x)
        out["dx"], out["dw"] = dx, torch.cat(dw)
    return out


def _exact_step(s):
    c, f64 = s["case"], torch.float64
    b1, b2 = BETAS
    t = int(s["step"]) + 1

    def two_to(e):
        return ((e.to(torch.int64) + 1023) << 52).view(f64)

    def held(moment, window):
        """What an 8-bit moment stands for."""
        codes, exps = moment
        n = codes.view(-1, BLOCK).to(torch.int64)
        size = n if window == 31 else n % 128
        place = size + 8 * (exps.to(torch.int64)[:, None] - window)
        value = (1 + (place % 8).to(f64) / 8) * two_to(place // 8 - 127)
        value = torch.where(size == 0, torch.zeros_like(value), value)
        return (torch.where(n >= 128, -value, value) if window == 15 else value).view(-1)

    def keep(x, window, u):
        """x rounded to 4 significant bits, up with the probability of what is cut off, within the block's window."""
        x = x.view(-1, BLOCK)
        e = torch.frexp(x)[1] - 1
        unit = two_to(e - 3)
        size = torch.floor(x.abs() / unit + u.view(-1, BLOCK)) * unit
        top = x.abs().amax(1, keepdim=True)
        unit = two_to(torch.frexp(top)[1] - 4)
        least = 1.125 * two_to(torch.frexp(torch.ceil(top / unit) * unit)[1] - 1 - window)
        size = torch.where(size < least, least if window == 31 else torch.zeros_like(least), size)
        size = torch.where(x == 0, torch.zeros_like(size), size)
        return torch.where(x < 0, -size, size).view(-1)

    g = s["g"].to(f64)
    out = {"p": None, "copy": None, "norm": None}
    if c["clip"]:
        out["norm"] = torch.linalg.vector_norm(g).view(1)
        g = g * min(1.0, CLIP / float(out["norm"]))
    m, v = (held(s["m"], 15), held(s["v"], 31)) if c["bits"] == 8 else (s["m"].to(f64), s["v"].to(f64))
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g ** 2 * (1 - b2)
    p = s["p"].to(f64)
    p = p - LR * (m / (1 - b1 ** t) / ((v / (1 - b2 ** t)) ** 0.5 + EPS) + s["decays"].to(f64)[s["tensor"]] * p)
    del g
    low, more = _draws(p.numel(), s["seed"], s["step"] + 1) if c["random"] else (None, None)
    if c["par"] == "bf16" and c["random"]:
        unit = two_to(torch.frexp(p)[1] - 8)
        out["p"] = torch.where(p == 0, p, torch.sign(p) * torch.floor(p.abs() / unit + more / 65536) * unit)
    else:
        out["p"] = p
    out["copy"] = p if s["copy"] is not None else None
    if c["bits"] == 8:
        half = torch.full((), 0.5, dtype=f64, device="cuda").expand(p.numel())
        um, uv = (half, half) if low is None else (((low & 0xFFFF) + 0.5) / 65536, ((low >> 16) + 0.5) / 65536)
        m, v = keep(m, 15, um), keep(v, 31, uv)
    out["m"], out["v"] = m, v
    return out
