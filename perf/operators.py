"""The operators of one pipeline stage, as cases that can be timed and compared.

Three operators, each in its directions:

head   softmax cross entropy of the last stage over a large vocabulary.
       ``head_forward``: loss and log-sum-exp of every token; ``head_step``:
       the same, then the gradients of the activations and of the output matrix.
kept   activation checkpoints in 8 bits.  ``kept_roundtrip``: pack and unpack;
       ``kept_wgrad``: the weight gradient taken from a packed activation,
       added to the microbatches' running sum.
join   the norm after a block, its gate, the residual scale and sum, and the
       norm before the next block.  ``join_forward`` and ``join_backward``.

``run`` computes a case either in plain torch operations in 32 bits or, where
``own`` is true, with the package's ``stage`` calls.
"""
import math

import torch

own = False

#: Columns that share one scale in an 8-bit checkpoint.
BLOCK = 64
EPS = 1e-6


def listed():
    return [
        # one token scored against a small vocabulary: a serving call, all latency and one read of the matrix
        {"name": "head_f_one_token", "op": "head_forward", "T": 1, "V": 32000, "H": 2048, "left_out": 0.0, "weighted": False},
        # evaluation of one microbatch on the last stage
        {"name": "head_f_4096", "op": "head_forward", "T": 4096, "V": 131072, "H": 4096, "left_out": 0.05, "weighted": False},
        # a ragged microbatch with an odd vocabulary, a fifth of its tokens masked and the rest weighted
        {"name": "head_step_ragged", "op": "head_step", "T": 777, "V": 50257, "H": 1000, "left_out": 0.2, "weighted": True},
        # a full training microbatch on the last stage
        {"name": "head_step_8192", "op": "head_step", "T": 8192, "V": 131072, "H": 4096, "left_out": 0.05, "weighted": False},
        # a few odd rows kept: the last, short microbatch of a batch
        {"name": "kept_odd", "op": "kept_roundtrip", "T": 7, "H": 1001},
        # a long microbatch's activation kept from its forward to its backward
        {"name": "kept_16384", "op": "kept_roundtrip", "T": 16384, "H": 8192},
        # the W op of a narrow layer on a short microbatch
        {"name": "wgrad_short", "op": "kept_wgrad", "T": 200, "N": 1024, "H": 1000},
        # the W op of a wide layer
        {"name": "wgrad_8192", "op": "kept_wgrad", "T": 8192, "N": 8192, "H": 8192},
        # one token through a block's end: a serving call, nothing kept
        {"name": "join_f_one_token", "op": "join_forward", "T": 1, "H": 4096, "groups": 1, "alpha": 1.0, "keep": False},
        # a long microbatch's F at a block's end, y and the block's output kept in 8 bits and read back
        {"name": "join_f_16384", "op": "join_forward", "T": 16384, "H": 8192, "groups": 1, "alpha": 0.5, "keep": True},
        # three sequences with a gate each, odd width
        {"name": "join_b_odd", "op": "join_backward", "T": 513, "H": 1001, "groups": 3, "alpha": 0.7, "packed": False},
        # the same long microbatch's B, from the 8-bit checkpoints
        {"name": "join_b_16384", "op": "join_backward", "T": 16384, "H": 8192, "groups": 4, "alpha": 0.5, "packed": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 64, sometimes of 8, sometimes odd."""
    n, to = _spread(rng, lo, hi), rng.choice((64, 64, 64, 8, 1))
    return max(to, n // to * to)


def draw(rng):
    op = rng.choice(("head_forward", "head_step", "kept_roundtrip", "kept_wgrad", "join_forward", "join_backward"))
    c = {"op": op}
    if op in ("head_forward", "head_step"):
        c.update(T=_spread(rng, 1, 8192), V=_spread(rng, 100, 131072), H=_width(rng, 64, 4096),
                 left_out=rng.choice((0.0, 0.05, 0.5)), weighted=op == "head_step" and rng.random() < 0.3)
    elif op == "kept_roundtrip":
        c.update(T=_spread(rng, 1, 16384), H=_width(rng, 64, 8192))
    elif op == "kept_wgrad":
        c.update(T=_spread(rng, 1, 8192), N=_width(rng, 64, 8192), H=_width(rng, 64, 8192))
    else:
        groups = rng.choice((1, 1, 2, 5))
        c.update(T=groups * _spread(rng, 1, 16384 // groups), H=_width(rng, 64, 8192), groups=groups,
                 alpha=rng.choice((1.0, 0.5)))
        c["keep" if op == "join_forward" else "packed"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs

def _two_to(e):
    """2 to the whole number e (-126..126) in 32 bits, without rounding: half of all values of the largest binade are ties."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _kept(x):
    """The 8-bit checkpoint of x [T, H]: whole numbers q [T, H] and one exponent per row and block of columns."""
    T, H = x.shape
    nb = -(-H // BLOCK)
    xp = torch.zeros(T, nb * BLOCK, device=x.device)
    xp[:, :H] = x.float()
    xp = xp.view(T, nb, BLOCK)
    amax = xp.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 7, -126).clamp(-126, 121)
    # the step is a power of two, so that both the division and the values are exact
    q = (xp * _two_to(-e[:, :, None])).round().clamp(-127, 127)
    return q.view(T, nb * BLOCK)[:, :H].to(torch.int8), e.to(torch.int8)


def _values(q, e):
    """What a checkpoint stands for, in 32 bits."""
    return q.float() * _two_to(e).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    op, T, H = case["op"], case["T"], case["H"]
    s = {"case": dict(case)}
    if op in ("head_forward", "head_step"):
        V = case["V"]
        # a normalised activation against rows whose logits are a few units wide, as late in training
        s["x"] = normal(T, H)
        s["w"] = normal(V, H, scale=2.0 / math.sqrt(H))
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        gone = torch.rand(T, generator=g, device="cuda") < case["left_out"]
        s["target"] = torch.where(gone, -100, target)
        s["weight"] = torch.rand(T, generator=g, device="cuda") + 0.5 if case["weighted"] else None
        s["scale"] = 1.0 / T
    elif op == "kept_roundtrip":
        # activations with a few wide channels
        s["x"] = (torch.randn(T, H, generator=g, device="cuda")
                  * torch.exp(1.5 * torch.randn(H, generator=g, device="cuda"))).to(torch.bfloat16)
    elif op == "kept_wgrad":
        N = case["N"]
        s["dy"] = normal(T, N, scale=1e-2)
        s["q"], s["e"] = _kept(normal(T, H))
        s["sum"] = torch.randn(N, H, generator=g, device="cuda") * (1e-2 * math.sqrt(T))
    else:
        s["f"] = normal(T, H, scale=0.3)
        s["w_post"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        s["w_pre"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        s["gate"] = normal(case["groups"], H, scale=0.5)
        s["rows_per_gate"] = T // case["groups"]
        if op == "join_forward":
            s["x"] = normal(T, H, scale=2.0)
        else:
            s["y"] = normal(T, H, scale=2.0)
            s["dh"] = normal(T, H, scale=1e-2)
            s["dy"] = normal(T, H, scale=1e-2)
            for name, of in (("rstd_post", "f"), ("rstd_pre", "y")):
                s[name] = torch.rsqrt(s[of].float().square().mean(1) + EPS)
            if case["packed"]:
                s["f"], s["y"] = _kept(s["f"]), _kept(s["y"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from pipeline_schedule_simulation_gb300 import stage

    c = s["case"]
    op = c["op"]
    if op == "head_forward":
        return stage.head_forward(s["x"], s["w"], s["target"])
    if op == "head_step":
        r = stage.head_forward(s["x"], s["w"], s["target"])
        r.update(stage.head_backward(s["x"], s["w"], s["target"], r["lse"], scale=s["scale"], weight=s["weight"]))
        return r
    if op == "kept_roundtrip":
        return stage.unpack(stage.pack(s["x"]))
    if op == "kept_wgrad":
        # a new tensor, so that the running sum in the state stays what it was
        return stage.weight_grad(s["dy"], stage.Packed(s["q"], s["e"]), add=s["sum"])
    if op == "join_forward":
        r = stage.join_forward(s["x"], s["f"], s["w_post"], s["w_pre"], s["gate"], rows_per_gate=s["rows_per_gate"],
                               alpha=c["alpha"], eps=EPS, keep=c["keep"])
        if c["keep"]:
            r["kept_y"], r["kept_f"] = stage.unpack(r["kept_y"]), stage.unpack(r["kept_f"])
        return r
    y, f = (stage.Packed(*s["y"]), stage.Packed(*s["f"])) if c["packed"] else (s["y"], s["f"])
    return stage.join_backward(s["dh"], s["dy"], y, f, s["rstd_post"], s["rstd_pre"], s["w_post"], s["w_pre"], s["gate"],
                               rows_per_gate=s["rows_per_gate"], alpha=c["alpha"])


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("head_forward", "head_step"):
        x, w, target = s["x"].float(), s["w"].float(), s["target"]
        keep = (target >= 0) & (target < c["V"])
        at = torch.where(keep, target, 0)[:, None]
        logits = x @ w.t()
        top = logits.amax(1, keepdim=True)
        lse = (logits - top).exp().sum(1, keepdim=True).log() + top
        r = {"loss": torch.where(keep, (lse - logits.gather(1, at))[:, 0], 0.0), "lse": lse[:, 0]}
        if op == "head_step":
            d = logits.sub_(lse).exp_()
            d.scatter_add_(1, at, torch.full_like(lse, -1.0))
            row = keep.float() if s["weight"] is None else torch.where(keep, s["weight"], 0.0)
            d.mul_((row * s["scale"])[:, None])
            r["dx"] = (d @ w).to(torch.bfloat16)
            r["dw"] = (d.t() @ x).to(torch.bfloat16)
        return r
    if op == "kept_roundtrip":
        return _values(*_kept(s["x"])).to(torch.bfloat16)
    if op == "kept_wgrad":
        return s["sum"] + s["dy"].float().t() @ _values(s["q"], s["e"])
    w_post, w_pre = s["w_post"].float(), s["w_pre"].float()
    gate = s["gate"].float().repeat_interleave(s["rows_per_gate"], 0)
    if op == "join_forward":
        x, f = s["x"].float(), s["f"].float()
        r1 = torch.rsqrt(f.square().mean(1) + EPS)
        y = c["alpha"] * x + gate * w_post * (f * r1[:, None])
        r2 = torch.rsqrt(y.square().mean(1) + EPS)
        r = {"y": y.to(torch.bfloat16), "h": (y * r2[:, None] * w_pre).to(torch.bfloat16), "rstd_post": r1, "rstd_pre": r2}
        if c["keep"]:
            r["kept_y"] = _values(*_kept(r["y"])).to(torch.bfloat16)
            r["kept_f"] = _values(*_kept(s["f"])).to(torch.bfloat16)
        return r
    y, f = (_values(*s["y"]), _values(*s["f"])) if c["packed"] else (s["y"].float(), s["f"].float())
    dh, dy = s["dh"].float(), s["dy"].float()
    n2 = y * s["rstd_pre"][:, None]
    t = dh * w_pre
    d = dy + s["rstd_pre"][:, None] * (t - n2 * (t * n2).mean(1, keepdim=True))
    n1 = f * s["rstd_post"][:, None]
    t = d * gate * w_post
    df = s["rstd_post"][:, None] * (t - n1 * (t * n1).mean(1, keepdim=True))
    return {"dx": (c["alpha"] * d).to(torch.bfloat16), "df": df.to(torch.bfloat16), "dw_pre": (dh * n2).sum(0),
            "dw_post": (d * gate * n1).sum(0),
            "dgate": (d * n1).view(c["groups"], s["rows_per_gate"], -1).sum(1) * w_post}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, T, H = case["op"], case["T"], case["H"]
    blocks = -(-H // BLOCK)
    kept = T * (H + blocks)  # bytes of one checkpoint
    if op == "head_forward":
        return {"bytes": 2 * T * H + 2 * case["V"] * H + 8 * T + 8 * T, "flops": 2 * T * case["V"] * H}
    if op == "head_step":  # three products; both inputs read and both gradients written
        return {"bytes": 4 * T * H + 4 * case["V"] * H + 16 * T, "flops": 6 * T * case["V"] * H}
    if op == "kept_roundtrip":
        return {"bytes": 4 * T * H + 2 * kept, "flops": 4 * T * H}
    if op == "kept_wgrad":
        return {"bytes": 2 * T * case["N"] + kept + 8 * case["N"] * H, "flops": 2 * T * case["N"] * H}
    if op == "join_forward":
        n = 8 * T * H + 8 * T
        return {"bytes": n + (4 * kept + 4 * T * H if case["keep"] else 0), "flops": 12 * T * H}
    return {"bytes": 8 * T * H + (2 * kept if case["packed"] else 4 * T * H) + 8 * T, "flops": 25 * T * H}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """The outputs from the definitions in 64 bits; None for a case that would take too long."""
    s = prepare(case, seed)
    op, T, H = case["op"], case["T"], case["H"]
    f64 = torch.float64

    def checkpoint(x):
        T_, H_ = x.shape
        v = torch.nn.functional.pad(x.to(f64), (0, -H_ % BLOCK)).reshape(T_, -1, BLOCK)
        a = v.abs().max(2, keepdim=True).values
        # the magnitude with its fraction bits cleared is the power of two below it
        below = (a.view(torch.int64) & (0x7FF << 52)).view(f64)
        step = torch.where(a > 0, below / 64, torch.ones_like(a))
        return ((v / step).round().clamp(-127, 127) * step).reshape(T_, -1)[:, :H_]

    def stands_for(kept):
        q, e = kept
        step = ((e.to(torch.int64) + 1023) << 52).view(f64)
        return torch.cat([q[:, b * BLOCK:(b + 1) * BLOCK].to(f64) * step[:, b:b + 1] for b in range(e.shape[1])], 1)

    if op in ("head_forward", "head_step"):
        V = case["V"]
        if (2 if op == "head_forward" else 8) * T * V * H > 1.5e13:
            return None
        x, target = s["x"].to(f64), s["target"]
        cut = [(a, min(V, a + 16384)) for a in range(0, V, 16384)]
        rows = torch.arange(T, device="cuda")
        inside = target.ge(0) & target.lt(V)
        parts, picked = [], torch.zeros(T, dtype=f64, device="cuda")
        for a, b in cut:
            l = x @ s["w"][a:b].to(f64).t()
            parts.append(torch.logsumexp(l, 1))
            here = inside & (target >= a) & (target < b)
            picked[here] = l[rows[here], target[here] - a]
        lse = torch.logsumexp(torch.stack(parts), 0)
        out = {"loss": (lse - picked) * inside, "lse": lse}
        if op == "head_step":
            c = inside.to(f64) * s["scale"]
            if s["weight"] is not None:
                c = c * s["weight"].to(f64)
            out["dx"] = torch.zeros(T, H, dtype=f64, device="cuda")
            dws = []
            for a, b in cut:
                w = s["w"][a:b].to(f64)
                p = torch.exp(x @ w.t() - lse[:, None])
                here = inside & (target >= a) & (target < b)
                p[rows[here], target[here] - a] -= 1
                p *= c[:, None]
                out["dx"] += p @ w
                dws.append(p.t() @ x)
            out["dw"] = torch.cat(dws)
        return out
    if op == "kept_roundtrip":
        return checkpoint(s["x"])
    if op == "kept_wgrad":
        if 2 * T * case["N"] * H > 1.5e13:
            return None
        total = s["sum"].to(f64)
        return total.addmm_(s["dy"].to(f64).t(), stands_for((s["q"], s["e"])))
    which = torch.arange(T, device="cuda") // s["rows_per_gate"]
    gate, w_post, w_pre = s["gate"].to(f64), s["w_post"].to(f64), s["w_pre"].to(f64)
    if op == "join_forward":
        f = s["f"].to(f64)
        r1 = 1 / torch.sqrt((f * f).sum(1) / H + EPS)
        y = s["x"].to(f64) * case["alpha"] + (gate * w_post)[which] * f * r1[:, None]
        r2 = 1 / torch.sqrt((y * y).sum(1) / H + EPS)
        out = {"y": y, "h": y * w_pre * r2[:, None], "rstd_post": r1, "rstd_pre": r2}
        if case["keep"]:
            out["kept_y"], out["kept_f"] = None, checkpoint(s["f"])  # y is rounded before it is kept
        return out
    # the gradients by the chain rule through each norm's square sum
    y, f = (stands_for(s["y"]), stands_for(s["f"])) if case["packed"] else (s["y"].to(f64), s["f"].to(f64))
    r1, r2, dh = s["rstd_post"].to(f64)[:, None], s["rstd_pre"].to(f64)[:, None], s["dh"].to(f64)
    up = dh * w_pre
    d = s["dy"].to(f64) + up * r2 - y * r2 ** 3 * ((up * y).sum(1, keepdim=True) / H)
    a = (gate * w_post)[which]
    df = d * a * r1 - f * r1 ** 3 * ((d * a * f).sum(1, keepdim=True) / H)
    per = torch.zeros(case["groups"], H, dtype=f64, device="cuda").index_add_(0, which, d * f * r1)
    return {"dx": d * case["alpha"], "df": df, "dw_pre": (dh * y * r2).sum(0), "dw_post": (gate * per).sum(0),
            "dgate": per * w_post}
