"""The AdamW step over the tensors of a stage and the norm of its gradients
(stage.AdamW, stage.grad_norm) against the definitions in 64 bits."""
import math

import pytest
import torch

import stage_ref as R
import step_ref as Q

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


def _random(g, n, dtype, scale=1.0, offset=0):
    buf = torch.full((n + offset + 3,), 7.0, dtype=dtype, device="cuda")
    buf[offset:offset + n] = (torch.randn(n, generator=g, device="cuda") * scale).to(dtype)
    return buf, buf[offset:offset + n]


# lengths around a lane's 8 elements, a block's 64 and a thread block's 2048; and offsets that break every alignment
SIZES = [0, 1, 7, 8, 63, 64, 65, 2047, 2048, 2049, 5000, 100003, 256, 1]
OFFSETS = [0, 1, 0, 3, 8, 0, 5, 0, 1, 16, 2, 0, 4, 1]


class Many:
    """Tensors of all lengths inside larger buffers, and what a step makes of them."""

    def __init__(self, S, p_dtype, g_dtype, bits, copied=False, seed=None, steps=0, **kw):
        g = R.generator(3)
        self.buffers, self.params, self.copies, self.grads = [], [], [], []
        for n, o in zip(SIZES, OFFSETS):
            b, p = _random(g, n, p_dtype, 0.02, o)
            self.params.append(p)
            self.buffers.append((b, p, o, n))
            if copied:
                b, c = _random(g, n, BF16, 1.0, o)
                self.copies.append(c)
                self.buffers.append((b, c, o, n))
            self.grads.append(_random(g, n, g_dtype, 1e-3, o)[1])
        self.decay = [0.1 * (i % 3) for i in range(len(SIZES))]
        self.kw = dict(betas=(0.9, 0.95), eps=1e-8)
        self.opt = S.AdamW(self.params, bits=bits, copies=self.copies if copied else None, weight_decay=self.decay, seed=seed,
                           **self.kw, **kw)
        self.starts, at = [], 0
        for n in SIZES:
            self.starts.append(at)
            at += -(-n // 64) * 64
        self.total = at

    def flat(self, tensors):
        out = torch.zeros(self.total, dtype=R.F64, device="cuda")
        for t, a, n in zip(tensors, self.starts, SIZES):
            out[a:a + n] = t.double()
        return out

    def moments(self):
        s = self.opt.state
        if self.opt.bits == 32:
            return s["m"].double(), s["v"].double()
        return Q.decode(s["m"], s["m_exp"], 15), Q.decode(s["v"], s["v_exp"], 31)

    def want(self, t, lr, clip=1.0, grads=None):
        decay = self.flat([torch.full((n,), d) for n, d in zip(SIZES, self.decay)])
        m, v = self.moments()
        return Q.step(self.flat(self.params), self.flat(grads or self.grads), m, v, t, lr, self.kw["betas"], self.kw["eps"],
                      decay, clip)

    def check(self, want, seed=None):
        torch.cuda.synchronize()
        p, bound = want["p"]
        if self.params[0].dtype is BF16:
            # to nearest: half a step; at random: less than one, of either neighbour
            bound = bound + (Q.U16 if seed is None else 2 * Q.U16) * p.abs() * (1 + 1e-6) + R.TINY
        R.check(self.flat(self.params), (p, bound), "p")
        if self.copies:
            R.check(self.flat(self.copies), (p, want["p"][1] + Q.U16 * p.abs() + R.TINY), "copy")
        s = self.opt.state
        if self.opt.bits == 32:
            R.check(s["m"], want["m"], "m")
            R.check(s["v"], want["v"], "v")
        else:
            Q.check_small(s["m"], s["m_exp"], want["m"], 15, "m", seed is None)
            Q.check_small(s["v"], s["v_exp"], want["v"], 31, "v", seed is None)
        for b, view, o, n in self.buffers:  # nothing beside the tensors
            assert (b[:o] == 7).all() and (b[o + n:] == 7).all()


@pytest.mark.parametrize("p_dtype,copied", [(F32, False), (F32, True), (BF16, False)])
@pytest.mark.parametrize("g_dtype", [F32, BF16])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("seed", [None, 12345678901])
def test_steps(S, p_dtype, copied, g_dtype, bits, seed):
    """Three steps from nothing, each against the definition from what the one before it left."""
    many = Many(S, p_dtype, g_dtype, bits, copied, seed)
    for t in range(1, 4):
        want = many.want(t, 1e-2)
        many.opt.step(many.grads, 1e-2)
        many.check(want, seed)
        assert int(many.opt.state["step"]) == t
    m, v = many.opt.moments()
    for got, want in zip((m, v), many.moments()):
        assert torch.equal(got.double(), want)


@pytest.mark.parametrize("bits", [8, 32])
def test_tensors_of_all_types_at_once(S, bits):
    g = R.generator(4)
    kinds = [(a, b, c) for a in (F32, BF16) for b in (F32, BF16) for c in (False, True) if a is F32 or not c] * 120
    params = [_random(g, 70 + i % 130, a, 0.02)[1] for i, (a, _, _) in enumerate(kinds)]
    grads = [_random(g, 70 + i % 130, b, 1e-3)[1] for i, (_, b, _) in enumerate(kinds)]
    copies = [torch.empty_like(p, dtype=BF16) if c else None for p, (_, _, c) in zip(params, kinds)]
    old = [p.clone() for p in params]
    opt = S.AdamW(params, bits=bits, copies=copies, weight_decay=0.1)  # 720 tensors: more than one launch takes
    assert len(params) > 640
    opt.step(grads, 1e-2)
    for p, c, q, x in zip(params, copies, old, grads):
        z = torch.zeros(p.numel(), device="cuda")
        want, bound = Q.step(q, x, z, z, 1, 1e-2, (0.9, 0.999), 1e-8, 0.1)["p"]
        R.check(p, (want, bound + (Q.U16 * want.abs() if p.dtype is BF16 else 0)), "p")
        if c is not None:
            assert torch.equal(c, p.to(BF16))


@pytest.mark.parametrize("bits", [8, 32])
def test_clip_and_norm(S, bits):
    many = Many(S, F32, BF16, bits)
    norm = S.grad_norm(many.grads)
    true = many.flat(many.grads).square().sum().sqrt()
    assert abs(norm.double() - true) <= 1e-6 * true
    for max_norm in (float(true) / 3, float(true) * 3):
        want = many.want(int(many.opt.state["step"]) + 1, 1e-2, min(1.0, max_norm / float(norm)))
        many.opt.step(many.grads, 1e-2, norm=norm, max_norm=max_norm)
        many.check(want)


def test_a_norm_that_was_changed_counts_as_it_is(S):
    """What a norm was before its rounding is used only while it rounds to what the tensor holds."""
    def run(change):
        p, g = torch.ones(100, device="cuda"), torch.linspace(1, 2, 100, device="cuda")
        opt = S.AdamW([p], eps=1.0)
        norm = change(S.grad_norm([g]))
        opt.step([g], 1.0, norm=norm, max_norm=1.0)
        return p, norm

    def doubled(norm):
        return norm.mul_(2)

    p, norm = run(doubled)
    q, _ = run(lambda norm: torch.full_like(norm, 2 * float(norm)))
    assert torch.equal(p, q)
    r, _ = run(lambda norm: norm)
    assert not torch.equal(p, r)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("value", [math.nan, math.inf, 1e30])
def test_a_norm_that_is_no_number_changes_nothing(S, bits, value):
    many = Many(S, F32, F32, bits, copied=True, seed=5)
    many.opt.step(many.grads, 1e-2)
    before = [b.clone() for b, *_ in many.buffers] + [t.clone() for t in many.opt.state.values()]
    many.grads[6][10] = value
    norm = S.grad_norm(many.grads)
    assert not torch.isfinite(norm).any()
    many.opt.step(many.grads, 1e-2, norm=norm, max_norm=1.0)
    after = [b for b, *_ in many.buffers] + list(many.opt.state.values())
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    many.grads[6][10] = 0
    want = many.want(2, 1e-2)
    many.opt.step(many.grads, 1e-2)
    many.check(want, 5)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_gradient_that_is_no_number_stays_in_its_block(S, bits, value):
    many = Many(S, F32, F32, bits)
    many.grads[10][100] = value  # of 5000
    want = many.want(1, 1e-2)
    many.opt.step(many.grads, 1e-2)
    first = 64 if bits == 8 else 100
    bad = torch.zeros(many.total, dtype=torch.bool, device="cuda")
    a = many.starts[10]
    bad[a + first:a + (128 if bits == 8 else 101)] = True
    m, v = many.moments()
    assert m[bad].isnan().all() if bits == 8 else not m[bad].isfinite().any()
    p = many.flat(many.params)
    assert p[a + 100].isnan()
    bad[a + 100] = True
    p_ok = torch.ones_like(bad)
    p_ok[a + 100] = False
    R.check(p[p_ok], (want["p"][0][p_ok], want["p"][1][p_ok]))
    assert torch.isfinite(m[~bad]).all() and torch.isfinite(v[~bad]).all()


def test_gradients_of_zero_and_small_ones(S):
    """m and v of 0 make no step; a v that its block's largest outweighs by more than 31 binades is not held as 0."""
    for bits in (8, 32):
        p = torch.ones(256, device="cuda")
        opt = S.AdamW([p], bits=bits)
        opt.step([torch.zeros(256, device="cuda")], 1e-2)
        assert (p == 1).all() and (opt.moments()[0] == 0).all() and (opt.moments()[1] == 0).all()
    p, g = torch.zeros(64, device="cuda"), torch.full((64,), 1e-12, device="cuda")
    g[0], g[1] = 1e3, -1e-18
    opt = S.AdamW([p], bits=8, eps=0.0)
    opt.step([g], 1e-2)
    m, v = opt.moments()
    assert (v > 0).all() and m[0] > 0 and (m[1:] == 0).all()
    g.zero_()
    q = p.clone()
    opt.step([g], 1e-2)
    assert torch.isfinite(p).all() and (p - q).abs().max() <= 1e-2 * 10
    # gradients whose squares are no normal numbers
    p, g = torch.zeros(64, device="cuda"), torch.linspace(1e-24, 1e-20, 64, device="cuda")
    opt = S.AdamW([p], bits=8)
    opt.step([g], 1e-2)
    m, v = opt.moments()
    want = Q.step(torch.zeros(64, device="cuda"), g, torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda"), 1, 1e-2,
                  (0.9, 0.999), 1e-8, 0.0)
    assert ((m.double() - want["m"][0]).abs() <= want["m"][0] * 2 ** -4 + 1e-30).all()
    assert ((v.double() - want["v"][0]).abs() <= want["v"][0] * 2 ** -4 + 2.0 ** -129).all()


@pytest.mark.parametrize("what", ["m", "v", "p"])
def test_random_rounding_is_right_on_average(S, what):
    """65536 elements of one value: each becomes one of its two neighbours, and their mean is the value to within 5
    deviations (half a step over the root of their number) and the 2^-17 of a step that 16 random bits resolve."""
    n = 65536
    p = torch.full((n,), 0.7, device="cuda").to(BF16)
    g = torch.full((n,), 0.37, device="cuda")
    opt = S.AdamW([p], bits=8, seed=9, betas=(0.9, 0.99))
    opt.step([g], 0.01)
    x, unit = {"m": (0.1 * 0.37, 2.0 ** -8), "v": (0.01 * 0.37 ** 2, 2.0 ** -13),
               "p": (float(torch.tensor(0.7).to(BF16)) - 0.01, 2.0 ** -8)}[what]
    got = {"m": opt.moments()[0], "v": opt.moments()[1], "p": p}[what].double()
    lo = math.floor(x / unit) * unit
    assert ((got - lo).abs() < 1e-12).logical_or((got - lo - unit).abs() < 1e-12).all() and got.unique().numel() == 2
    share = x / unit - math.floor(x / unit)
    slack = unit * (5 * math.sqrt(share * (1 - share) / n) + 2 ** -16) + 1e-6 * x
    assert abs(float(got.mean()) - x) <= slack
    # by place: the first and second half of each block alike, and neighbours independent
    up = (got > lo + unit / 2).double()
    assert abs(float(up.view(-1, 64)[:, :32].mean() - up.view(-1, 64)[:, 32:].mean())) <= 5 * math.sqrt(4 * share * (1 - share) / n)
    both = float((up[1:] * up[:-1]).mean())
    assert abs(both - share ** 2) <= 6 / math.sqrt(n)


def test_small_changes_move_moments_on_average(S):
    """v of 1 under gradients of 0 with beta2 = 0.999: 0.999^200 after 200 steps, on average (nearest: still 1).  Of
    65536 elements that each lose or keep a whole step of 1/16 to 1/8 the mean is off by less than 0.01."""
    n = 65536
    for seed, want in ((1, 0.999 ** 200), (None, 1.0)):
        state = {"m": torch.zeros(n, dtype=torch.uint8, device="cuda"), "v": torch.full((n,), 248, dtype=torch.uint8, device="cuda"),
                 "m_exp": torch.zeros(n // 64, dtype=torch.uint8, device="cuda"),
                 "v_exp": torch.full((n // 64,), 127, dtype=torch.uint8, device="cuda"),
                 "step": torch.zeros(1, dtype=torch.int64, device="cuda")}
        opt = S.AdamW([torch.zeros(n, device="cuda")], bits=8, seed=seed, state=state)
        assert (opt.moments()[1] == 1).all()
        g = torch.zeros(n, device="cuda")
        for _ in range(200):
            opt.step([g], 1e-3)
        assert abs(float(opt.moments()[1].double().mean()) - want) < 0.01


def test_random_bits_depend_on_seed_and_step_alone(S):
    def run(seed, steps, split=False):
        p = torch.full((5000,), 0.7, device="cuda").to(BF16)
        g = torch.linspace(-1, 1, 5000, device="cuda")
        opt = S.AdamW([p], bits=8, seed=seed)
        for i in range(steps):
            if split and i == 1:
                opt = S.AdamW([p], bits=8, seed=seed, state=opt.state)  # from a checkpoint
            opt.step([g], 1e-2)
        return [p, *opt.state.values()]

    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    assert same(run(3, 3), run(3, 3)) and same(run(3, 3), run(3, 3, split=True))
    for other in (4, 3 + (1 << 32), 0):
        assert not same(run(3, 3), run(other, 3))
    a, b = run(3, 1), run(3, 2)
    assert not torch.equal(a[1], b[1])


def test_captured_steps_count_on(S):
    """A step with its norm, captured once and replayed: numbers, random bits and a learning rate on the device go on as
    in calls made one by one.  Two captured steps share no memory."""
    def make():
        g = R.generator(6)
        return Many(S, F32, F32, 8, copied=True, seed=77), torch.full((1,), 1e-2, device="cuda")

    one, lr = make()
    two, lr2 = make()
    third, lr3 = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for m, rate in ((two, lr2), (third, lr3)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            m.opt.step(m.grads, rate, norm=S.grad_norm(m.grads), max_norm=0.05)
        graphs.append(graph)
    torch.cuda.synchronize()
    assert int(two.opt.state["step"]) == 0
    for i in range(4):
        for m, rate in ((one, lr), (two, lr2), (third, lr3)):
            rate.fill_(1e-2 / (i + 1))
            m.grads[11].mul_(1.5)
        torch.cuda.synchronize()
        one.opt.step(one.grads, lr, norm=S.grad_norm(one.grads), max_norm=0.05)
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
    for m in (two, third):
        assert int(m.opt.state["step"]) == 4
        for a, b in zip([b for b, *_ in one.buffers] + list(one.opt.state.values()),
                        [b for b, *_ in m.buffers] + list(m.opt.state.values())):
            assert torch.equal(a, b)


@pytest.mark.parametrize("given", [False, True])
def test_a_captured_step_follows_a_norm_that_is_computed_outside(S, given):
    """Only the step is captured; before each replay grad_norm writes the same tensor, and what it was before its
    rounding where the step reads it: all as in calls one by one, to the last bit."""
    def make():
        return Many(S, F32, F32, 8, copied=True, seed=77)

    one, two = make(), make()
    norm = S.grad_norm(two.grads, out=torch.empty(1, device="cuda") if given else None)
    wide = norm._wide
    at = wide.data_ptr()
    del wide
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        two.opt.step(two.grads, 1e-2, norm=norm, max_norm=0.05)
    for i in range(4):
        for m in (one, two):
            m.grads[11].mul_(1.37)
        assert S.grad_norm(two.grads, out=norm) is norm and norm._wide.data_ptr() == at
        torch.cuda.empty_cache()
        graph.replay()
        one.opt.step(one.grads, 1e-2, norm=S.grad_norm(one.grads), max_norm=0.05)
        torch.cuda.synchronize()
        for a, b in zip([b for b, *_ in one.buffers] + list(one.opt.state.values()),
                        [b for b, *_ in two.buffers] + list(two.opt.state.values())):
            assert torch.equal(a, b)


def test_other_stream_and_current_device(S):
    many, plain = Many(S, F32, F32, 8, seed=1), Many(S, F32, F32, 8, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = S.grad_norm(many.grads, stream=side)
    many.opt.step(many.grads, 1e-2, norm=norm, max_norm=0.01, stream=side)
    m, v = many.opt.moments(stream=side)
    plain.opt.step(plain.grads, 1e-2, norm=S.grad_norm(plain.grads), max_norm=0.01)
    torch.cuda.synchronize()
    for a, b in zip(many.params, plain.params):
        assert torch.equal(a, b)
    assert torch.equal(m, plain.opt.moments()[0])


@pytest.mark.parametrize("bits", [8, 32])
def test_scratch_belongs_to_the_steps_stream(S, bits):
    """A step on another stream, waiting there when its optimizer goes: nothing is written into memory that the first
    stream has been given since."""
    many, plain = Many(S, F32, F32, bits, seed=1), Many(S, F32, F32, bits, seed=1)
    plain.opt.step(plain.grads, 1e-2)
    state = many.opt.state
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # 50 ms or so
    many.opt.step(many.grads, 1e-2, stream=side)
    many.opt = None
    given = [torch.full((256,), 255, dtype=torch.uint8, device="cuda") for _ in range(2000)]
    torch.cuda.synchronize()
    assert all((t == 255).all() for t in given)
    for a, b in zip(many.params + list(state.values()), plain.params + list(plain.opt.state.values())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [8, 32])
def test_a_captured_step_outlives_its_optimizer(S, bits):
    """The graph writes into the tensors that its owner keeps, and into nothing that the allocator has given away."""
    many, plain = Many(S, F32, F32, bits, seed=1), Many(S, F32, F32, bits, seed=1)
    state = many.opt.state
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        many.opt.step(many.grads, 1e-2)
    many.opt = None
    given = [torch.full((256,), 255, dtype=torch.uint8, device="cuda") for _ in range(2000)]
    for _ in range(3):
        graph.replay()
        plain.opt.step(plain.grads, 1e-2)
    torch.cuda.synchronize()
    assert all((t == 255).all() for t in given)
    for a, b in zip(many.params + list(state.values()), plain.params + list(plain.opt.state.values())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [0, 1, 4095, 16384, 16385, 3 << 20, 40_000_003])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm(S, n, dtype, offset):
    """Sums that keep what is cut off: the norm is off by its own rounding and the 2^-44 or so of 2^20 lost rests."""
    x = _random(R.generator(n), n, dtype, 3.0, offset)[1]
    for grads in ([x], [x, x[:n // 2], x[:0]]):
        want = sum(g.double().square().sum() for g in grads) ** 0.5
        got = S.grad_norm(grads)
        assert abs(got.double() - want) <= 2.0 ** -24 * 1.001 * want
        assert abs(got._wide - want) <= 2.0 ** -40 * want
        ws = torch.full((max(1, 8 * 100000),), 255, dtype=torch.uint8, device="cuda")
        out = torch.empty(1, device="cuda")
        assert S.grad_norm(grads, out=out, workspace=ws) is out and torch.equal(out, got)


@pytest.mark.parametrize("n", [1, 9, 5000, 3 << 20])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-10, 1e-18, 1e-21, 1e-25, 1e-38, 1e-40])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_of_small_gradients(S, n, dtype, scale, offset):
    """Gradients whose squares are subnormal in 32 bits, or nothing: rounded once, as large ones are (the norm itself may
    be subnormal: half its step then).  Alone, and with a tensor, an element and a run of elements that are larger."""
    g = R.generator(n)
    x = _random(g, n, dtype, scale, offset)[1]
    assert n == 1 or (x != 0).any()  # (bf16's least number is 9.2e-41: one element of 1e-40 may be 0)
    y, z = x.clone(), x.clone()
    y[n // 2] = scale * 1000
    z[:n // 3] *= 1024
    for grads in ([x], [y], [z], [x, x[:0], y, z], [x, torch.full((3,), scale * 64, device="cuda")], [x, torch.zeros(70000, device="cuda")]):
        want = sum(q.double().square().sum() for q in grads) ** 0.5
        got = S.grad_norm(grads)
        assert abs(got.double() - want) <= 2.0 ** -24 * 1.001 * want + 2.0 ** -150
        assert abs(got._wide - want) <= 2.0 ** -40 * want
    ones = torch.ones(1, device="cuda")
    assert float(S.grad_norm([x, ones])) == float((1 + x.double().square().sum()).sqrt().float())


def test_norm_of_many_tensors(S):
    g = R.generator(8)
    grads = [torch.randn(int(n), generator=g, device="cuda").to(F32 if i % 3 else BF16)
             for i, n in enumerate(torch.randint(1, 9000, (1500,)))]
    want = sum(x.double().square().sum() for x in grads) ** 0.5
    assert abs(S.grad_norm(grads).double() - want) <= 1e-6 * want
    assert float(S.grad_norm([], out=torch.ones(1, device="cuda"))) == 0


def test_offsets_past_32_bits(S):
    """A tensor of more than 2^32 elements, moments and parameters in fewer bits, and one behind it."""
    n = (1 << 32) + 70
    p = torch.zeros(n, dtype=BF16, device="cuda")
    q = torch.zeros(100, dtype=BF16, device="cuda")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-3:] = 1.0
    g[5] = -2.0
    opt = S.AdamW([p, q], bits=8)
    assert abs(float(S.grad_norm([g])) - math.sqrt(7)) < 1e-5
    opt.step([g, torch.ones_like(q)], 0.5)
    assert (p[-3:] == -0.5).all() and p[5] == 0.5 and (q == -0.5).all()
    assert int((p != 0).sum()) == 4
    v = opt.state["v"]
    assert int((v != 0).sum()) == 104


def test_refusals(S):
    z = lambda *s, d=F32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    for bad, kind in (((), ValueError), ([z(4).cpu()], ValueError), ([z(4, d=torch.float16)], TypeError),
                      ([z(4, 4).t()[:3]], ValueError), ([z(3), 5], TypeError), (z(4), TypeError)):
        with pytest.raises(kind):
            S.AdamW(bad)
    for kw, kind in ((dict(bits=16), ValueError), (dict(betas=(1.0, 0.9)), ValueError), (dict(betas=(0.9, math.nan)), ValueError),
                     (dict(eps=-1.0), ValueError), (dict(seed=-1), ValueError), (dict(seed=1.5), ValueError),
                     (dict(weight_decay=[0.1]), ValueError), (dict(weight_decay=math.inf), ValueError),
                     (dict(copies=[None]), ValueError), (dict(copies=[z(4), None]), TypeError),
                     (dict(copies=[z(5, d=BF16), None]), ValueError), (dict(state={}), ValueError),
                     (dict(state={"m": z(64), "v": z(128), "step": z(1, d=torch.int64)}), ValueError)):
        with pytest.raises(kind):
            S.AdamW([z(4), z(8)], **kw)
    with pytest.raises(TypeError):
        S.AdamW([z(4, d=BF16)], copies=[z(4, d=BF16)])
    p = z(8)
    for twice in ([p, p], [p[:5], p[4:]], [z(8), p[2:3], z(4), p]):
        with pytest.raises(ValueError, match="overlap"):
            S.AdamW(twice)
    S.AdamW([p[:5], p[5:], p[5:5]])
    m, step = z(64), z(1, d=torch.int64)
    for state in ({"m": m, "v": m, "step": step}, {"m": m, "v": z(64), "step": m[:2].view(torch.int64)}):
        with pytest.raises(ValueError, match="overlap"):
            S.AdamW([p], state=state)
    opt = S.AdamW([z(4), z(2, 3)])
    for args, kw, kind in ((([z(4)], 1.0), {}, ValueError), (([z(4), z(6)], 1.0), {}, ValueError),
                           (([z(4), z(2, 3, d=torch.float16)], 1.0), {}, TypeError), (([z(4), z(3, 2).t()], 1.0), {}, ValueError),
                           (([z(4), z(2, 3).cpu()], 1.0), {}, ValueError), (([z(4), z(2, 3)], math.nan), {}, ValueError),
                           (([z(4), z(2, 3)], 1.0), dict(norm=z(1)), ValueError), (([z(4), z(2, 3)], 1.0), dict(max_norm=1.0), ValueError),
                           (([z(4), z(2, 3)], 1.0), dict(norm=z(1), max_norm=0.0), ValueError),
                           (([z(4), z(2, 3)], z(2)), {}, ValueError)):
        with pytest.raises(kind):
            opt.step(*args, **kw)
    assert int(opt.state["step"]) == 0
    p = z(4)
    opt = S.AdamW([p])
    p.data = z(4)
    with pytest.raises(ValueError, match="memory"):
        opt.step([z(4)], 1.0)
    for grads, kind in (([], ValueError), ([z(4).cpu()], ValueError), ([z(4), z(4, d=torch.int64)], TypeError), (z(4), TypeError)):
        with pytest.raises(kind):
            S.grad_norm(grads)


def test_a_copy_or_a_state_that_moved_is_refused(S):
    """A copy's values would go to where it used to be, moments to a tensor that may be too short."""
    z = lambda *s, d=F32: torch.ones(*s, dtype=d, device="cuda")  # noqa: E731
    params, copies = [z(4), z(2, 3), z(5)], [z(4, d=BF16), None, z(5, d=BF16)]
    opt = S.AdamW(params, copies=copies, bits=8)
    opt.step([z(4), z(2, 3), z(5)], 0.5)
    old = copies[2]
    was = copies[2].data
    old.data = z(5, d=BF16)
    with pytest.raises(ValueError, match="memory"):
        opt.step([z(4), z(2, 3), z(5)], 0.5)
    assert int(opt.state["step"]) == 1
    old.data = was
    m = opt.state["m"]
    was, m.data = m.data, z(64, d=torch.uint8)
    for call in (lambda: opt.step([z(4), z(2, 3), z(5)], 0.5), opt.moments):
        with pytest.raises(ValueError, match="memory"):
            call()
    m.data = was
    opt.step([z(4), z(2, 3), z(5)], 0.5)
    assert torch.equal(copies[2], params[2].to(BF16)) and torch.equal(copies[0], params[0].to(BF16))


@pytest.mark.parametrize("bits", [8, 32])
def test_the_least_eps(S, bits):
    """Moments of 0 make no step with any eps that is taken; smaller ones than 2^-126 are refused."""
    p = torch.ones(100, device="cuda")
    g = torch.zeros(100, device="cuda")
    S.AdamW([p], bits=bits, eps=2.0 ** -126).step([g], 1e-2)
    assert (p == 1).all()
    g[5] = 2.0
    S.AdamW([p], bits=bits, eps=2.0 ** -126).step([g], 0.25)  # m / sqrt(v) is 1
    assert abs(float(p[5]) - 0.75) <= 2 ** -19 and (p[:5] == 1).all() and (p[6:] == 1).all()
    for eps in (1e-40, 1e-46, 1e-300, 3.1e38, math.inf, math.nan):
        with pytest.raises(ValueError, match="eps"):
            S.AdamW([p], bits=bits, eps=eps)


def test_autograd_notices_a_step(S):
    """What was saved for a backward pass before a step is refused after it, as after an optimizer of PyTorch's."""
    master, grad = torch.ones(8, 8, device="cuda"), torch.ones(8, 8, device="cuda")
    copy = torch.ones(8, 8, dtype=BF16, device="cuda")
    opt = S.AdamW([master], copies=[copy])
    for saved in (master, copy):
        x = torch.ones(2, 8, dtype=saved.dtype, device="cuda", requires_grad=True)
        y = (x @ saved).sum()
        opt.step([grad], 1e-2)
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
        (x @ saved).sum().backward()  # a new pass sees the new values
        want = saved.double().sum(1)  # a sum of 8 equal numbers: 7 additions, 2^-24 of it each at most, and bf16's rounding
        assert ((x.grad.double() - want).abs() <= (7 * 2.0 ** -24 + (Q.U16 if saved is copy else 0)) * want).all()
    # parameters that were made in inference mode have no version; a captured step bumps it once
    with torch.inference_mode():
        p = torch.ones(4, device="cuda")
    S.AdamW([p]).step([torch.ones(4, device="cuda")], 0.5)
    assert torch.allclose(p, torch.full_like(p, 0.5), atol=1e-5)
