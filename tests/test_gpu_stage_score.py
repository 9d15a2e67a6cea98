"""Log probabilities of given tokens, entropy, alternatives and their gradients
(stage.score_forward, score_backward) against the definitions in 64 bits."""
import math

import pytest
import torch

import score_ref as Q
import stage_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


def _target(g, T, V, out=0.1):
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[torch.rand(T, generator=g, device="cuda") < out] = -100
    return t


def _grid_inputs(T, V, H, seed):
    g = R.generator(seed)
    return Q.grid(g, T, H), Q.grid(g, V, H, scale=2.0 ** round(math.log2(2 / math.sqrt(H)))), _target(g, T, V)


def _check(got, want, names):
    torch.cuda.synchronize()
    for k in names:
        if k == "top_index":
            assert torch.equal(got[k], want[k]), k
        else:
            R.check(got[k], want[k], k)


# one token and two (read by the row), then products: ragged edges of every tile, few and many column tiles, and enough
# tiles for pairs of blocks
SHAPES = [(1, 1, 1), (1, 257, 64), (2, 1000, 8), (2, 5003, 1001), (3, 40, 16), (5, 100, 1001), (64, 64, 64), (127, 300, 72),
          (129, 513, 136), (300, 5000, 63), (1000, 1031, 520), (3, 50257, 96), (700, 130, 2048), (2100, 2500, 1200),
          (1537, 3001, 264), (1, 128000, 256)]


@pytest.mark.parametrize("T,V,H", SHAPES)
@pytest.mark.parametrize("k", [0, 1, 7, 32])
def test_forward(S, T, V, H, k):
    k = min(k, V)
    x, w, target = _grid_inputs(T, V, H, T + 7 * V + H)
    got = S.score_forward(x, w, target, top=k)
    want = Q.score(x, w, target, k, exact=True)
    _check(got, want, ["logp", "lse", "entropy"] + (["top_logp", "top_index"] if k else []))
    assert set(got) == set(want)
    assert (got["logp"][target < 0] == 0).all()


@pytest.mark.parametrize("T", [3, 4, 8, 16, 37, 64, 128])
@pytest.mark.parametrize("V,H", [(32000, 128), (50257, 72)])
@pytest.mark.parametrize("k", [0, 8, 20, 32])
def test_a_batch_of_single_tokens(S, T, V, H, k):
    """One token of each sequence against a vocabulary of tens of thousands."""
    x, w, target = _grid_inputs(T, V, H, T + k)
    want = Q.score(x, w, target, k, exact=True)
    _check(S.score_forward(x, w, target, top=k), want, want)


@pytest.mark.parametrize("T", [3, 16, 130, 700])
@pytest.mark.parametrize("V", [47, 300, 511, 1000, 2433, 3000, 4865])
@pytest.mark.parametrize("k", [16, 17, 20, 32])
def test_tiles_of_few_columns(S, T, V, k):
    """Tiles whose second pieces are empty, fewer pieces than alternatives, more alternatives than are sorted at a time:
    the same by which lane looks at which piece."""
    x, w, target = _grid_inputs(T, V, 64, T + V)
    want = Q.score(x, w, target, k, exact=True)
    _check(S.score_forward(x, w, target, top=k), want, want)


@pytest.mark.parametrize("k", [0, 1, 6])
def test_both_joins(S, k):
    """Around the numbers of tokens from which a block joins the pieces of eight: to the last bit the same alternatives,
    and each token's numbers as in a call of its own kind."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    x, w, t = _grid_inputs(4 * sms + 9, 2000, 64, 41)
    for T in (2, 3, 4, 5, 3 * sms, 3 * sms + 1, 4 * sms, 4 * sms + 1, 4 * sms + 9):
        got, want = S.score_forward(x[:T], w, t[:T], top=k), Q.score(x[:T], w, t[:T], k, exact=True)
        _check(got, want, want)


@pytest.mark.parametrize("T,V,H", [(2, 3000, 512), (200, 3000, 512)])
def test_forward_off_the_grid(S, T, V, H):
    """Logits that are rounded: an alternative's own logit is no further below the true one of its rank than they are off."""
    g = R.generator(1)
    x, w, target = R.normal(g, T, H), R.normal(g, V, H, scale=2 / math.sqrt(H)), _target(g, T, V)
    got, want = S.score_forward(x, w, target, top=9), Q.score(x, w, target, 9)
    _check(got, want, ["logp", "lse", "entropy", "top_logp"])
    l = x.double() @ w.double().t()
    l = l.gather(1, got["top_index"]) - l.gather(1, want["top_index"])
    assert (l.abs() <= 2 * want["lse"][1][:, None]).all()
    assert all(len(set(r)) == 9 for r in got["top_index"].tolist())


@pytest.mark.parametrize("T", [1, 2, 3, 130])
@pytest.mark.parametrize("V", [33, 700, 20000])
@pytest.mark.parametrize("k", [1, 5, 32])
def test_equal_logits_come_by_column(S, T, V, k):
    """All logits equal, and then but a few: every bound is met by more columns than there are places."""
    w = torch.ones(V, 8, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(T, 8, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    r = S.score_forward(x, w, t, top=k)
    assert torch.equal(r["top_index"], torch.arange(k, device="cuda").expand(T, k))
    R.check(r["entropy"], (torch.full((T,), math.log(V), device="cuda", dtype=R.F64), torch.tensor(1e-4, device="cuda")))
    # a few in the middle are larger, one is larger still, and there are two values among the first
    at = torch.tensor([V // 2, V // 3, V - 1], device="cuda")
    w[at] = 2
    w[V // 2] = 3
    w[::7] *= -1
    want = Q.score(x, w, t, k, exact=True)
    _check(S.score_forward(x, w, t, top=k), want, ["logp", "lse", "entropy", "top_logp", "top_index"])


@pytest.mark.parametrize("T,V,H", [(2, 700, 64), (3, 300, 64), (40, 20000, 64), (130, 700, 2048)])
@pytest.mark.parametrize("k", [1, 5, 32])
def test_logits_of_minus_zero(S, T, V, H, k):
    """Logits that are 0, of either sign, alone or above negative ones: equal, so the first columns, each piece's within
    its places, and the rows beside them as they were."""
    x, w, t = _grid_inputs(T, V, H, 31)
    clean = S.score_forward(x, w, t, top=k)
    first = torch.arange(k, device="cuda")
    x = x.clone()
    for sign in (0.0, -0.0):
        x[::2] = sign  # every other row
        for rows in (-w.abs(), w.abs(), w):
            r = S.score_forward(x, rows, t, top=k)
            assert (r["top_index"][::2] == first).all()
            R.check(r["top_logp"][::2], (torch.full_like(r["top_logp"][::2], -math.log(V)).double(), torch.tensor(1e-4, device="cuda")))
        for n in clean:
            assert torch.equal(r[n][1::2], clean[n][1::2]), n
    # -0 as the largest logit: products of positive numbers with -0, and some that are negative
    y = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.full((V, H), -0.0, dtype=torch.bfloat16, device="cuda")
    rows[::3, 0] = -1.0
    want = Q.score(y, rows, t, k, exact=True)
    _check(S.score_forward(y, rows, t, top=k), want, ["logp", "lse", "entropy", "top_logp", "top_index"])


@pytest.mark.parametrize("T", [1, 70])
def test_rising_and_falling_logits(S, T):
    """Logits that rise along the vocabulary, so that every tile beats the one before it; and that fall."""
    V, H = 60000, 16
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    i = torch.arange(V, device="cuda")
    w[:, 0], w[:, 1] = (i // 256).to(torch.bfloat16), (i % 256).to(torch.bfloat16)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 1.0, 1 / 256
    x[1::2] *= -1
    t = torch.arange(T, device="cuda")
    _check(S.score_forward(x, w, t, top=20), Q.score(x, w, t, 20, exact=True), ["logp", "lse", "entropy", "top_logp", "top_index"])


@pytest.mark.parametrize("T", [2, 40])
def test_nan_and_infinities_stay_in_their_row(S, T):
    """Columns past the vocabulary are never alternatives; a NaN comes behind everything."""
    V, H = 300, 64
    x, w, t = _grid_inputs(T, V, H, 5)
    t = t.clamp_min(0)
    clean = S.score_forward(x, w, t, top=12)
    w = w.clone()
    w[:, 0] = w[:, 0].abs() + 1
    y = x.clone()
    y[0, 0] = math.nan
    r = S.score_forward(y, w, t, top=12)
    assert all(r[k][0].isnan().all() for k in ("logp", "lse", "entropy", "top_logp")) and (r["top_index"][0] == -1).all()
    for value, lse in ((math.inf, math.inf), (-math.inf, -math.inf)):
        y[0, 0] = value
        r = S.score_forward(y, w, t, top=12)
        assert r["lse"][0] == lse and r["entropy"][0].isnan() and not r["logp"][0].isfinite()
        assert torch.equal(r["top_index"][0], torch.arange(12, device="cuda"))  # all equal
    w0 = w.clone()
    w0[:, 0] = 0
    w0[5, 0], w0[7, 0] = math.nan, math.nan
    r = S.score_forward(x, w0, t, top=12)  # two columns without a number
    assert not ((r["top_index"] == 5) | (r["top_index"] == 7)).any() and (r["top_index"] >= 0).all()
    w1 = torch.full((40, H), math.nan, dtype=torch.bfloat16, device="cuda")
    w1[17] = 1
    r = S.score_forward(x, w1, t % 40, top=3)
    assert (r["top_index"] == torch.tensor([17, -1, -1], device="cuda")).all() and r["top_logp"].isnan().all()
    assert torch.isfinite(clean["entropy"]).all()


def test_impossible_columns(S):
    """Logits of minus infinity beside finite ones: probability 0, nothing added to the entropy."""
    V, H, T = 500, 32, 60
    x, w, t = _grid_inputs(T, V, H, 6)
    x, w = x.clone(), w.clone()
    x[:, 0], w[:, 0] = 1, 0
    w[::3, 0] = -math.inf
    t = torch.where(t % 3 == 0, t + 1, t.clamp_min(1))
    some = torch.arange(V, device="cuda") % 3 != 0
    to = torch.nonzero(some)[:, 0]
    small = torch.searchsorted(to, t)
    want = Q.score(x, w[some], small, 8, exact=True)
    got = S.score_forward(x, w, t, top=8)
    _check(got, want, ["logp", "lse", "entropy", "top_logp"])
    assert torch.equal(got["top_index"], to[want["top_index"]])
    g = R.generator(7)
    a, b = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    want = Q.score(x, w[some], small, 0, a, b, exact=True)
    r = S.score_backward(x, w, t, got["lse"], a, entropy=got["entropy"], dentropy=b, outputs=("dw",))
    R.check(r["dw"][some], want["dw"], "dw")
    assert (r["dw"][~some] == 0).all()


def test_chunks_of_tokens(S):
    """More tokens than are taken at a time."""
    T, V, H, k = 5000, 131072, 64, 32
    x, w, t = _grid_inputs(T, V, H, 8)
    got = S.score_forward(x, w, t, top=k)
    rows = torch.arange(0, T, 97, device="cuda")
    want = Q.score(x[rows], w, t[rows], k, exact=True)
    _check({n: v[rows] for n, v in got.items()}, want, want)
    assert S.score_forward_workspace(x, w, k) < 5 << 30


@pytest.mark.parametrize("T,V,H,stride,offset", [(1, 300, 64, 67, 1), (130, 300, 64, 64, 1), (77, 515, 100, 104, 8),
                                                 (77, 515, 100, 133, 3)])
def test_strides_and_offsets(S, T, V, H, stride, offset):
    g = R.generator(9)
    x, w = R.normal(g, T, H, stride=stride, offset=offset), R.normal(g, V, H, scale=0.2, stride=stride, offset=offset)
    t, a, b = _target(g, T, V), torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    bx = torch.full((T, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    bw = torch.full((V, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    got = S.score_forward(x, w, t, top=4)
    got.update(S.score_backward(x, w, t, got["lse"], a, entropy=got["entropy"], dentropy=b,
                                out={"dx": bx[:, :H], "dw": bw[:, :H]}))
    _check(got, Q.score(x, w, t, 4, a, b), ["logp", "lse", "entropy", "top_logp", "dx", "dw"])
    assert (bx[:, H:] == 7).all() and (bw[:, H:] == 7).all()


@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (1, 257, 64), (5, 100, 1001), (64, 64, 64), (129, 513, 136), (300, 5000, 63),
                                   (700, 130, 2048), (2100, 2500, 1200), (3, 50257, 96)])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradients(S, T, V, H, entropy):
    g = R.generator(T + V + H)
    x, w, t = R.normal(g, T, H), R.normal(g, V, H, scale=2 / math.sqrt(H)), _target(g, T, V)
    a = torch.randn(T, generator=g, device="cuda")
    b = torch.randn(T, generator=g, device="cuda") if entropy else None
    f = S.score_forward(x, w, t)
    got = S.score_backward(x, w, t, f["lse"], a, entropy=f["entropy"] if entropy else None, dentropy=b)
    want = Q.score(x, w, t, 0, a, b)
    _check(got, want, ["dx", "dw"])
    assert (got["dx"][t < 0] == 0).all()


def test_gradients_by_differences(S):
    """(L(x + h) - L(x - h)) / 2h along random directions, L from score_forward's outputs, against dx.  h is a power of
    two times whole numbers, so that x +- h is exact; the quotient is off by its third-order term, a few h^2 of the
    gradient, and by what L's outputs are off, over h."""
    T, V, H = 12, 90, 64
    g = R.generator(10)
    x, w, t = Q.grid(g, T, H), Q.grid(g, V, H, scale=0.25), _target(g, T, V)
    a, b = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")

    def loss(x):
        r = S.score_forward(x, w, t)
        return (a * r["logp"] + torch.where(t >= 0, b, 0.0) * r["entropy"]).double()

    f = S.score_forward(x, w, t)
    dx = S.score_backward(x, w, t, f["lse"], a, entropy=f["entropy"], dentropy=b, outputs=("dx",))["dx"].double()
    h = 2.0 ** -6
    for seed in range(4):
        u = torch.randint(-1, 2, (T, H), generator=R.generator(seed), device="cuda").to(torch.bfloat16)
        # |x| < 4 in steps of 2^-3 and h = 2^-6: 8 significant bits hold x +- h where |x| < 2
        u = torch.where(x.abs() < 1.9, u, 0)
        diff = (loss(x + h * u) - loss(x - h * u)) / (2 * h)
        along = (dx * u.double()).sum(1)
        s = (w.double() @ u.double().t()).abs().amax(0)  # how far the logits move for h = 1
        # third derivatives of logp and entropy along a direction are at most some 8 s^3 (H + 1); outputs off by 2e-5
        allowed = (a.abs() + b.abs()).double() * (8 * s ** 3 * h * h * (math.log(V) + 1) / 6 + 2e-5 * 6 / h) + 2 ** -8 * dx.abs().sum(1)
        assert ((diff - along).abs() <= allowed).all()


def test_without_entropy_it_is_the_losss_gradient(S):
    g = R.generator(11)
    x, w, t = R.normal(g, 200, 128), R.normal(g, 1000, 128, scale=0.2), _target(g, 200, 1000)
    a = torch.randn(200, generator=g, device="cuda")
    lse = S.head_forward(x, w, t)["lse"]
    one, two = S.score_backward(x, w, t, lse, a), S.head_backward(x, w, t, lse, weight=a, scale=-1.0)
    assert torch.equal(one["dx"], two["dx"]) and torch.equal(one["dw"], two["dw"])


def test_left_out_rows_are_not_read(S):
    x, w, t = _grid_inputs(70, 300, 64, 12)
    t = t.clamp_min(0)
    t[::5] = torch.tensor([-100, -1, 300, 1 << 40, -(1 << 40)], device="cuda").repeat(3)[:14]
    a, b = torch.ones(70, device="cuda"), torch.full((70,), 0.5, device="cuda")
    f = S.score_forward(x, w, t, top=3)
    clean = S.score_backward(x, w, t, f["lse"], a, entropy=f["entropy"], dentropy=b)
    R.check(clean["dw"], Q.score(x, w, t, 0, a, b)["dw"])
    x = x.clone()
    x[::5] = torch.tensor([math.nan, math.inf, -math.inf, 1e38], device="cuda").repeat(16).to(torch.bfloat16)
    f2 = S.score_forward(x, w, t, top=3)
    got = S.score_backward(x, w, t, f2["lse"], a, entropy=f2["entropy"], dentropy=b)
    keep = R.left_in(t, 300)
    for k in f:
        assert torch.equal(f[k][keep], f2[k][keep]), k
    assert (f2["logp"][~keep] == 0).all()
    for k in clean:
        assert torch.equal(clean[k], got[k]), k


def test_entropy_is_read_only_where_its_gradient_is_not_zero(S):
    x, w, t = _grid_inputs(30, 200, 64, 13)
    f = S.score_forward(x, w, t)
    a, b = torch.ones(30, device="cuda"), torch.zeros(30, device="cuda")
    ent = torch.full((30,), math.nan, device="cuda")
    one = S.score_backward(x, w, t, f["lse"], a, entropy=ent, dentropy=b)
    want = Q.score(x, w, t, 0, a, b, exact=True)
    _check(one, want, ["dx", "dw"])


def test_no_rows(S):
    w = torch.ones(10, 16, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    t, z = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    r = S.score_forward(x, w, t, top=4)
    assert r["logp"].shape == (0,) and r["entropy"].shape == (0,) and r["top_index"].shape == (0, 4)
    b = S.score_backward(x, w, t, r["lse"], z, entropy=z, dentropy=z)
    assert b["dx"].shape == (0, 16) and (b["dw"] == 0).all()
    acc = torch.full((10, 16), 3.0, device="cuda")
    S.score_backward(x, w, t, r["lse"], z, outputs=("dw",), add=True, out={"dw": acc})
    assert (acc == 3).all()


def test_float_sum_over_microbatches(S):
    g = R.generator(14)
    T, V, H = 150, 333, 72
    w = R.normal(g, V, H, scale=0.2)
    acc = torch.zeros(V, H, device="cuda")
    total = bound = 0
    for i in range(2):
        x, t = R.normal(g, T, H), _target(g, T, V)
        a, b = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
        f = S.score_forward(x, w, t)
        S.score_backward(x, w, t, f["lse"], a, entropy=f["entropy"], dentropy=b, outputs=("dw",), add=True, out={"dw": acc})
        v, e = Q.score(x, w, t, 0, a, b)["dw"]
        total, bound = total + v, bound + e
    R.check(acc, (total, bound))


@pytest.mark.parametrize("T", [1, 300])
def test_same_on_every_call_and_with_given_memory(S, T):
    x, w, t = _grid_inputs(T, 9000, 256, 15)
    first = S.score_forward(x, w, t, top=11)
    ws = torch.full((S.score_forward_workspace(x, w, 11),), 255, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 127):
        ws.fill_(fill)
        out = {k: torch.empty_like(v) for k, v in first.items()}
        r = S.score_forward(x, w, t, top=11, out=out, workspace=ws)
        for k in first:
            assert r[k] is out[k] and torch.equal(first[k], r[k]), k


def test_stream_graph_and_other_thread_of_work(S):
    """Captured on a side stream and replayed on new inputs, with a call on another stream at the same time."""
    x, w, t = _grid_inputs(100, 4000, 128, 16)
    y, _, u = _grid_inputs(100, 4000, 128, 17)
    a, b = torch.randn(100, device="cuda"), torch.randn(100, device="cuda")
    want = []
    for q, r in ((x, t), (y, u)):
        f = S.score_forward(q, w, r, top=6)
        f.update(S.score_backward(q, w, r, f["lse"], a, entropy=f["entropy"], dentropy=b))
        want.append(f)
    side = torch.cuda.Stream()
    sx, st = x.clone(), t.clone()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        f = S.score_forward(sx, w, st, top=6)
        f.update(S.score_backward(sx, w, st, f["lse"], a, entropy=f["entropy"], dentropy=b))
    sx.copy_(y)
    st.copy_(u)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    graph.replay()
    again = S.score_forward(x, w, t, top=6, stream=other)
    torch.cuda.synchronize()
    for k in want[1]:
        assert torch.equal(f[k], want[1][k]), k
    for k in again:
        assert torch.equal(again[k], want[0][k]), k
    assert S.wait_failure() == 0


def test_two_captured_calls_share_their_workspace(S):
    """Replayed in turn: each call clears what it needs of the workspace."""
    a, b = _grid_inputs(600, 5000, 64, 18), _grid_inputs(40, 9000, 128, 19)
    want = [S.score_forward(*q, top=7) for q in (a, b)]
    ws = torch.full((max(S.score_forward_workspace(*q[:2], 7) for q in (a, b)),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, got = [], []
    for q in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got.append(S.score_forward(*q, top=7, workspace=ws))
        graphs.append(g)
    for i in (0, 1, 0, 0, 1):
        for t in got[i].values():
            t.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        for k in want[i]:
            assert torch.equal(got[i][k], want[i][k]), k


def test_refusals(S):
    x, w, t = _grid_inputs(4, 20, 8, 20)
    f = torch.zeros(4, device="cuda")
    for top in (-1, 21, 33, 1.0, True, None):
        with pytest.raises(ValueError, match="top"):
            S.score_forward(x, w, t, top=top)
    wide = torch.zeros(4, 6, device="cuda")
    for kw, kind in ((dict(top=3, out={"top_logp": wide[:, :3]}), ValueError), (dict(out={"logp": f[:3]}), ValueError),
                     (dict(top=3, out={"top_index": wide[:, :3].contiguous()}), TypeError), (dict(workspace=t), TypeError)):
        with pytest.raises((kind, ValueError)):
            S.score_forward(x, w, t, **kw)
    with pytest.raises(ValueError):
        S.score_forward(x, w[:, :4], t)
    for kw in (dict(entropy=f), dict(dentropy=f), dict(entropy=f, dentropy=f[:3]), dict(outputs=("dy",)), dict(add=True)):
        with pytest.raises(ValueError):
            S.score_backward(x, w, t, f, f, **kw)
