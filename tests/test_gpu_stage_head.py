"""The last stage's loss and its gradients (stage.head_forward, head_backward)
against the definitions in 64 bits, with the bounds of stage_ref."""
import math

import pytest
import torch

import stage_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


def _inputs(T, V, H, seed, out=0.1, **kw):
    g = R.generator(seed)
    x, w = R.normal(g, T, H, **kw), R.normal(g, V, H, scale=2 / math.sqrt(H), **kw)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[torch.rand(T, generator=g, device="cuda") < out] = -100
    weight = torch.rand(T, generator=g, device="cuda") + 0.5
    return x, w, target, weight


def _both(S, x, w, target, scale=1.0, weight=None, **kw):
    r = S.head_forward(x, w, target)
    r.update(S.head_backward(x, w, target, r["lse"], scale=scale, weight=weight, **kw))
    torch.cuda.synchronize()
    return r


# one token, ragged edges of every tile, widths that are no multiple of 8, narrow and wide
SHAPES = [(1, 1, 1), (1, 257, 64), (2, 1000, 8), (5, 100, 1001), (64, 64, 64), (127, 300, 72), (128, 512, 128),
          (129, 513, 136), (255, 777, 200), (300, 5000, 63), (1000, 1031, 520), (3, 50257, 96), (700, 130, 2048),
          # enough tiles for pairs of blocks in every product
          (2100, 2500, 1200), (1537, 3001, 264), (2049, 5001, 531)]


@pytest.mark.parametrize("T,V,H", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_loss_and_gradients(S, T, V, H, weighted):
    x, w, target, weight = _inputs(T, V, H, 100 * T + V + H)
    weight = weight if weighted else None
    got = _both(S, x, w, target, scale=1 / T, weight=weight)
    want = R.head(x, w, target, 1 / T, weight)
    for k in ("loss", "lse", "dx", "dw"):
        R.check(got[k], want[k], k)
    assert (got["loss"][target < 0] == 0).all() and (got["dx"][target < 0] == 0).all()


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("V,H,stride,offset", [(1, 8, 8, 0), (7, 4096, 4096, 0), (5000, 1001, 1001, 1), (40000, 264, 272, 8),
                                               (9999, 4104, 4105, 3), (3000, 16384, 16384, 0)])
def test_few_tokens(S, T, V, H, stride, offset):
    """Both sides of the limit up to which w is read by the row: aligned and unaligned rows, more and fewer rows than
    there are warps, widths on both sides of what shared memory holds."""
    x, w, target, _ = _inputs(T, V, H, T + V + H, stride=stride, offset=offset)
    if T > 2:
        target[1] = -1
    got = S.head_forward(x, w, target)
    want = R.head(x, w, target)
    for k in ("loss", "lse"):
        R.check(got[k], want[k], k)


@pytest.mark.parametrize("T,V,H,stride,offset", [(130, 300, 64, 64, 1), (130, 300, 64, 67, 0), (77, 515, 100, 104, 8),
                                                 (77, 515, 100, 133, 3)])
def test_strides_and_offsets(S, T, V, H, stride, offset):
    """Rows inside a larger buffer of NaN: nothing outside them is read, nothing outside the outputs is written."""
    x, w, target, weight = _inputs(T, V, H, 5, stride=stride, offset=offset)
    bx = torch.full((T, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    bw = torch.full((V, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    got = _both(S, x, w, target, weight=weight, out={"dx": bx[:, :H], "dw": bw[:, :H]})
    want = R.head(x, w, target, 1.0, weight)
    for k in ("loss", "lse", "dx", "dw"):
        R.check(got[k], want[k], k)
    assert (bx[:, H:] == 7).all() and (bw[:, H:] == 7).all()


def test_large_logits(S):
    """Logits of some hundreds: the sums are relative to the largest one."""
    x, w, target, _ = _inputs(40, 600, 64, 6)
    w = (w * 30).to(torch.bfloat16)
    got, want = _both(S, x, w, target), R.head(x, w, target)
    for k in want:
        R.check(got[k], want[k], k)


def test_left_out_rows_are_not_read(S):
    """A left-out token's activation may hold anything, and every target outside the vocabulary leaves out."""
    x, w, target, _ = _inputs(70, 300, 64, 7, out=0.0)
    target[::5] = torch.tensor([-100, -1, 300, 1 << 40, -(1 << 40)], device="cuda").repeat(3)[:14]
    want = R.head(x, w, target)
    clean = _both(S, x, w, target)
    x[::5] = torch.tensor([math.nan, math.inf, -math.inf, 1e38], device="cuda").repeat(16)
    got = _both(S, x, w, target)
    for k in ("loss", "dx", "dw"):
        R.check(got[k], want[k], k)
        assert torch.equal(got[k], clean[k]), k


def test_no_token_left(S):
    x, w, target, _ = _inputs(33, 200, 64, 8, out=1.1)
    got = _both(S, x, w, target)
    assert (got["loss"] == 0).all() and (got["dx"] == 0).all() and (got["dw"] == 0).all()
    assert torch.isfinite(got["lse"]).all()


def test_nan_and_infinite_logits_stay_in_their_row(S):
    x, w, target, _ = _inputs(20, 300, 64, 9, out=0.0)
    w = w.abs()
    x[3, 0] = math.nan
    x[4, 1] = math.inf    # logits +inf
    x[5, 2] = -math.inf   # logits -inf: exp adds up to 0
    got = S.head_forward(x, w, target)
    torch.cuda.synchronize()
    assert got["lse"][3].isnan() and got["lse"][4] == math.inf and got["lse"][5] == -math.inf
    rest = torch.tensor([i for i in range(20) if i not in (3, 4, 5)], device="cuda")
    want = R.head(x[rest], w, target[rest])
    R.check(got["loss"][rest], want["loss"])


def test_no_rows(S):
    w = torch.ones(10, 16, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    r = S.head_forward(x, w, t)
    assert r["loss"].shape == (0,) and r["lse"].shape == (0,)
    b = S.head_backward(x, w, t, r["lse"])
    assert b["dx"].shape == (0, 16) and (b["dw"] == 0).all()
    acc = torch.full((10, 16), 3.0, device="cuda")
    S.head_backward(x, w, t, r["lse"], outputs=("dw",), add=True, out={"dw": acc})
    assert (acc == 3).all()


def test_float_sum_over_microbatches(S):
    """dw as a float running sum: two microbatches add up to the two gradients."""
    (x, w, target, _), (x2, _, target2, _) = _inputs(90, 400, 72, 10), _inputs(60, 400, 72, 11)
    acc = torch.zeros(400, 72, device="cuda")
    lse, lse2 = S.head_forward(x, w, target)["lse"], S.head_forward(x2, w, target2)["lse"]
    S.head_backward(x, w, target, lse, outputs=("dw",), out={"dw": acc})
    S.head_backward(x2, w, target2, lse2, outputs=("dw",), add=True, out={"dw": acc})
    a, b = R.head(x, w, target)["dw"], R.head(x2, w, target2)["dw"]
    R.check(acc, (a[0] + b[0], a[1] + b[1] + R.U32 * (a[0].abs() + b[0].abs())))


def test_b_and_w_apart_give_the_same(S):
    x, w, target, weight = _inputs(200, 900, 128, 12)
    lse = S.head_forward(x, w, target)["lse"]
    both = S.head_backward(x, w, target, lse, weight=weight, scale=0.5)
    dx = S.head_backward(x, w, target, lse, weight=weight, scale=0.5, outputs=("dx",))
    dw = S.head_backward(x, w, target, lse, weight=weight, scale=0.5, outputs=("dw",))
    assert set(dx) == {"dx"} and set(dw) == {"dw"}
    assert torch.equal(both["dx"], dx["dx"]) and torch.equal(both["dw"], dw["dw"])


def test_gradients_against_differences(S):
    """The change of the loss along a direction, by central differences in 64 bits."""
    T, V, H = 50, 333, 48
    x, w, target, weight = _inputs(T, V, H, 13)
    got = _both(S, x, w, target, scale=1 / T, weight=weight)
    bound = R.head(x, w, target, 1 / T, weight)
    g = R.generator(14)
    keep = R.left_in(target, V)

    def loss(xx, ww):
        l = xx @ ww.t()
        at = torch.where(keep, target, 0)[:, None]
        return (torch.where(keep, weight.double(), 0.0) * (torch.logsumexp(l, 1) - l.gather(1, at)[:, 0])).sum() / T

    for k in ("dx", "dw"):
        u = torch.randn((x if k == "dx" else w).shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5  # truncation ~ h^2 = 1e-10, rounding ~ 1e-16 / h = 1e-11
        ux, uw = (u, 0 * w.double()) if k == "dx" else (0 * x.double(), u)
        diff = (loss(x.double() + h * ux, w.double() + h * uw) - loss(x.double() - h * ux, w.double() - h * uw)) / (2 * h)
        assert abs((got[k].double() * u).sum() - diff) <= (bound[k][1] * u.abs()).sum() + 1e-8, k


def test_same_on_every_call_and_on_another_stream(S):
    x, w, target, weight = _inputs(300, 2000, 256, 15)
    first = _both(S, x, w, target, weight=weight)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(max(S.head_forward_workspace(x, w), S.head_backward_workspace(x, w)), dtype=torch.uint8,
                     device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    again = S.head_forward(x, w, target, workspace=ws, stream=s)
    again.update(S.head_backward(x, w, target, again["lse"], weight=weight, workspace=ws, stream=s))
    s.synchronize()
    for k in first:
        assert torch.equal(first[k], again[k]), k


def test_offsets_past_32_bits(S):
    """Rows far apart: element offsets beyond 2^31."""
    T, V, H = 3, 5, 64
    stride = (1 << 30) + 64
    buf = torch.zeros(T * stride, dtype=torch.bfloat16, device="cuda")
    g = R.generator(16)
    x = buf.as_strided((T, H), (stride, 1))
    x.copy_(R.normal(g, T, H))
    w, target = R.normal(g, V, H, scale=0.2), torch.tensor([0, 4, 2], device="cuda")
    got = S.head_forward(x, w, target)
    lse = got["lse"]
    want = R.head(x, w, target)
    R.check(got["loss"], want["loss"])
    grads = S.head_backward(x, w, target, lse)
    R.check(grads["dw"], want["dw"])
    # the same rows as the output matrix
    t2 = torch.tensor([0, 2], device="cuda")
    out = torch.zeros_like(buf).as_strided((T, H), (stride, 1))
    y = w[:2]
    lse2 = S.head_forward(y, x, t2)["lse"]
    r = S.head_backward(y, x, t2, lse2, out={"dw": out})
    R.check(r["dw"], R.head(y, x, t2)["dw"])


def test_refusals_on_the_gpu(S):
    x, w, target, _ = _inputs(8, 50, 32, 17)
    lse = S.head_forward(x, w, target)["lse"]
    with pytest.raises(ValueError, match="w: expected shape"):
        S.head_forward(x, w[:, :16], target)
    with pytest.raises(TypeError, match="x: expected dtype"):
        S.head_forward(x.float(), w, target)
    with pytest.raises(TypeError, match="target: expected dtype"):
        S.head_forward(x, w, target.int())
    with pytest.raises(ValueError, match="target: expected shape"):
        S.head_forward(x, w, target[1:])
    with pytest.raises(ValueError, match="contiguous rows"):
        S.head_forward(x.t().contiguous().t(), w, target)
    with pytest.raises(ValueError, match="workspace"):
        S.head_forward(x, w, target, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="outputs"):
        S.head_backward(x, w, target, lse, outputs=("dz",))
    with pytest.raises(ValueError, match="add"):
        S.head_backward(x, w, target, lse, add=True)
    with pytest.raises(ValueError, match="dx: expected shape"):
        S.head_backward(x, w, target, lse, out={"dx": torch.empty(8, 31, dtype=torch.bfloat16, device="cuda")})
    with pytest.raises(S.PPSchedError):  # a workspace that is not aligned
        n = S.head_forward_workspace(x, w)
        S.head_forward(x, w, target, workspace=torch.empty(n + 1, dtype=torch.uint8, device="cuda")[1:])


def test_in_a_graph_and_no_wait_ran_out(S):
    """Captured calls give what direct ones give, again and again; and no wait inside the products ran out so far."""
    x, w, target, weight = _inputs(500, 3000, 264, 18)
    first = _both(S, x, w, target, weight=weight)
    packed = S.pack(x)
    grad = S.weight_grad(x, packed)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = S.head_forward(x, w, target)
        again.update(S.head_backward(x, w, target, again["lse"], weight=weight))
        grad2 = S.weight_grad(x, S.pack(x))
    for _ in range(3):
        for t in (*again.values(), grad2):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(first[k], again[k]) for k in first) and torch.equal(grad, grad2)
    assert S.wait_failure() == 0
