"""The join of a block to the residual stream (stage.join_forward,
join_backward) against the definitions in 64 bits, with stage_ref's bounds."""
import math

import pytest
import torch

import stage_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


def _inputs(T, H, groups, seed, **kw):
    g = R.generator(seed)
    r = {"x": R.normal(g, T, H, scale=2.0, **kw), "f": R.normal(g, T, H, scale=0.3, **kw),
         "dh": R.normal(g, T, H, scale=0.1, **kw), "dy": R.normal(g, T, H, scale=0.1, **kw),
         "w_post": R.normal(g, H) + 1, "w_pre": R.normal(g, H) + 1,
         "gate": None if groups == 0 else R.normal(g, groups, H, scale=0.5)}
    r["rows"] = 0 if groups <= 1 else -(-T // groups)
    return r


def _forward(S, a, alpha, **kw):
    return S.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], a["gate"], rows_per_gate=a["rows"], alpha=alpha,
                          eps=EPS, **kw)


def _backward(S, a, y, f, r1, r2, alpha, dy=True, **kw):
    return S.join_backward(a["dh"], a["dy"] if dy else None, y, f, r1, r2, a["w_post"], a["w_pre"], a["gate"],
                           rows_per_gate=a["rows"], alpha=alpha, **kw)


# widths on both sides of every variant's limit, and odd ones; groups 0: no gate
CASES = [(1, 1, 1), (1, 64, 0), (3, 63, 3), (7, 1001, 1), (33, 1024, 2), (40, 1025, 5), (50, 2048, 1), (20, 2049, 4),
         (17, 4096, 17), (19, 4097, 1), (31, 8192, 2), (9, 8193, 3), (5, 16384, 1), (400, 1536, 2), (700, 1360, 1), (350, 5120, 1), (2000, 72, 7), (513, 1000, 3)]


@pytest.mark.parametrize("T,H,groups", CASES)
def test_forward(S, T, H, groups):
    a = _inputs(T, H, groups, T + H)
    want = R.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], a["gate"], a["rows"], 0.7, EPS)
    plain = _forward(S, a, 0.7)
    kept = _forward(S, a, 0.7, keep=True)
    for k in want:
        R.check(plain[k], want[k], k)
        assert torch.equal(plain[k], kept[k]), k
    for k, of in (("kept_y", kept["y"]), ("kept_f", a["f"])):
        q, e = R.pack(of)
        assert torch.equal(kept[k].q, q) and torch.equal(kept[k].e, e), k


@pytest.mark.parametrize("T,H,groups", CASES)
@pytest.mark.parametrize("packed", [False, True])
def test_backward(S, T, H, groups, packed):
    a = _inputs(T, H, groups, 2 * T + H)
    fw = _forward(S, a, 0.7, keep=packed)
    y, f = (fw["kept_y"], fw["kept_f"]) if packed else (fw["y"], a["f"])
    yv, fv = (R.value(y.q, y.e), R.value(f.q, f.e)) if packed else (y, f)
    for dy in (True, False):
        got = _backward(S, a, y, f, fw["rstd_post"], fw["rstd_pre"], 0.7, dy=dy)
        want = R.join_backward(a["dh"], a["dy"] if dy else None, yv, fv, fw["rstd_post"], fw["rstd_pre"], a["w_post"],
                               a["w_pre"], a["gate"], a["rows"], 0.7)
        assert set(got) == set(want)
        for k in want:
            R.check(got[k], want[k], k)


@pytest.mark.parametrize("H,stride,offset", [(96, 97, 0), (96, 104, 1), (100, 104, 8), (1100, 1111, 5)])
def test_strides_and_offsets(S, H, stride, offset):
    """Rows inside buffers of NaN: nothing beside them is read or written."""
    T = 37
    a = _inputs(T, H, 2, 3, stride=stride, offset=offset)
    w = torch.full((H + 1,), math.nan, dtype=torch.bfloat16, device="cuda")
    w[1:] = a["w_pre"]
    a["w_pre"] = w[1:]
    bufs = [torch.full((T, stride), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    fw = _forward(S, a, 1.0, out={"y": bufs[0][:, :H], "h": bufs[1][:, :H]}, keep=True)
    want = R.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], a["gate"], a["rows"], 1.0, EPS)
    for k in want:
        R.check(fw[k], want[k], k)
    q, e = R.pack(fw["y"])
    assert torch.equal(fw["kept_y"].q, q)
    got = _backward(S, a, fw["y"], a["f"], fw["rstd_post"], fw["rstd_pre"], 1.0,
                    out={"dx": bufs[2][:, :H], "df": bufs[3][:, :H]})
    want = R.join_backward(a["dh"], a["dy"], fw["y"], a["f"], fw["rstd_post"], fw["rstd_pre"], a["w_post"], a["w_pre"],
                           a["gate"], a["rows"], 1.0)
    for k in want:
        R.check(got[k], want[k], k)
    # checkpoints at any stride and offset too
    buf = torch.full((2, T, stride + 1), 55, dtype=torch.int8, device="cuda")
    py, pf = (S.pack(t, out=S.Packed(b[:, 1:H + 1], torch.empty(T, -(-H // 64), dtype=torch.int8, device="cuda")))
              for b, t in zip(buf, (fw["y"], a["f"])))
    got = _backward(S, a, py, pf, fw["rstd_post"], fw["rstd_pre"], 1.0)
    want = R.join_backward(a["dh"], a["dy"], R.value(py.q, py.e), R.value(pf.q, pf.e), fw["rstd_post"], fw["rstd_pre"],
                           a["w_post"], a["w_pre"], a["gate"], a["rows"], 1.0)
    for k in want:
        R.check(got[k], want[k], k)
    assert all((b[:, H:] == 7).all() for b in bufs)


def test_rows_of_zeros_and_non_finite_rows(S):
    """A row of zeros has rstd 1/sqrt(eps); NaN and infinities stay in their row, and gradients of other rows hold."""
    T, H = 12, 200
    a = _inputs(T, H, 1, 4)
    for k in ("x", "f", "dh", "dy"):
        a[k][2] = 0
    fw = _forward(S, a, 1.0, keep=True)
    assert (fw["h"][2] == 0).all() and abs(fw["rstd_pre"][2].item() * math.sqrt(EPS) - 1) < 1e-6
    got = _backward(S, a, fw["kept_y"], fw["kept_f"], fw["rstd_post"], fw["rstd_pre"], 1.0)
    assert (got["dx"][2] == 0).all() and (got["df"][2] == 0).all() and torch.isfinite(got["dw_pre"]).all()
    a["f"][3, 7], a["x"][4, 9] = math.nan, math.inf
    bad = _forward(S, a, 1.0)
    assert bad["h"][3].isnan().all() and bad["y"][4, 9] == math.inf
    rest = [i for i in range(T) if i not in (3, 4)]
    for k in ("y", "h", "rstd_post", "rstd_pre"):
        assert torch.equal(bad[k][rest], fw[k][rest]), k


def test_no_rows_and_unused_gates(S):
    H = 40
    a = _inputs(0, H, 1, 5)
    fw = _forward(S, a, 1.0, keep=True)
    assert fw["y"].shape == (0, H)
    got = _backward(S, a, fw["y"], a["f"], fw["rstd_post"], fw["rstd_pre"], 1.0)
    assert (got["dw_pre"] == 0).all() and (got["dw_post"] == 0).all() and (got["dgate"] == 0).all()
    a = _inputs(10, H, 1, 6)
    a["gate"], a["rows"] = R.normal(R.generator(7), 5, H), 4  # 3 gates are used
    fw = _forward(S, a, 1.0)
    got = _backward(S, a, fw["y"], a["f"], fw["rstd_post"], fw["rstd_pre"], 1.0)
    want = R.join_backward(a["dh"], a["dy"], fw["y"], a["f"], fw["rstd_post"], fw["rstd_pre"], a["w_post"], a["w_pre"],
                           a["gate"], 4, 1.0)
    for k in want:
        R.check(got[k], want[k], k)
    assert (got["dgate"][3:] == 0).all()


def test_gradients_against_differences(S):
    """The change of sum(h * dh + y * dy) along directions of every input, by central differences in 64 bits.
    The gradient is taken from the unrounded y's bf16 neighbour, which may move it by 2^-8 of each term: the
    function is checked at an y that is a bf16 number (x is chosen so)."""
    T, H, groups = 12, 72, 3
    a = _inputs(T, H, groups, 8)
    d = {k: a[k].double() for k in ("x", "f", "w_post", "w_pre", "gate")}
    rows = a["rows"]

    def parts(v):
        g = v["gate"].repeat_interleave(rows, 0)
        n1 = v["f"] * (v["f"].square().mean(1, keepdim=True) + EPS).rsqrt()
        y = v["x"] + g * v["w_post"] * n1
        return y, y * (y.square().mean(1, keepdim=True) + EPS).rsqrt() * v["w_pre"]

    y16 = parts(d)[0].to(torch.bfloat16)
    d["x"] = d["x"] + (y16.double() - parts(d)[0])  # now y is y16
    r1 = (d["f"].square().mean(1) + EPS).rsqrt().float()
    r2 = (y16.double().square().mean(1) + EPS).rsqrt().float()
    got = _backward(S, a, y16, a["f"], r1, r2, 1.0)
    bound = R.join_backward(a["dh"], a["dy"], y16, a["f"], r1, r2, a["w_post"], a["w_pre"], a["gate"], rows, 1.0)

    def loss(v):
        y, h = parts(v)
        return (h * a["dh"].double()).sum() + (y * a["dy"].double()).sum()

    g = R.generator(9)
    for out, of in (("dx", "x"), ("df", "f"), ("dw_post", "w_post"), ("dw_pre", "w_pre"), ("dgate", "gate")):
        u = torch.randn(d[of].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        diff = (loss({**d, of: d[of] + h * u}) - loss({**d, of: d[of] - h * u})) / (2 * h)
        # r1 and r2 were rounded to 32 bits: 2^-24 of every term, 3 of them in a product
        slack = 4 * R.U32 * (got[out].double() * u).abs().sum()
        assert abs((got[out].double() * u).sum() - diff) <= (bound[out][1] * u.abs()).sum() + slack + 1e-7, out


def test_same_on_every_call_and_on_another_stream(S):
    a = _inputs(700, 1000, 7, 10)
    first = _forward(S, a, 0.5, keep=True)
    back = _backward(S, a, first["kept_y"], first["kept_f"], first["rstd_post"], first["rstd_pre"], 0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = _forward(S, a, 0.5, keep=True, stream=s)
    back2 = _backward(S, a, again["kept_y"], again["kept_f"], again["rstd_post"], again["rstd_pre"], 0.5, stream=s)
    s.synchronize()
    for k in ("y", "h", "rstd_post", "rstd_pre"):
        assert torch.equal(first[k], again[k]), k
    for k in back:
        assert torch.equal(back[k], back2[k]), k


def test_offsets_past_32_bits(S):
    T, H = 3, 128
    stride = (1 << 30) + 64
    a = _inputs(T, H, 1, 11)
    want = R.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], a["gate"], 0, 1.0, EPS)
    far = torch.zeros(T * stride, dtype=torch.bfloat16, device="cuda").as_strided((T, H), (stride, 1))
    far.copy_(a["x"])
    out = torch.zeros(T * stride, dtype=torch.bfloat16, device="cuda").as_strided((T, H), (stride, 1))
    a["x"] = far
    fw = _forward(S, a, 1.0, out={"y": out})
    for k in want:
        R.check(fw[k], want[k], k)
    got = _backward(S, a, fw["y"], a["f"], fw["rstd_post"], fw["rstd_pre"], 1.0, out={"dx": far})
    want = R.join_backward(a["dh"], a["dy"], fw["y"], a["f"], fw["rstd_post"], fw["rstd_pre"], a["w_post"], a["w_pre"],
                           a["gate"], 0, 1.0)
    for k in want:
        R.check(got[k], want[k], k)


def test_refusals_on_the_gpu(S):
    a = _inputs(8, 100, 2, 12)
    fw = _forward(S, a, 1.0, keep=True)
    with pytest.raises(ValueError, match="f: expected shape"):
        S.join_forward(a["x"], a["f"][1:], a["w_post"], a["w_pre"])
    with pytest.raises(ValueError, match="w_post: expected shape"):
        S.join_forward(a["x"], a["f"], a["w_post"][1:], a["w_pre"])
    with pytest.raises(ValueError, match="gate"):  # 2 rows, one gate for all
        S.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], a["gate"])
    with pytest.raises(ValueError, match="gate"):  # 8 tokens, 3 to a gate: 3 gates
        S.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], a["gate"], rows_per_gate=3)
    with pytest.raises(ValueError, match="rows_per_gate"):
        S.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], rows_per_gate=3)
    with pytest.raises(S.PPSchedError):
        S.join_forward(a["x"], a["f"], a["w_post"], a["w_pre"], eps=-1.0)
    with pytest.raises(TypeError, match="two checkpoints or two tensors"):
        _backward(S, a, fw["kept_y"], a["f"], fw["rstd_post"], fw["rstd_pre"], 1.0)
    with pytest.raises(TypeError, match="rstd_pre: expected dtype"):
        _backward(S, a, fw["y"], a["f"], fw["rstd_post"], fw["rstd_pre"].double(), 1.0)
    wide = torch.zeros(2, 16385, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(S.PPSchedError):
        S.join_forward(wide, wide, wide[0], wide[0])
