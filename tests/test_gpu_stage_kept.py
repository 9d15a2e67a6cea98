"""Activation checkpoints in 8 bits (stage.pack, unpack, weight_grad) against
their definition: the checkpoint bit for bit, the weight gradient within the
bounds of stage_ref."""
import math

import pytest
import torch

import stage_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from pipeline_schedule_simulation_gb300 import stage
    return stage


def _activation(T, H, seed, **kw):
    g = R.generator(seed)
    x = R.normal(g, T, H, **kw)
    wide = torch.exp(1.5 * torch.randn(H, generator=g, device="cuda"))
    x.copy_((x.float() * wide).to(torch.bfloat16))
    return x


SHAPES = [(1, 1), (1, 64), (3, 63), (7, 1001), (64, 65), (33, 128), (100, 1000), (257, 4096), (2, 65536)]


@pytest.mark.parametrize("T,H", SHAPES)
def test_pack_and_unpack_bit_for_bit(S, T, H):
    x = _activation(T, H, T + H)
    p = S.pack(x)
    q, e = R.pack(x)
    assert torch.equal(p.q, q) and torch.equal(p.e, e)
    assert torch.equal(S.unpack(p).double(), R.value(q, e))
    # half a step of each block's largest magnitude at most
    a = torch.nn.functional.pad(x.double(), (0, -H % 64)).view(T, -1, 64).abs().amax(2)
    assert ((S.unpack(p).double() - x.double()).abs() <= a.repeat_interleave(64, 1)[:, :H] / 128).all()


@pytest.mark.parametrize("stride,offset,qstride", [(104, 0, 100), (100, 0, 112), (103, 1, 101), (200, 8, 128)])
def test_strides_and_offsets(S, stride, offset, qstride):
    T, H = 37, 100
    x = _activation(T, H, 3, stride=stride, offset=offset)
    qb = torch.full((T, qstride), 99, dtype=torch.int8, device="cuda")
    eb = torch.full((T, 5), 99, dtype=torch.int8, device="cuda")
    p = S.pack(x, out=S.Packed(qb[:, :H], eb[:, :2]))
    q, e = R.pack(x)
    assert torch.equal(p.q, q) and torch.equal(p.e, e)
    assert (qb[:, H:] == 99).all() and (eb[:, 2:] == 99).all()
    back = torch.full((T, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    S.unpack(p, out=back[:, :H])
    assert torch.equal(back[:, :H].double(), R.value(q, e)) and (back[:, H:] == 7).all()


def test_extreme_values(S):
    """Ties, the value that would round to 128, both ends of the exponent, zeros, infinities and NaN."""
    x = torch.zeros(12, 130, device="cuda")
    x[0, :4] = torch.tensor([127.5, -127.5, 0.5, 1.5])          # step 1: 127.5 is held as 127, ties go to even
    x[1, 0], x[1, 64] = 3.3895e38, 1.0                          # bf16's largest
    x[2, 0], x[2, 64] = 2.0 ** -126, 2.0 ** -133                # its smallest normal and subnormal number
    x[3, 5], x[4, 70], x[5, 129] = math.inf, -math.inf, math.nan
    x[6, :] = -0.0
    x[7, :] = torch.arange(130) / 8
    x[8, 63], x[8, 64] = 1e30, 1e-30                            # neighbours in two blocks
    x[9, 3], x[9, 4] = math.nan, math.inf
    x[10, :64] = 2.0 ** -120 * torch.arange(64)
    x = x.to(torch.bfloat16)
    p = S.pack(x)
    q, e = R.pack(x)
    assert torch.equal(p.q, q) and torch.equal(p.e, e)
    got, want = S.unpack(p).double(), R.value(q, e)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0), want.nan_to_num(0))
    assert want[3, :64].isnan().all() and not want[3, 64:].isnan().any()
    assert p.q[0, 0] == 127 and p.q[0, 2] == 0 and p.q[0, 3] == 2


def test_no_rows(S):
    x = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    p = S.pack(x)
    assert p.shape == (0, 100) and S.unpack(p).shape == (0, 100)
    dy = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    assert (S.weight_grad(dy, p) == 0).all()
    add = torch.full((8, 100), 2.0, device="cuda")
    assert torch.equal(S.weight_grad(dy, p, add=add), add)
    assert S.weight_grad(dy, p, add=add, out=add) is add and (add == 2).all()


@pytest.mark.parametrize("T,N,H", [(1, 1, 1), (1, 64, 64), (3, 70, 1001), (63, 128, 64), (65, 129, 65), (200, 1024, 1000),
                                   (128, 256, 256), (129, 257, 264), (1000, 40, 72), (4096, 64, 130), (511, 520, 511),
                                   # enough tiles for pairs of blocks
                                   (100, 2000, 2010), (300, 1411, 2000), (65, 3000, 1025),
                                   # long sums: whole lines, parts of K
                                   (2050, 2000, 1500), (2048, 1300, 2052), (5000, 136, 140)])
@pytest.mark.parametrize("how", ["new", "add", "in place"])
def test_weight_grad(S, T, N, H, how):
    g = R.generator(T + N + H)
    dy = R.normal(g, T, N, scale=0.1)
    p = S.pack(_activation(T, H, T * N + H))
    v = R.value(p.q, p.e)
    add = None if how == "new" else torch.randn(N, H, generator=g, device="cuda")
    before = None if add is None else add.clone()
    got = S.weight_grad(dy, p, add=add, out=add if how == "in place" else None)
    R.check(got, R.weight_grad(dy, v, before), how)
    if how == "add":
        assert torch.equal(add, before)


@pytest.mark.parametrize("stride,offset", [(77, 0), (80, 1), (96, 8)])
def test_weight_grad_strides(S, stride, offset):
    T, N, H = 130, 75, 90
    dy = R.normal(R.generator(1), T, N, stride=stride, offset=offset)
    x = _activation(T, H, 2)
    q, e = R.pack(x)
    qb = torch.full((T, 93), 55, dtype=torch.int8, device="cuda")
    qb[:, 1:91] = q
    add = torch.randn(75, 200, device="cuda")[:, 7:97]
    out = torch.full((75, 91), 7.0, device="cuda")
    got = S.weight_grad(dy, S.Packed(qb[:, 1:91], e), add=add, out=out[:, :90])
    R.check(got, R.weight_grad(dy, R.value(q, e), add))
    assert (out[:, 90:] == 7).all()


def test_weight_grad_is_exact_on_small_whole_numbers(S):
    """Whole numbers whose sums fit 24 bits: no rounding anywhere."""
    g = R.generator(4)
    T, N, H = 300, 200, 192
    dy = torch.randint(-8, 9, (T, N), generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randint(-127, 128, (T, H), generator=g, device="cuda").to(torch.bfloat16)
    x[:, ::64] = 127.0  # every block's step is 1
    p = S.pack(x)
    assert torch.equal(S.unpack(p), x)
    assert torch.equal(S.weight_grad(dy, p).double(), dy.double().t() @ x.double())


def test_weight_grad_nan_stays_in_its_block(S):
    x = _activation(50, 192, 5)
    x[7, 70] = math.inf
    p = S.pack(x)
    dy = R.normal(R.generator(6), 50, 33)
    got = S.weight_grad(dy, p)
    assert got[:, 64:128].isnan().all() and torch.isfinite(got[:, :64]).all() and torch.isfinite(got[:, 128:]).all()


def test_weight_grad_against_differences(S):
    """dw of sum(dy * (v w^T)) along a direction, by differences in 64 bits (the function is linear)."""
    g = R.generator(8)
    T, N, H = 64, 48, 100
    dy, p = R.normal(g, T, N), S.pack(_activation(T, H, 9))
    v = R.value(p.q, p.e)
    u, w = (torch.randn(N, H, generator=g, device="cuda", dtype=torch.float64) for _ in range(2))
    f = lambda m: (dy.double() * (v @ m.t())).sum()  # noqa: E731
    diff = (f(w + 0.5 * u) - f(w - 0.5 * u))
    got, bound = S.weight_grad(dy, p), R.weight_grad(dy, v)[1]
    assert abs((got.double() * u).sum() - diff) <= (bound * u.abs()).sum() + 1e-9 * abs(diff)


def test_same_on_every_call_and_on_another_stream(S):
    g = R.generator(10)
    dy, p = R.normal(g, 3000, 130), S.pack(_activation(3000, 200, 11))
    first = S.weight_grad(dy, p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = S.weight_grad(dy, p, stream=s)
    s.synchronize()
    assert torch.equal(first, again)


def test_offsets_past_32_bits(S):
    T, H = 3, 96
    stride = (1 << 30) + 64
    buf = torch.zeros(T * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((T, H), (stride, 1))
    x.copy_(_activation(T, H, 12))
    qbuf = torch.zeros(T * stride, dtype=torch.int8, device="cuda").as_strided((T, H), (stride, 1))
    p = S.pack(x, out=S.Packed(qbuf, torch.zeros(T, 2, dtype=torch.int8, device="cuda")))
    q, e = R.pack(x)
    assert torch.equal(p.q, q)
    back = torch.zeros_like(buf).as_strided((T, H), (stride, 1))
    assert torch.equal(S.unpack(p, out=back).double(), R.value(q, e))
    R.check(S.weight_grad(x, p), R.weight_grad(x, R.value(q, e)))


def test_refusals_on_the_gpu(S):
    x = _activation(8, 100, 13)
    p = S.pack(x)
    with pytest.raises(TypeError, match="x: expected dtype"):
        S.pack(x.float())
    with pytest.raises(ValueError, match="e: expected shape"):
        S.Packed(p.q, p.e[:, :1])
    with pytest.raises(TypeError, match="q: expected dtype"):
        S.Packed(x, p.e)
    with pytest.raises(TypeError, match="Packed"):
        S.unpack(x)
    with pytest.raises(ValueError, match="out: expected shape"):
        S.unpack(p, out=torch.empty(8, 99, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="rows"):
        S.weight_grad(x[1:], p)
    with pytest.raises(ValueError, match="add: expected shape"):
        S.weight_grad(x, p, add=torch.zeros(100, 101, device="cuda"))
    with pytest.raises(TypeError, match="out: expected dtype"):
        S.weight_grad(x, p, out=torch.zeros(100, 100, dtype=torch.bfloat16, device="cuda"))
