"""The block operators at the edges of their values: infinities and overflow, steps far below
one, arguments that are not there."""
import pytest
import torch

import block_reference as ref
import test_block_gpu as tb
from block_reference import U32, f64, half_step
from state_space_model_06_b200 import m3

F32 = torch.float32


def nearest_e4m3(p, m):
    """448 p / m rounded to the nearest e4m3 value, ties to even, and how far it lies from the
    middle of two (relative).  p and m are exact products of two fp32 values: 448 p and a middle
    (five bits) times m are exact in 64 bits, so the comparison is."""
    q = 448 * p.abs() / m
    unit = torch.ldexp(torch.ones_like(q), torch.frexp(q.clamp(min=2.0 ** -6)).exponent - 4)
    k = torch.floor(q / unit)
    gap = 448 * p.abs() - (k + 0.5) * unit * m
    up = torch.where(gap == 0, k % 2 == 1, gap > 0)
    return torch.copysign((k + up) * unit, p), gap.abs() / (448 * p.abs() + 1e-300)


def near_middles(rows, d, weighted, seed):
    """Rows and weights whose quotients lie next to the middle of two e4m3 steps, but for a group's
    largest; the exact products and each value's largest."""
    n = -(-d // 128)
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn((rows, d), generator=g)
    w = 1 + 0.2 * torch.randn(d, generator=g) if weighted else torch.ones(d)
    p = x.double() * w.double()
    at = torch.arange(d) // 128
    pad = torch.zeros(rows, n * 128, dtype=torch.float64)
    pad[:, :d] = p.abs()
    top, where = pad.view(rows, n, 128).max(-1)
    # every other value of a group is the fp32 value next to a middle of two steps
    keep = torch.zeros(rows, n * 128, dtype=torch.bool)
    keep.scatter_(1, where + 128 * torch.arange(n), True)
    steps = torch.arange(8, 16).double() + 0.5
    middle = steps[torch.randint(0, 8, (rows, d), generator=g)] * \
        2.0 ** torch.randint(-9, 5, (rows, d), generator=g)
    near = (middle * top[:, at] / 448 / w.double()).float()
    x = torch.where(keep[:, :d], x, torch.copysign(near, x))
    return x, w, x.double() * w.double(), top[:, at]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [2048, 1000])
@pytest.mark.parametrize("weighted", [True, False])
def test_norm_e4m3_values_are_the_nearest(weighted, d):
    """Values next to the middle of two e4m3 steps: each goes to the nearer one, and those in the
    middle itself (without a weight there are some) to the even one."""
    rows = 96
    x, w, p, top = near_middles(rows, d, weighted, 55)
    want, gap = nearest_e4m3(p, top)
    assert (gap < 2.0 ** -22).sum() > 0.9 * rows * d
    dims = m3.NormDims(rows, d, m3.M3_F32, m3.M3_F32, m3.M3_OUT_E4M3)
    q = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
    m3.m3_norm_fwd(dims, x.cuda(), None, w.cuda() if weighted else None, 1e-6, q,
                   m3.alloc_norm_scales(dims))
    got = f64(q.float())
    assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("weights", [None, [1.0], [0.5, 0.625, 0.75, 1.0, 1.25, 1.875], [1.0, 1.0625]])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d", [2048, 1000])
def test_norm_e4m3_of_short_values(d, residual, weights):
    """bf16 values without weights, or with weights of few bits: about one in a hundred lies in the
    middle of two steps.  Weights of four bits and of five, one more than the short way takes."""
    g = torch.Generator().manual_seed(56)
    x = torch.randn((64, d), generator=g).bfloat16()
    res = torch.randn((64, d), generator=g).bfloat16() if residual else None
    r = x if res is None else (x.float() + res.float()).bfloat16()
    n = -(-d // 128)
    pad = torch.zeros(64, n * 128, dtype=torch.float64)
    w = None if weights is None else torch.tensor(weights)[torch.randint(0, len(weights), (d,),
                                                                         generator=g)]
    p = r.double() if w is None else r.double() * w.double()
    pad[:, :d] = p.abs()
    top = pad.view(64, n, 128).amax(-1)[:, torch.arange(d) // 128]
    want, gap = nearest_e4m3(p, top)
    assert (gap == 0).sum() > 64 * d / 1000
    dims = m3.NormDims(64, d, m3.M3_BF16, m3.M3_BF16, m3.M3_OUT_E4M3)
    q = torch.empty(64, d, dtype=torch.float8_e4m3fn, device="cuda")
    m3.m3_norm_fwd(dims, x.cuda(), None if res is None else res.cuda(),
                   None if w is None else w.cuda(), 1e-6, q,
                   m3.alloc_norm_scales(dims))
    assert torch.equal(f64(q.float()), want)


@pytest.mark.gpu
def test_norm_e4m3_of_short_values_and_huge_weights():
    """Weights that are powers of two up to 2^126: 448 times a product is past fp32, y is not."""
    g = torch.Generator().manual_seed(59)
    x = torch.randn((16, 1024), generator=g).clamp(-1, 1).bfloat16()
    w = 2.0 ** torch.tensor([0.0, 60, 100, 112, 116, 118, 122, 126]).repeat_interleave(128)
    p = x.double() * w.double()
    top = p.abs().view(16, 8, 128).amax(-1)
    want, _ = nearest_e4m3(p, top.repeat_interleave(128, 1))
    dims = m3.NormDims(16, 1024, m3.M3_BF16, m3.M3_BF16, m3.M3_OUT_E4M3)
    q = torch.empty(16, 1024, dtype=torch.float8_e4m3fn, device="cuda")
    sc = m3.alloc_norm_scales(dims)
    m3.m3_norm_fwd(dims, x.cuda(), None, w.cuda(), 1e-6, q, sc)
    scale = top / 448 / torch.sqrt(x.double().square().mean(1, keepdim=True) + 1e-6)
    assert (scale < 2.0 ** 119).all()
    tb.near(sc, scale, (tb.rounds(1024) + 4) * U32 * scale, "scales")
    assert torch.equal(f64(q.float()), want)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [512, 500])
def test_norm_infinite_products_have_nan_scales(d):
    """An infinite weight, and a product of finite factors that overflows: the group holds an
    infinity, so its scale is NaN, in wide rows and narrow ones; the other groups are as without."""
    g = torch.Generator().manual_seed(51)
    x, w = torch.randn((3, d), generator=g).cuda(), 1 + torch.rand(d, generator=g).cuda()
    dims = m3.NormDims(3, d, m3.M3_F32, m3.M3_F32, m3.M3_OUT_E4M3)

    def run(w):
        q = torch.empty(3, d, dtype=torch.float8_e4m3fn, device="cuda")
        sc = m3.alloc_norm_scales(dims)
        m3.m3_norm_fwd(dims, x, None, w, 1e-6, q, sc)
        return q.float(), sc

    x[:, 130], x[:, 300] = 4.0, 0.5
    q0, s0 = run(w)
    w[130] = 3.0e38                  # y = 4 / rms * 3e38 is past the largest fp32 value
    w[300] = float("-inf")
    q, sc = run(w)
    assert torch.isnan(sc[:, 1:3]).all() and torch.isnan(q[:, 128:384]).all()
    assert torch.equal(sc[:, [0, 3]], s0[:, [0, 3]])
    assert torch.equal(q[:, :128], q0[:, :128]) and torch.equal(q[:, 384:], q0[:, 384:])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [2048, 1000])
def test_norm_e4m3_beside_a_spoiled_group(d):
    """Open values of a warp whose other group is NaN, and the other way round."""
    rows = 24
    x, w, p, top = near_middles(rows, d, True, 57)
    want, _ = nearest_e4m3(p, top)
    w[300], w[700] = float("inf"), float("nan")
    spoiled = torch.zeros(d, dtype=torch.bool)
    spoiled[256:384] = spoiled[640:768] = True
    dims = m3.NormDims(rows, d, m3.M3_F32, m3.M3_F32, m3.M3_OUT_E4M3)
    q = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
    sc = m3.alloc_norm_scales(dims)
    m3.m3_norm_fwd(dims, x.cuda(), None, w.cuda(), 1e-6, q, sc)
    q = f64(q.float())
    assert torch.equal(q[:, ~spoiled], want[:, ~spoiled]) and torch.isnan(q[:, spoiled]).all()
    assert torch.isnan(sc[:, [2, 5]]).all() and torch.isnan(sc).sum() == 2 * rows


@pytest.mark.gpu
def test_norm_e4m3_below_the_floor():
    """Groups whose largest y is next to 2^-100: above it their own scale, below it the floor's."""
    rows, d = 16, 1024
    g = torch.Generator().manual_seed(58)
    x, w = torch.randn((rows, d), generator=g), 1 + torch.rand(d, generator=g)
    for i, e in enumerate((-99, -101, -103, -106, -110, -120, -126)):
        w[128 * i:128 * (i + 1)] *= 2.0 ** e
    dims = m3.NormDims(rows, d, m3.M3_F32, m3.M3_F32, m3.M3_OUT_E4M3)
    q = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
    sc = m3.alloc_norm_scales(dims)
    m3.m3_norm_fwd(dims, x.cuda(), None, w.cuda(), 1e-6, q, sc)
    y, _ = ref.norm(x.double(), None, w.double(), 1e-6, F32)
    scale = y.view(rows, 8, 128).abs().amax(-1).clamp(min=2.0 ** -100) / 448
    tb.near(sc, scale, (tb.rounds(d) + 4) * U32 * scale, "scales")
    assert (scale[:, 0] > 2.0 ** -100 / 448).all() and (scale[:, 1:7] == 2.0 ** -100 / 448).sum() > 70
    v = y / scale.repeat_interleave(128, 1)
    # half a step of the value that is rounded, off by the roundings of the mean, the root and y
    tb.near(q.float(), v, tb.e4m3_steps(v) * (1 + 2.0 ** -10) + tb.rounds(d) * U32 * v.abs(), "values")


def test_binding_names_what_is_missing():
    """A call's first tensor decides its device: without it the call ends as with any other
    argument that is needed and not there."""
    for call in (lambda: m3.m3_conv_fwd(m3.ConvDims(1, 8, 4), 3, *[None] * 5),
                 lambda: m3.m3_conv_step(m3.ConvDims(1, 8, 4), *[None] * 5),
                 lambda: m3.m3_sel_fwd(m3.SelDims(1, 8, 1, 4), 3, *[None] * 11),
                 lambda: m3.m3_sel_step(m3.SelDims(1, 8, 1, 4), *[None] * 10),
                 lambda: m3.m3_norm_fwd(m3.NormDims(2, 8), None, None, None, 1e-6, None),
                 lambda: m3.m3_norm_bwd(m3.NormDims(2, 8), None, None, 1e-6, *[None] * 6)):
        with pytest.raises(m3.M3Error) as e:
            call()
        assert e.value.status == m3.M3_ERR_NULL


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["prompt", "step"])
def test_scan_step_after_softplus(call):
    """The step itself: from a zero state, x = B = 1 leave h = delta.

    With U = 2^-24 and v < 0, u = e^v is off by 1.22 |v| U for its argument (the rounded product
    |v| log2(e), and log2(e) itself) and by 4 U for the hardware's exponential.  s = u / (2 + u)
    adds 1 U for the sum, 2 U for the reciprocal and 1 U for the product; 2 atanh(s) = log(1 + u)
    magnifies what has come together so far by at most 1.09 (s <= 1/3), and adds 2 U for the
    series, its fit and the last sum.  In all (1.33 |v| + 11) U.  For v > 0 the same is relative
    to the smaller of two positive terms, whose sum rounds once more."""
    n = 4096
    v = torch.linspace(-85.0, 40.0, n)
    dt = v.cuda()
    want = torch.logaddexp(f64(dt), torch.zeros(1, dtype=torch.float64))
    one, h = torch.ones(1, n, device="cuda"), torch.zeros(1, n, 1, device="cuda")
    bc, A = torch.ones(1, 1, 1, device="cuda"), -torch.ones(n, 1, device="cuda")
    d = m3.SelDims(1, n, 1, 1, m3.M3_F32)
    y, flags = torch.empty_like(one), m3.M3_FLAG_DT_SOFTPLUS
    if call == "step":
        m3.m3_sel_step(d, one, dt[None], A, bc, bc, None, None, None, h, y, flags=flags)
    else:
        m3.m3_sel_fwd(d, 1, one[None], dt[None, None], A, bc[None], bc[None], None, None, None, h,
                      y[None], None, flags=flags)
    tol = (1.33 * f64(dt).abs() + 12) * U32 * want
    tb.near(h.view(-1), want, tol, "delta")
    assert torch.equal(y.view(-1), h.view(-1))


def minus_infinity(T, ch, N, seed):
    """A prompt with softplus where some steps' dt is -inf, in 64 bits too, and an equal one with
    -1000 there (whose softplus is 0 as well) for the bounds."""
    c, _, sp = tb.scan_inputs((2, T, ch, 1, N, F32, "z D bias softplus"), seed)
    r = {k: f64(v) for k, v in c.items()}
    for t in (c["dt"], r["dt"]):
        t[0, 3, 1], t[1, T - 1, 2], t[:, T // 2] = -1000.0, -1000.0, -1000.0
    bound = ref.scan_bounds(T, N, ch, r["A"], torch.clamp(r["dt"], min=-20), r["bias"], True)
    for t in (c["dt"], r["dt"]):
        t[t == -1000.0] = float("-inf")
    return c, r, bound


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 200])
def test_scan_step_of_minus_infinity(T):
    """With softplus a dt of -inf is a step of zero: the token leaves the state, and nothing
    becomes infinite or NaN, forward and backward."""
    ch, N = 8, 16
    c, r, rel = minus_infinity(T, ch, N, 52)
    lens = [T, T]
    y, h = tb.run_scan((2, T, ch, 1, N, F32, ""), c, None, True)
    (want_y, want_h), (mag_y, mag_h) = (ref.scan(*r.values(), lens, True, absolute=a)
                                        for a in (False, True))
    tb.near(h, want_h, rel * mag_h + 1e-37, "h")
    tb.near(y, want_y, half_step(F32) * want_y.abs() + (rel + 2.0 ** -20) * mag_y + 1e-37, "y")
    g = torch.Generator().manual_seed(53)
    dy, dhT = tb.rnd(g, 2, T, ch), tb.rnd(g, 2, ch, N)
    want, mag = (ref.scan_bwd(*r.values(), lens, True, f64(dy), f64(dhT), absolute=a)
                 for a in (False, True))
    d = m3.SelDims(2, ch, 1, N, m3.M3_F32)
    gr = {k: tb.nan_like(v) for k, v in m3.alloc_sel_grads(d, T).items()}
    m3.m3_sel_bwd(d, T, c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["bias"],
                  c["h"], dy, dhT, gr, m3.alloc_sel_bwd_workspace(d, T),
                  flags=m3.M3_FLAG_DT_SOFTPLUS)
    for k, v in gr.items():
        tol = (2 * rel + 2.0 ** -19 + U32 * (ch + 2 * T + 1)) * mag[k] + 1e-37
        tb.near(v, want[k], tol, k)


@pytest.mark.gpu
@pytest.mark.parametrize("T,workspace", [(40, False), (300, True)])
@pytest.mark.parametrize("name", ["x", "dt", "B", "z", "C"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_scan_where_an_infinity_goes(name, value, T, workspace):
    """x, dt and B spoil the state and the outputs from their token on, z and C the outputs of
    their token alone; x, dt and z those of their channel, B and C those of their group."""
    case = (1, T, 12, 2, 16, F32, "z D bias softplus")
    c, _, sp = tb.scan_inputs(case, 54)
    base, h0 = tb.run_scan(case, c, None, sp, workspace)
    at, per = 33, slice(6, 12) if name in ("B", "C") else slice(7, 8)
    if name in ("B", "C"):
        c[name][0, at, 1, 3] = value
    else:
        c[name][0, at, 7] = value
    y, h = tb.run_scan(case, c, None, sp, workspace)
    bad = torch.zeros_like(base, dtype=torch.bool)
    bad[0, at:at + 1 if name in ("z", "C") else T, per] = True
    assert not torch.isfinite(y[bad]).any()
    assert torch.equal(y[~bad], base[~bad])
    others = [i for i in range(12) if not per.start <= i < per.stop]
    assert torch.equal(h[:, others], h0[:, others])
    if name in ("z", "C"):
        assert torch.equal(h, h0)
    elif name == "B":
        assert not torch.isfinite(h[0, per, 3]).any()
    else:
        assert not torch.isfinite(h[0, per]).any()
