"""Block operators (m3_conv_*, m3_sel_*, m3_norm_*) on the GPU against their plain 64-bit forms,
at the sizes, strides and lengths where they can go wrong.

Tolerances: an output is off by half a step of its type, and by the 32-bit errors of its terms,
counted against the sum of their absolute values (block_reference)."""
import pytest
import torch

import block_reference as ref
from block_reference import EX2, U32, f64, half_step
from state_space_model_06_b200 import m3

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rnd(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def near(got, want, tol, what):
    """Every element of got within tol (same shape) of want."""
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / tol).nan_to_num(9e9).max()))


def nan_like(t):
    return torch.full_like(t, float("nan"))


# ---------------------------------------------------------------- convolution

CONV = [  # b, T, C, W, dtype, options
    (2, 37, 64, 4, BF, "silu bias"),
    (1, 1, 8, 4, BF, "silu bias"),
    (1, 2, 24, 4, F32, "bias"),                   # shorter than the window
    (3, 130, 33, 3, BF, "silu bias"),             # odd channels: element by element
    (2, 65, 40, 2, F32, "silu"),
    (2, 50, 72, 8, BF, "silu bias"),
    (2, 9, 16, 1, F32, "silu bias"),              # no state
    (2, 300, 1032, 4, BF, "silu bias sliced"),
    (2, 70, 64, 4, F32, "silu bias ragged"),
    (5, 129, 20, 4, BF, "ragged sliced"),
    (3, 40, 36, 4, F32, "silu bias odd"),         # rows that start off 16 bytes
    (2, 33, 64, 4, BF, "silu bias tfirst"),       # [T][b][C] in memory
    (1, 1200, 2048, 4, BF, "silu bias"),
]


def conv_inputs(case, seed):
    b, T, C, W, io, opt = case
    g = torch.Generator().manual_seed(seed)
    x = rnd(g, b, T, C, dtype=io)
    if "sliced" in opt:
        x = rnd(g, b, T, 2 * C, dtype=io)[..., C:]
    if "odd" in opt:
        x = rnd(g, b, T, C + 3, dtype=io)[..., 1:C + 1]
    if "tfirst" in opt:
        x = rnd(g, T, b, C, dtype=io).transpose(0, 1)
    w = rnd(g, C, W, std=W ** -0.5)
    bias = rnd(g, C, std=0.3) if "bias" in opt else None
    state = rnd(g, b, W - 1, C, dtype=io)
    lens = None
    if "ragged" in opt:
        lens = torch.tensor([T, 0, 1, 2, T // 2, T + 9, -3][:b], dtype=torch.int32).cuda()
    return x, w, bias, state, lens, "silu" in opt


def conv_tol(case, args, lens, act, y):
    """W products and sums and the bias on |terms|, SiLU's slope (at most 1.1) on top, and the
    sigmoid's own relative error (bf16: a few 2^-21 of the hardware functions)."""
    x, w, bias, state = (f64(v) for v in args)
    mag = ref.conv(x.abs(), w.abs(), None if bias is None else bias.abs(), state.abs(), lens, False)[0]
    return half_step(case[4]) * y.abs() + 1.1 * (case[3] + 3) * U32 * mag + \
        (2.0 ** -20 * (y.abs() + mag) if act else 0) + 1e-37


@pytest.mark.parametrize("case", CONV)
def test_conv_fwd(case):
    b, T, C, W, io, _ = case
    x, w, bias, state, sl, act = conv_inputs(case, 1)
    lens = ref.lengths(sl, b, T)
    y, new = ref.conv(*(f64(v) for v in (x, w, bias, state)), lens, act)
    tol = conv_tol(case, (x, w, bias, state), lens, act, y)
    d = m3.ConvDims(b, C, W, m3.io_dtype_of(io))
    out = nan_like(torch.empty(b, T, C, dtype=io, device="cuda"))
    m3.m3_conv_fwd(d, T, x, w, bias, state, out, seqlens=sl, flags=m3.M3_FLAG_SILU if act else 0)
    near(out, y, tol, "y")
    assert torch.equal(f64(state), new)


@pytest.mark.parametrize("case", CONV)
def test_conv_step_continues_a_prompt(case):
    """Three single tokens after a prompt, in place on x."""
    b, T, C, W, io, opt = case
    x, w, bias, state, sl, act = conv_inputs(case, 2)
    flags = m3.M3_FLAG_SILU if act else 0
    d = m3.ConvDims(b, C, W, m3.io_dtype_of(io))
    want = f64(state)
    m3.m3_conv_fwd(d, T, x, w, bias, state, torch.empty(b, T, C, dtype=io, device="cuda"),
                   seqlens=sl, flags=flags)
    want = ref.conv(f64(x), f64(w), f64(bias), want, ref.lengths(sl, b, T), act)[1]
    g = torch.Generator().manual_seed(3)
    for _ in range(3):
        wide = rnd(g, b, C + 5, dtype=io)
        tok = wide[:, :C] if "odd" in opt else wide[:, :C].contiguous()
        y, new = ref.conv(f64(tok)[:, None], f64(w), f64(bias), want, [1] * b, act)
        tol = conv_tol(case, (tok[:, None], w, bias, state), [1] * b, act, y)[:, 0]
        m3.m3_conv_step(d, tok, w, bias, state, tok, flags=flags)
        near(tok, y[:, 0], tol, "y")
        assert torch.equal(f64(state), new)
        want = new


@pytest.mark.parametrize("case", CONV)
def test_conv_bwd(case):
    b, T, C, W, io, opt = case
    x, w, bias, state, sl, act = conv_inputs(case, 4)
    g = torch.Generator().manual_seed(5)
    dy = rnd(g, b, T, C, dtype=io)
    if sl is not None:          # rows past a length are looked at by nothing
        for i, n in enumerate(ref.lengths(sl, b, T)):
            dy[i, n:] = float("inf")
            x[i, n:] = float("nan")
    lens = ref.lengths(sl, b, T)
    args = [f64(v) for v in (x, w, bias, state)]
    want = ref.conv_bwd(*args, lens, act, f64(dy))
    mag = ref.conv_bwd(*args, lens, act, f64(dy), absolute=True)
    d = m3.ConvDims(b, C, W, m3.io_dtype_of(io))
    gr = {k: nan_like(v) for k, v in m3.alloc_conv_grads(d, T).items()}
    ws = m3.alloc_conv_bwd_workspace(d, T)
    before = state.clone()
    m3.m3_conv_bwd(d, T, x, w, bias, state, dy, gr, ws, seqlens=sl,
                   flags=m3.M3_FLAG_SILU if act else 0)
    assert torch.equal(before, state)
    # the activation's slope moves with pre's error: |act''| <= 1/2 on (W + 3) U32 |terms|
    pre = (args[1].abs().sum(1).max() * max(float(args[0].nan_to_num().abs().max()),
                                            float(args[3].abs().max()) if args[3].numel() else 0.0)
           + (0 if bias is None else float(args[2].abs().max())))
    rel = (W + 6) * U32 + (2.0 ** -19 + 0.5 * (W + 3) * U32 * float(pre) * 8 if act else 0)
    for k in ("dx", "dweight", "dbias", "dstate"):
        if k == "dbias" and bias is None:
            continue
        if k == "dx":
            tol = half_step(io) * want[k].abs() + rel * mag[k] + 1e-37
        else:                    # summed over up to 128 tokens of a run, then over the runs
            tol = (rel + (128 + b * T / 8 + 8) * U32) * mag[k] + 1e-37
        near(gr[k], want[k], tol, k)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("C", [64, 37])
@pytest.mark.parametrize("W", range(1, 9))
def test_conv_every_width(W, C, io):
    """Each filter width, wide rows and narrow ones, forward and backward."""
    case = (2, 45, C, W, io, "silu bias")
    test_conv_fwd(case)
    test_conv_bwd(case)


# ---------------------------------------------------------------- selective scan

SCAN = [  # b, T, ch, G, N, dtype, options
    (2, 37, 64, 1, 16, BF, "z D bias softplus"),
    (1, 1, 8, 1, 16, BF, "z D bias softplus"),
    (2, 65, 130, 2, 16, F32, "z D bias softplus"),
    (1, 33, 20, 1, 1, F32, "softplus"),
    (2, 40, 36, 3, 4, F32, "z bias softplus"),
    (1, 70, 24, 1, 7, BF, "D"),                       # steps as they are
    (2, 96, 48, 1, 24, F32, "z D bias softplus odd"),
    (1, 50, 40, 1, 33, BF, "z D bias softplus sliced"),
    (2, 66, 16, 2, 64, F32, "z D bias softplus"),
    (1, 40, 12, 1, 100, F32, "z D bias softplus"),
    (1, 35, 10, 1, 256, BF, "z D softplus"),
    (4, 70, 72, 1, 16, F32, "z D bias softplus ragged"),
    (6, 129, 65, 1, 8, BF, "z D bias softplus ragged sliced"),
    (2, 64, 32, 1, 16, BF, "z D bias softplus tfirst"),
    (1, 600, 96, 1, 16, F32, "z D bias softplus"),     # segmented
    (2, 513, 40, 2, 20, BF, "z D bias softplus ragged"),
    (1, 31, 200, 1, 2, F32, "z D bias softplus"),
]


def scan_inputs(case, seed):
    b, T, ch, G, N, io, opt = case
    g = torch.Generator().manual_seed(seed)

    def act(*tail):
        n = 1
        for v in tail:
            n *= v
        if "sliced" in opt:
            t = rnd(g, b, T, 2 * n + 8, dtype=io)[..., n:2 * n]
        elif "odd" in opt:
            t = rnd(g, b, T, n + 5, dtype=io)[..., 3:n + 3]
        elif "tfirst" in opt:
            t = rnd(g, T, b, n, dtype=io).transpose(0, 1)
        else:
            t = rnd(g, b, T, n, dtype=io)
        return t.unflatten(-1, tail) if len(tail) > 1 else t

    words = opt.split()
    c = dict(x=act(ch), dt=act(ch), A=None, B=act(G, N), C=act(G, N))
    if "softplus" not in words:
        c["dt"] = c["dt"].abs() * 0.1
    c["A"] = -torch.exp(rnd(g, ch, N, std=0.7))
    c["D"] = rnd(g, ch) if "D" in words else None
    c["z"] = act(ch) if "z" in words else None
    c["bias"] = rnd(g, ch) - 2.0 if "bias" in words else None
    c["h"] = rnd(g, b, ch, N)
    sl = None
    if "ragged" in words:
        sl = torch.tensor([T, 0, 1, T // 2, T + 9, -3][:b], dtype=torch.int32).cuda()
    return c, sl, "softplus" in words


def poison(c, sl, b, T):
    """Rows past a length hold NaN: nothing may read them."""
    if sl is not None:
        for i, n in enumerate(ref.lengths(sl, b, T)):
            for k in ("x", "dt", "B", "C", "z"):
                c[k][i, n:] = float("nan")


def clean(c, sl, b, T):
    out = {k: f64(v) for k, v in c.items()}
    if sl is not None:
        for i, n in enumerate(ref.lengths(sl, b, T)):
            for k in ("x", "dt", "B", "C", "z"):
                out[k][i, n:] = 0
    return out


def run_scan(case, c, sl, sp, workspace=True):
    b, T, ch, G, N, io, _ = case
    d = m3.SelDims(b, ch, G, N, m3.io_dtype_of(io))
    y = torch.full((b, T, ch), float("nan"), dtype=io, device="cuda")
    h = c["h"].clone()
    ws = m3.alloc_sel_workspace(d, T).fill_(255) if workspace else None
    m3.m3_sel_fwd(d, T, c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["bias"], h, y,
                  ws, seqlens=sl, flags=m3.M3_FLAG_DT_SOFTPLUS if sp else 0)
    return y, h


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("case", SCAN)
def test_scan_fwd(case, workspace):
    b, T, ch, G, N, io, _ = case
    c, sl, sp = scan_inputs(case, 11)
    poison(c, sl, b, T)
    lens, r = ref.lengths(sl, b, T), clean(c, sl, b, T)
    want_y, want_h = ref.scan(*r.values(), lens, sp)
    mag_y, mag_h = ref.scan(*r.values(), lens, sp, absolute=True)
    rel = ref.scan_bounds(T, N, ch, r["A"], r["dt"], r["bias"], sp)
    y, h = run_scan(case, c, sl, sp, workspace)
    near(h, want_h, rel * mag_h + 1e-37, "h")
    near(y, want_y, half_step(io) * want_y.abs() + (rel + 2.0 ** -20) * mag_y + 1e-37, "y")
    for i, n in enumerate(lens):
        assert not f64(y)[i, n:].any()


@pytest.mark.parametrize("case", SCAN)
def test_scan_step_continues_a_prompt(case):
    b, T, ch, G, N, io, opt = case
    c, sl, sp = scan_inputs(case, 12)
    _, h = run_scan(case, c, sl, sp)
    d = m3.SelDims(b, ch, G, N, m3.io_dtype_of(io))
    fresh, _, _ = scan_inputs((b, 3, ch, G, N, io, opt), 13)
    for t in range(3):
        one = {k: fresh[k][:, t] if k in ("x", "dt", "B", "C", "z") and fresh[k] is not None
               else c[k] for k in c}
        r = {k: (f64(v)[:, None] if k in ("x", "dt", "B", "C", "z") and v is not None else f64(v))
             for k, v in dict(one, h=h).items()}
        want_y, want_h = ref.scan(*r.values(), [1] * b, sp)
        mag_y, mag_h = ref.scan(*r.values(), [1] * b, sp, absolute=True)
        rel = ref.scan_bounds(1, N, ch, r["A"], r["dt"], r["bias"], sp)
        y = one["x"] if t == 1 else torch.full((b, ch), float("nan"), dtype=io, device="cuda")
        m3.m3_sel_step(d, one["x"], one["dt"], c["A"], one["B"], one["C"], c["D"], one["z"],
                       c["bias"], h, y, flags=m3.M3_FLAG_DT_SOFTPLUS if sp else 0)
        near(h, want_h, rel * mag_h + 1e-37, "h")
        near(y, want_y[:, 0], (half_step(io) * want_y.abs() + (rel + 2.0 ** -20) * mag_y)[:, 0]
             + 1e-37, "y")


@pytest.mark.parametrize("case", SCAN)
def test_scan_bwd(case):
    b, T, ch, G, N, io, opt = case
    c, sl, sp = scan_inputs(case, 14)
    poison(c, sl, b, T)
    g = torch.Generator().manual_seed(15)
    dy = rnd(g, b, T, ch, dtype=io)
    dhT = rnd(g, b, ch, N) if N != 7 else None
    lens, r = ref.lengths(sl, b, T), clean(c, sl, b, T)
    rdy = f64(dy)
    if sl is not None:
        for i, n in enumerate(lens):
            dy[i, n:] = float("inf")
            rdy[i, n:] = 0
    want = ref.scan_bwd(*r.values(), lens, sp, rdy, f64(dhT))
    mag = ref.scan_bwd(*r.values(), lens, sp, rdy, f64(dhT), absolute=True)
    # two passes through the recurrence (states and adjoints) and the sums over channels or rows
    rel = 2 * ref.scan_bounds(T, N, ch, r["A"], r["dt"], r["bias"], sp) + 2.0 ** -19
    d = m3.SelDims(b, ch, G, N, m3.io_dtype_of(io))
    gr = {k: nan_like(v) for k, v in m3.alloc_sel_grads(d, T, gate=c["z"] is not None).items()}
    ws = m3.alloc_sel_bwd_workspace(d, T).fill_(255)
    h0 = c["h"].clone()
    m3.m3_sel_bwd(d, T, c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["bias"],
                  c["h"], dy, dhT, gr, ws, seqlens=sl, flags=m3.M3_FLAG_DT_SOFTPLUS if sp else 0)
    assert torch.equal(h0, c["h"])
    if c["D"] is None:
        gr.pop("dD")
    if c["bias"] is None:
        gr.pop("ddt_bias")
    for k, v in gr.items():
        sums = U32 * (ch if k in ("dB", "dC") else b * T if v.dtype == F32 and k != "dh" else 0)
        tol = (rel + sums) * mag[k] + 1e-37
        if k in ("dx", "ddt", "dB", "dC", "dz"):
            tol = tol + half_step(io) * want[k].abs()
        near(v, want[k], tol, k)
    again = {k: nan_like(v) for k, v in gr.items()}
    again.setdefault("dD", torch.empty(ch, device="cuda"))
    again.setdefault("ddt_bias", torch.empty(ch, device="cuda"))
    m3.m3_sel_bwd(d, T, c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["bias"],
                  c["h"], dy, dhT, again, ws, seqlens=sl,
                  flags=m3.M3_FLAG_DT_SOFTPLUS if sp else 0)
    for k, v in gr.items():
        assert torch.equal(v, again[k]), k          # the same from run to run


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("ch", [48, 21])
@pytest.mark.parametrize("N", [1, 3, 4, 5, 8, 12, 16, 20, 32, 40, 64, 72, 128, 200, 256])
def test_scan_every_state_count(N, ch, io):
    """Each lane shape, with wide rows and narrow ones: prompts (in one piece and in segments),
    single tokens, backward over one tile and over several."""
    opt = "z D bias softplus"
    test_scan_fwd((1, 140, ch, 1, N, io, opt), True)
    test_scan_fwd((1, 70, ch, 1, N, io, opt), False)
    test_scan_step_continues_a_prompt((2, 5, ch, 1, N, io, opt))
    test_scan_bwd((1, 70, ch, 1, N, io, opt))
    test_scan_bwd((2, 9, ch, 1, N, io, opt))


def test_scan_step_of_very_many_sequences():
    """More sequences than a grid's second axis holds."""
    test_scan_step_continues_a_prompt((66000, 1, 4, 1, 4, F32, "z D bias softplus"))


def test_scan_without_skip_forms_no_nan():
    """Without D an infinite x is not multiplied by zero: B and C are ones, so y is infinite."""
    c, sl, sp = scan_inputs((1, 3, 8, 1, 4, F32, "softplus"), 18)
    c["C"].fill_(1.0)
    c["B"].fill_(1.0)
    c["x"][0, 1] = float("inf")
    y, _ = run_scan((1, 3, 8, 1, 4, F32, ""), c, sl, sp)
    assert torch.isfinite(y[0, 0]).all() and (y[0, 1:] == float("inf")).all()
    d = m3.SelDims(1, 8, 1, 4, m3.M3_F32)
    ys = torch.empty(1, 8, device="cuda")
    m3.m3_sel_step(d, c["x"][:, 1], c["dt"][:, 1], c["A"], c["B"][:, 1], c["C"][:, 1], None, None,
                   None, c["h"], ys, flags=m3.M3_FLAG_DT_SOFTPLUS)
    assert (ys == float("inf")).all()


def test_scan_extreme_steps():
    """Decays that underflow, steps of zero, and softplus far out on both sides."""
    b, T, ch, N = 1, 40, 32, 16
    case = (b, T, ch, 1, N, F32, "z D bias softplus")
    c, sl, sp = scan_inputs(case, 16)
    c["dt"][:, ::4] = 300.0
    c["dt"][:, 1::4] = -300.0
    c["A"][:, ::2] = -50.0
    c["A"][:, 1] = 0.0
    c["z"][:, ::3] = -100.0
    c["z"][:, 1::3] = 100.0
    c["bias"].zero_()
    r = clean(c, None, b, T)
    want_y, want_h = ref.scan(*r.values(), [T], sp)
    mag_y, mag_h = ref.scan(*r.values(), [T], sp, absolute=True)
    rel = ref.scan_bounds(T, N, ch, r["A"], r["dt"], r["bias"], sp)
    y, h = run_scan(case, c, sl, sp)
    near(h, want_h, rel * mag_h + 1e-37, "h")
    near(y, want_y, (half_step(F32) + 2.0 ** -20 + rel) * mag_y + 1e-37, "y")


def test_scan_infinity_stays_in_its_channel():
    case = (1, 40, 32, 1, 16, F32, "z D bias softplus")
    c, sl, sp = scan_inputs(case, 17)
    base, _ = run_scan(case, c, sl, sp)
    c["x"][0, 7, 5] = float("inf")
    y, _ = run_scan(case, c, sl, sp)
    assert torch.equal(base[0, :7], y[0, :7])
    keep = [i for i in range(32) if i != 5]
    assert torch.equal(base[..., keep], y[..., keep])
    assert not torch.isfinite(y[0, 7:, 5]).any()


# ---------------------------------------------------------------- norm

NORM = [  # rows, width, io, res, options
    (5, 2048, BF, F32, "w"),
    (1, 64, BF, BF, "w"),
    (3, 1, F32, F32, "w"),
    (7, 130, BF, F32, "w"),               # odd: element by element
    (9, 517, F32, F32, "w strided"),
    (33, 256, F32, BF, ""),
    (4, 1000, BF, None, "w"),
    (2, 8192, BF, BF, "w strided"),
    (3, 32768, BF, F32, "w"),
    (2, 16392, F32, F32, "w"),
    (130, 96, BF, BF, "w"),
    (2500, 512, BF, F32, "w"),
]


def norm_inputs(case, seed):
    rows, d, io, res, opt = case
    g = torch.Generator().manual_seed(seed)

    def mat(dtype, std=1.0):
        if dtype is None:
            return None
        if "strided" in opt:
            return rnd(g, rows, d + 16, std=std, dtype=dtype)[:, 8:d + 8]
        return rnd(g, rows, d, std=std, dtype=dtype)

    x, r = mat(io), mat(res, 2.0)
    w = 1 + rnd(g, d, std=0.3) if "w" in opt else None
    return x, r, w, mat


def rounds(d):
    """Roundings in a row in a 32-bit sum of d squares: 32 of a thread, the warp's, the block's."""
    return 32 + 5 + 32 + 8


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("case", NORM)
def test_norm_fwd(case, inplace):
    rows, d, io, res, opt = case
    x, r, w, _ = norm_inputs(case, 21)
    want, kept = ref.norm(f64(x), f64(r), f64(w), 1e-5, res or io)
    dims = m3.NormDims(rows, d, m3.io_dtype_of(io), m3.io_dtype_of(res or io))
    y = x if inplace else nan_like(x)
    ro = None if r is None else r if inplace else nan_like(r)
    m3.m3_norm_fwd(dims, x, r, w, 1e-5, y, None, ro)
    near(y, want, (half_step(io) + rounds(d) * U32) * want.abs() + 1e-37, "y")
    if r is not None:
        # the sum of two values that fp32 holds rounds once in 32 bits and once to its type
        f = (f64(x) + f64(r)) if inplace is False else None
        if f is not None:
            near(ro, f, half_step(res) * f.abs() * 1.01 + U32 * f.abs() + 1e-37, "residual")
        if res == F32 or not inplace:
            near(y, ref.norm(f64(ro), None, f64(w), 1e-5, F32)[0],
                 (half_step(io) + rounds(d) * U32) * want.abs() + 1e-37, "y of the kept residual")


def e4m3_steps(v):
    """Half a step of e4m3 at |v|: 2^-4 relative, 2^-10 at the smallest."""
    return torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10)


@pytest.mark.parametrize("case", NORM)
def test_norm_e4m3(case):
    rows, d, io, res, opt = case
    x, r, w, _ = norm_inputs(case, 22)
    if rows > 2:
        x[1] = 0
        if r is not None:
            r[1] = 0
    want, _ = ref.norm(f64(x), f64(r), f64(w), 1e-5, res or io)
    dims = m3.NormDims(rows, d, m3.io_dtype_of(io), m3.io_dtype_of(res or io), m3.M3_OUT_E4M3)
    q = torch.full((rows, d), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = nan_like(m3.alloc_norm_scales(dims))
    m3.m3_norm_fwd(dims, x, r, w, 1e-5, q, sc)
    n = -(-d // 128)
    pad = torch.zeros(rows, n * 128, dtype=torch.float64)
    pad[:, :d] = want.abs()
    scale = pad.view(rows, n, 128).amax(-1).clamp(min=2.0 ** -100) / 448
    near(sc, scale, (rounds(d) + 4) * U32 * scale, "scales")
    per = f64(sc).repeat_interleave(128, 1)[:, :d]
    v = f64(q.float()) * per
    near(v, want, (e4m3_steps(want / per) * (1 + 2.0 ** -10)) * per + rounds(d) * U32 * want.abs(),
         "values")
    assert float(f64(q.float()).abs().max()) <= 448
    if rows > 2:
        assert not f64(q.float())[1].any() and bool((sc[1] > 0).all())


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("case", NORM)
def test_norm_bwd(case, inplace):
    rows, d, io, res, opt = case
    g = torch.Generator().manual_seed(23)
    _, _, w, mat = norm_inputs(case, 24)
    r, dy, dres = mat(res or io, 2.0), mat(io), mat(res)
    want, want_w = ref.norm_bwd(f64(r), f64(w), 1e-5, f64(dy), f64(dres))
    mag, mag_w = ref.norm_bwd(f64(r), f64(w), 1e-5, f64(dy), f64(dres), absolute=True)
    dims = m3.NormDims(rows, d, m3.io_dtype_of(io), m3.io_dtype_of(res or io))
    dx = dy if inplace else nan_like(dy)
    dr = None if dres is None else dres if inplace else nan_like(dres)
    dw = None if w is None else nan_like(w)
    ws = m3.alloc_norm_bwd_workspace(dims).fill_(255)
    m3.m3_norm_bwd(dims, r, w, 1e-5, dy, dres, dx, dr, dw, ws)
    tol = 2 * (rounds(d) + 8) * U32 * mag + 1e-37
    near(dx, want, half_step(io) * want.abs() + tol, "dx")
    if dr is not None:
        near(dr, want, half_step(res) * want.abs() + tol, "dresidual")
    if w is not None:
        near(dw, want_w, (rows + rounds(d) + 16) * U32 * mag_w + 1e-37, "dweight")


@pytest.mark.parametrize("io,res", [(BF, BF), (BF, F32), (F32, BF), (F32, F32), (BF, None)])
@pytest.mark.parametrize("d", [8, 250, 256, 264, 512, 1000, 1024, 2048, 2056, 4096, 8192, 8200,
                               16384, 16390, 24576, 32768])
def test_norm_every_row_length(d, io, res):
    """Each number of threads a row, wide rows and narrow ones."""
    case = (5, d, io, res, "w")
    test_norm_fwd(case, False)
    test_norm_e4m3(case)
    test_norm_bwd(case, False)


def test_norm_non_finite_rows():
    """A NaN or an infinity spoils its own row and, in e4m3, its own group's scale."""
    x = torch.randn(4, 512, generator=torch.Generator().manual_seed(25)).cuda()
    x[1, 200] = float("nan")
    x[2, 300] = float("inf")
    dims = m3.NormDims(4, 512, m3.M3_F32, m3.M3_F32, m3.M3_OUT_E4M3)
    q = torch.empty(4, 512, dtype=torch.float8_e4m3fn, device="cuda")
    sc = m3.alloc_norm_scales(dims)
    m3.m3_norm_fwd(dims, x, None, None, 1e-6, q, sc)
    assert torch.isfinite(sc[0]).all() and torch.isfinite(sc[3]).all()
    assert torch.isnan(sc[1]).all()
    assert torch.isnan(sc[2, 2]) and torch.isfinite(sc[2, [0, 1, 3]]).all()
