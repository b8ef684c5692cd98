"""The block operators together, as a layer runs them: residual norm, input projection, short
convolution, projections of the step and of B and C, gated selective scan, output projection; over
ragged prompts in pieces and single tokens, and backward.  Beside that: the mixer's own scan on
the norm's output, streams, captured graphs, and rows that lie more than 2^31 elements apart."""
import pytest
import torch

import block_reference as ref
from block_reference import EX2, U32, f64, half_step
from state_space_model_06_b200 import m3
from test_block_gpu import near, rounds

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Layer:
    """One layer in 32 bits: its weights, and its calls of the library."""

    def __init__(self, b, d, D, N, W=4, seed=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).cuda()
        self.b, self.d, self.D, self.N, self.W = b, d, D, N, W
        self.wn, self.cw, self.cb = 1 + rnd(d, std=0.1), rnd(D, W, std=0.5), rnd(D, std=0.1)
        self.w_in, self.w_bc = rnd(d, 2 * D, std=d ** -0.5), rnd(D, 2 * N, std=D ** -0.5)
        self.w_dt, self.w_out = rnd(D, D, std=0.3 * D ** -0.5), rnd(D, d, std=D ** -0.5)
        self.A = -torch.exp(rnd(D, N, std=0.5))
        self.skip, self.bias = rnd(D), rnd(D, std=0.5) - 2
        self.conv = m3.ConvDims(b, D, W, m3.M3_F32)
        self.sel = m3.SelDims(b, D, 1, N, m3.M3_F32)
        self.state = torch.zeros(b, W - 1, D, device="cuda")
        self.h = torch.zeros(b, D, N, device="cuda")

    def run(self, x, res, T, lens=None):
        """Tokens x, res [b, T, d] (T None: one token, [b, d]) through the layer; every operator's
        inputs and outputs, as it saw them."""
        lead = (self.b,) if T is None else (self.b, T)
        rows = self.b * (1 if T is None else T)
        v = dict(x=x, res=res, state=self.state.clone(), h=self.h.clone(), lens=lens)
        v["y"], v["r"] = torch.empty_like(x), torch.empty_like(x)
        nd = m3.NormDims(rows, self.d, m3.M3_F32, m3.M3_F32)
        flat = lambda t: t.view(rows, self.d)
        m3.m3_norm_fwd(nd, flat(x), flat(res), self.wn, 1e-5, flat(v["y"]), None, flat(v["r"]))
        v["xz"] = v["y"] @ self.w_in
        v["u"] = torch.empty(*lead, self.D, device="cuda")
        v["o"] = torch.empty_like(v["u"])
        xc, v["z"] = v["xz"][..., :self.D], v["xz"][..., self.D:]      # views: halves of a row
        if T is None:
            m3.m3_conv_step(self.conv, xc, self.cw, self.cb, self.state, v["u"],
                            flags=m3.M3_FLAG_SILU)
        else:
            m3.m3_conv_fwd(self.conv, T, xc, self.cw, self.cb, self.state, v["u"], seqlens=lens,
                           flags=m3.M3_FLAG_SILU)
        v["bc"], v["dt"] = v["u"] @ self.w_bc, v["u"] @ self.w_dt
        B, C = (v["bc"][..., k * self.N:(k + 1) * self.N].unflatten(-1, (1, self.N))
                for k in (0, 1))
        args = (v["u"], v["dt"], self.A, B, C, self.skip, v["z"], self.bias)
        v["B"], v["C"] = B, C
        if T is None:
            m3.m3_sel_step(self.sel, *args, self.h, v["o"], flags=m3.M3_FLAG_DT_SOFTPLUS)
        else:
            m3.m3_sel_fwd(self.sel, T, *args, self.h, v["o"], m3.alloc_sel_workspace(self.sel, T),
                          seqlens=lens, flags=m3.M3_FLAG_DT_SOFTPLUS)
        v["out"] = v["o"] @ self.w_out
        return v

    def check(self, v, T):
        """Each operator against its 64-bit form on the inputs it saw."""
        one = (lambda t: f64(t)[:, None]) if T is None else f64
        n = 1 if T is None else T
        lens = ref.lengths(v["lens"], self.b, n)
        y, r = ref.norm(one(v["x"]), one(v["res"]), f64(self.wn), 1e-5, F32)
        near(one(v["y"]), y, (half_step(F32) + rounds(self.d) * U32) * y.abs() + 1e-37, "norm")
        xc, w, cb, st = one(v["xz"][..., :self.D]), f64(self.cw), f64(self.cb), f64(v["state"])
        u, new = ref.conv(xc, w, cb, st, lens, True)
        mag = ref.conv(xc.abs(), w.abs(), cb.abs(), st.abs(), lens, False)[0]
        near(one(v["u"]), u, 1.1 * (self.W + 3) * U32 * mag + 2.0 ** -20 * (u.abs() + mag) + 1e-37,
             "conv")
        args = [one(v["u"]), one(v["dt"]), f64(self.A), one(v["B"]), one(v["C"]), f64(self.skip),
                one(v["z"]), f64(self.bias), f64(v["h"])]
        o, h = ref.scan(*args, lens, True)
        mo, mh = ref.scan(*args, lens, True, absolute=True)
        rel = ref.scan_bounds(n, self.N, self.D, args[2], args[1], args[7], True)
        near(one(v["o"]), o, (half_step(F32) + rel + 2.0 ** -20) * mo + 1e-37, "scan")
        return new, h, rel * mh + 1e-37


def test_prompts_in_pieces_then_tokens():
    b, d, D, N = 3, 40, 64, 16
    layer = Layer(b, d, D, N)
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g).cuda()
    for T, lens in ((37, [37, 5, 0]), (70, [70, 1, 64]), (1, None), (2, [1, 2, 0])):
        sl = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
        v = layer.run(rnd(b, T, d), rnd(b, T, d), T, sl)
        new, h, tol = layer.check(v, T)
        assert torch.equal(f64(layer.state), new)
        near(layer.h, h, tol, "h")
    for _ in range(4):
        v = layer.run(rnd(b, d), rnd(b, d), None)
        new, h, tol = layer.check(v, None)
        assert torch.equal(f64(layer.state), new)
        near(layer.h, h, tol, "h")


def test_pieces_equal_the_whole():
    """A prompt in one call, in pieces and token by token leave the same state and outputs, up to
    twice what one of them may be off by."""
    b, d, D, N, T = 2, 24, 40, 16, 75
    g = torch.Generator().manual_seed(2)
    x, res = (torch.randn((b, T, d), generator=g).cuda() for _ in range(2))
    whole, parts = Layer(b, d, D, N), Layer(b, d, D, N)
    v = whole.run(x, res, T)
    outs = []
    for lo, hi in ((0, 33), (33, 34), (34, 70)):
        outs.append(parts.run(x[:, lo:hi].contiguous(), res[:, lo:hi].contiguous(), hi - lo)["o"])
    for t in range(70, T):
        outs.append(parts.run(x[:, t].contiguous(), res[:, t].contiguous(), None)["o"][:, None])
    # the same inputs reach the operators but for the products' own order of sums: d and D terms
    args = [f64(v[k]) for k in ("u", "dt")] + [f64(whole.A)] + [f64(v[k]) for k in ("B", "C")]
    zero = torch.zeros(b, D, N, dtype=torch.float64)
    mo, mh = ref.scan(*args, f64(whole.skip), f64(v["z"]), f64(whole.bias), zero, [T] * b, True,
                      absolute=True)
    rel = ref.scan_bounds(T, N, D, args[2], args[1], f64(whole.bias), True)
    # a product's entries move by (terms) U32 of its absolute sum, at most 8 here (inputs are unit
    # normal); five of them in a row enter y, each at most linearly with slope 8
    slack = 2 * rel + 5 * 8 * 8 * (d + D) * U32
    near(torch.cat(outs, 1), f64(v["o"]), slack * (mo + 1) + 1e-37, "y")
    near(parts.h, f64(whole.h), slack * (mh + 1) + 1e-37, "h")


def test_backward_of_a_layer():
    """The gradients flow back through the operators in turn; each is checked on what it saw."""
    b, d, D, N, T, W = 2, 24, 48, 16, 70, 4
    layer = Layer(b, d, D, N)
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g).cuda()
    layer.state.copy_(rnd(b, W - 1, D))
    layer.h.copy_(rnd(b, D, N))
    sl = torch.tensor([T, 41], dtype=torch.int32).cuda()
    lens = [T, 41]
    v = layer.run(rnd(b, T, d), rnd(b, T, d), T, sl)
    dout, dr_out = rnd(b, T, d), rnd(b, T, d)
    do = dout @ layer.w_out.t()
    gr = m3.alloc_sel_grads(layer.sel, T)
    # dz goes straight into its half of the projection's gradient
    dxz = torch.zeros(b, T, 2 * D, device="cuda")
    gr["dz"] = dxz[..., D:]
    args = (v["u"], v["dt"], layer.A, v["B"], v["C"], layer.skip, v["z"], layer.bias, v["h"])
    m3.m3_sel_bwd(layer.sel, T, *args, do, None, gr, m3.alloc_sel_bwd_workspace(layer.sel, T),
                  seqlens=sl, flags=m3.M3_FLAG_DT_SOFTPLUS)
    rargs = [f64(a) for a in args]
    want = ref.scan_bwd(*rargs, lens, True, f64(do), None)
    mag = ref.scan_bwd(*rargs, lens, True, f64(do), None, absolute=True)
    rel = 2 * ref.scan_bounds(T, N, D, rargs[2], rargs[1], rargs[7], True) + 2.0 ** -19 \
        + (D + b * T) * U32
    for k in gr:
        near(gr[k], want[k], rel * mag[k] + 1e-37, k)
    du = gr["dx"] + gr["ddt"] @ layer.w_dt.t() + \
        torch.cat([gr["dB"][:, :, 0], gr["dC"][:, :, 0]], -1) @ layer.w_bc.t()
    cg = m3.alloc_conv_grads(layer.conv, T)
    cg["dx"] = dxz[..., :D]
    m3.m3_conv_bwd(layer.conv, T, v["xz"][..., :D], layer.cw, layer.cb, v["state"], du, cg,
                   m3.alloc_conv_bwd_workspace(layer.conv, T), seqlens=sl, flags=m3.M3_FLAG_SILU)
    cargs = [f64(t) for t in (v["xz"][..., :D], layer.cw, layer.cb, v["state"])]
    want = ref.conv_bwd(*cargs, lens, True, f64(du))
    mag = ref.conv_bwd(*cargs, lens, True, f64(du), absolute=True)
    pre = float((cargs[1].abs().sum(1).max() * cargs[0].abs().max()) + cargs[2].abs().max())
    rel = (W + 6 + 128 + b * T) * U32 + 2.0 ** -19 + 4 * (W + 3) * U32 * pre
    for k in cg:
        near(cg[k], want[k], rel * mag[k] + 1e-37, k)
    assert not f64(dxz)[1, 41:].any()            # both halves: zeros past the length
    dy = (dxz @ layer.w_in.t()).view(b * T, d)
    nd = m3.NormDims(b * T, d, m3.M3_F32, m3.M3_F32)
    dx, dw = torch.empty_like(dy), torch.empty(d, device="cuda")
    dres = torch.empty_like(dy)
    r = v["r"].view(b * T, d)
    m3.m3_norm_bwd(nd, r, layer.wn, 1e-5, dy, dr_out.view(b * T, d), dx, dres, dw,
                   m3.alloc_norm_bwd_workspace(nd))
    nargs = (f64(r), f64(layer.wn), 1e-5, f64(dy), f64(dr_out).view(b * T, d))
    (w_dx, w_dw), (m_dx, m_dw) = ref.norm_bwd(*nargs), ref.norm_bwd(*nargs, absolute=True)
    near(dx, w_dx, 2 * (rounds(d) + 8) * U32 * m_dx + 1e-37, "dx")
    assert torch.equal(dx, dres)
    near(dw, w_dw, (b * T + rounds(d) + 16) * U32 * m_dw + 1e-37, "dweight")


def test_norm_feeds_the_mixer():
    """The residual norm before the mixer's scan: the scan's x is the norm's output as it lies."""
    b, T, H, P, N = 1, 96, 4, 64, 64
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g)
    x, res = rnd(b * T, H * P).to(BF).cuda(), rnd(b * T, H * P).cuda()
    y = torch.empty(b * T, H * P, dtype=BF, device="cuda")
    m3.m3_norm_fwd(m3.NormDims(b * T, H * P, m3.M3_BF16, m3.M3_F32), x, res, None, 1e-6, y, None,
                   res)
    d = m3.Dims(b, H, 1, P, N, 1, m3.M3_BF16)
    import oracle
    from gpu_helpers import rel_slices
    B, C = (rnd(b, T, 1, 1, N).mul(N ** -0.5).to(BF).cuda() for _ in range(2))
    dt, A = torch.rand((b, T, H), generator=g).mul(0.2).cuda(), -torch.ones(b, T, H).cuda()
    lam, th = torch.full((b, T, H), 0.6).cuda(), torch.zeros(b, T, 1, N // 2).cuda()
    st, out = m3.State(d), torch.empty(b, T, H, 1, P, dtype=BF, device="cuda")
    xs = y.view(b, T, H, 1, P)
    m3.m3_scan_fwd(d, T, 64, xs, B, C, dt, A, lam, th, None, st, out, m3.alloc_workspace(d, T, 64))
    yo = oracle.scan(*(f64(t).numpy() for t in (xs, B, C, dt, A, lam, th)))[0]
    assert rel_slices(f64(out).numpy(), yo, (1, 3, 4)) <= 2e-2


def everything(seed, T=130):
    """Forward and backward calls of every operator on buffers of their own: inputs, a function
    that makes the calls, and the outputs."""
    b, D, N, W = 2, 64, 16, 4
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).cuda()
    cd, sd = m3.ConvDims(b, D, W, m3.M3_F32), m3.SelDims(b, D, 1, N, m3.M3_F32)
    nd = m3.NormDims(b * T, D, m3.M3_F32, m3.M3_F32)
    i = dict(x=rnd(b, T, D), res=rnd(b, T, D), z=rnd(b, T, D), dt=rnd(b, T, D), B=rnd(b, T, 1, N),
             C=rnd(b, T, 1, N), dy=rnd(b, T, D))
    w, cw, A = rnd(D), rnd(D, W), -torch.exp(rnd(D, N))
    st0, h0 = rnd(b, W - 1, D), rnd(b, D, N)
    o = {k: torch.empty(b, T, D, device="cuda") for k in ("n", "r", "u", "y", "dx", "dr")}
    o["dw"] = torch.empty(D, device="cuda")
    o["st"], o["h"] = torch.empty_like(st0), torch.empty_like(h0)
    cg, sg = m3.alloc_conv_grads(cd, T), m3.alloc_sel_grads(sd, T)
    w1, w2 = m3.alloc_sel_workspace(sd, T), m3.alloc_sel_bwd_workspace(sd, T)
    w3, w4 = m3.alloc_conv_bwd_workspace(cd, T), m3.alloc_norm_bwd_workspace(nd)
    m = lambda t: t.view(b * T, D)

    def calls(stream=None):
        kw = dict(stream=stream)
        o["st"].copy_(st0)
        o["h"].copy_(h0)
        m3.m3_norm_fwd(nd, m(i["x"]), m(i["res"]), w, 1e-5, m(o["n"]), None, m(o["r"]), **kw)
        m3.m3_conv_fwd(cd, T, o["n"], cw, None, o["st"], o["u"], flags=m3.M3_FLAG_SILU, **kw)
        a = (o["u"], i["dt"], A, i["B"], i["C"], None, i["z"], None)
        m3.m3_sel_fwd(sd, T, *a, o["h"], o["y"], w1, flags=m3.M3_FLAG_DT_SOFTPLUS, **kw)
        m3.m3_sel_bwd(sd, T, *a, h0, i["dy"], None, sg, w2, flags=m3.M3_FLAG_DT_SOFTPLUS, **kw)
        m3.m3_conv_bwd(cd, T, o["n"], cw, None, st0, sg["dx"], cg, w3, flags=m3.M3_FLAG_SILU, **kw)
        m3.m3_norm_bwd(nd, m(o["r"]), w, 1e-5, m(cg["dx"]), None, m(o["dx"]), m(o["dr"]), o["dw"],
                       w4, **kw)

    outs = dict(o, **{"c_" + k: v for k, v in cg.items() if k != "dbias"},
                **{"s_" + k: v for k, v in sg.items() if k not in ("dD", "ddt_bias")})
    return i, calls, outs


def test_captured_graphs_replay_on_new_inputs():
    i, calls, outs = everything(5)
    calls()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    fresh, _, _ = everything(6)
    for k in i:
        i[k].copy_(fresh[k])
    for v in outs.values():
        v.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in outs.items()}
    calls()
    for k, v in outs.items():
        assert torch.equal(v, got[k]), k


def test_two_streams_at_once():
    """Two callers with workspaces of their own, on two streams, many times: each gets what it
    gets alone.  One passes its stream by argument."""
    _, first, out1 = everything(7, T=1100)
    _, second, out2 = everything(8, T=1100)
    first()
    second()
    torch.cuda.synchronize()
    alone = [{k: v.clone() for k, v in o.items()} for o in (out1, out2)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s1):
            first()
        with torch.cuda.stream(s2):
            second(stream=s2)
    torch.cuda.synchronize()
    for o, want in zip((out1, out2), alone):
        for k, v in o.items():
            assert torch.equal(v, want[k]), k


def test_rows_further_apart_than_32_bits():
    """Rows more than 2^31 elements apart, in and out."""
    far = 2 ** 31 + 64
    g = torch.Generator().manual_seed(9)
    buf = torch.zeros(far + 4096, dtype=BF, device="cuda")
    T, C = 6, 64
    view = buf.as_strided((2, T, C), (far, C, 1))
    x = torch.randn((2, T, C), generator=g).to(BF).cuda()
    view.copy_(x)
    w = torch.randn((C, 4), generator=g).cuda()
    d = m3.ConvDims(2, C, 4)
    run = lambda xs, ys: m3.m3_conv_fwd(d, T, xs, w, None,
                                        torch.zeros(2, 3, C, dtype=BF, device="cuda"), ys)
    near_y, far_y = torch.empty_like(x), buf[2048:].as_strided((2, T, C), (far, C, 1))
    run(x, near_y)
    run(view, far_y)
    assert torch.equal(near_y, far_y)
    sd = m3.SelDims(2, C, 1, 16)
    B, C2 = (torch.randn((2, T, 1, 16), generator=g).to(BF).cuda() for _ in range(2))
    A = -torch.ones(C, 16, device="cuda")
    run = lambda xs, ys: m3.m3_sel_fwd(sd, T, xs, xs, A, B, C2, None, xs, None,
                                       torch.zeros(2, C, 16, device="cuda"), ys, None,
                                       flags=m3.M3_FLAG_DT_SOFTPLUS)
    run(x, near_y)
    run(view, far_y)
    assert torch.equal(near_y, far_y)
    nd = m3.NormDims(2, T * C, m3.M3_BF16, m3.M3_BF16)
    flat = lambda t: t.as_strided((2, T * C), (t.stride(0), 1))
    m3.m3_norm_fwd(nd, x.view(2, -1), None, None, 1e-6, near_y.view(2, -1))
    m3.m3_norm_fwd(nd, flat(view), None, None, 1e-6, flat(far_y))
    assert torch.equal(near_y, far_y)


def test_empty_calls():
    """No tokens: states stay, parameter gradients are zero, dh is dhT."""
    b, D, N = 2, 16, 16
    cd, sd = m3.ConvDims(b, D, 4, m3.M3_F32), m3.SelDims(b, D, 1, N, m3.M3_F32)
    e = torch.empty(b, 0, D, device="cuda")
    bc = torch.empty(b, 0, 1, N, device="cuda")
    st, h = torch.randn(b, 3, D, device="cuda"), torch.randn(b, D, N, device="cuda")
    st0, h0 = st.clone(), h.clone()
    w, A, v = torch.randn(D, 4, device="cuda"), -torch.ones(D, N, device="cuda"), torch.ones(D, device="cuda")
    m3.m3_conv_fwd(cd, 0, e, w, v, st, e)
    m3.m3_sel_fwd(sd, 0, e, e, A, bc, bc, v, e, v, h, e, None)
    assert torch.equal(st, st0) and torch.equal(h, h0)
    cg, sg = m3.alloc_conv_grads(cd, 0), m3.alloc_sel_grads(sd, 0)
    for t in (*cg.values(), *sg.values()):
        t.fill_(float("nan"))
    m3.m3_conv_bwd(cd, 0, e, w, v, st, e, cg, m3.alloc_conv_bwd_workspace(cd, 0))
    m3.m3_sel_bwd(sd, 0, e, e, A, bc, bc, v, e, v, h, e, h0, sg, m3.alloc_sel_bwd_workspace(sd, 0))
    for k in ("dweight", "dbias", "dstate"):
        assert not cg[k].any(), k
    for k in ("dA", "dD", "ddt_bias"):
        assert not sg[k].any(), k
    assert torch.equal(sg["dh"], h0)
