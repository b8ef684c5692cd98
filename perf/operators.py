"""Cases of the block operators around the mixer: the short causal convolution, the selective
scan and the RMS norm with the residual's addition, over prompts, single tokens and backward.

A case is a dict of plain values.  ``op`` is "conv", "scan" or "norm"; ``dir`` is "prompt" (a
whole sequence, carrying the state), "step" (one token a sequence) or "train" (the backward
call).  ``run`` computes a case in its plain form, elementary torch operations in 32 bits, or
with ``own`` through the library's entry points.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100          # scales of all-zero groups stay finite and positive
SCALE_GROUP = 128


def listed():
    base = dict(gate=True, ragged=False, sliced=False, G=1)
    conv = dict(op="conv", W=4, ragged=False, sliced=False)
    norm = dict(op="norm", res="f32", out="io")
    return [
        # the 1.5B-scale layer's prompt (8 x 4096 tokens, 4096 channels): x is one half of the
        # input projection's output, so its rows are twice as long as the convolution reads
        dict(conv, name="conv_prompt_1p5b", dir="prompt", b=8, T=4096, D=4096, io="bf16",
             sliced=True),
        # one training micro-batch of the same layer
        dict(conv, name="conv_train", dir="train", b=4, T=2048, D=4096, io="bf16"),
        # serving, one token of one sequence: the smallest call, where latency counts
        dict(conv, name="conv_step_b1", dir="step", b=1, T=1, D=4096, io="bf16"),
        # prompts of a padded batch at the 1.5B scale: the largest forward scan
        dict(base, name="scan_prompt_1p5b", op="scan", dir="prompt", b=8, T=2048, D=4096, N=16,
             io="bf16", sliced=True),
        # one long prompt: few channels' worth of parallel work, a long axis
        dict(base, name="scan_long_b1", op="scan", dir="prompt", b=1, T=16384, D=2048, N=16,
             io="bf16"),
        # odd and ragged: 32-bit values, lengths of their own, sizes that divide nothing
        dict(base, name="scan_ragged_f32", op="scan", dir="prompt", b=3, T=509, D=1001, N=24,
             io="f32", ragged=True),
        # one training micro-batch: every gradient
        dict(base, name="scan_train", op="scan", dir="train", b=4, T=2048, D=4096, N=16,
             io="bf16"),
        # training in 32 bits, small and odd, two groups of channels sharing B and C
        dict(base, name="scan_train_odd_f32", op="scan", dir="train", b=2, T=777, D=522, N=16,
             G=2, io="f32"),
        # serving at batch 256: one token a sequence over the 32-bit state
        dict(base, name="scan_step_b256", op="scan", dir="step", b=256, T=1, D=4096, N=16,
             io="bf16"),
        # prompts through the norm into an 8-bit projection
        dict(norm, name="norm_prompt_e4m3", dir="prompt", rows=32768, d=2048, io="bf16",
             out="e4m3"),
        # one token of 8 sequences, residual in the io type
        dict(norm, name="norm_step_b8", dir="step", rows=8, d=2048, io="bf16", res="bf16"),
        # training
        dict(norm, name="norm_train", dir="train", rows=16384, d=2048, io="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("conv", "scan", "scan", "norm"))
    way = rng.choice(("prompt", "step", "train"))
    io = rng.choice(("bf16", "bf16", "f32"))
    if op == "norm":
        rows = _log_int(rng, 1, 256) if way == "step" else _log_int(rng, 16, 32768)
        d = _log_int(rng, 64, 8192)
        while rows * d > 2048 * 16384:
            rows = max(1, rows // 2)
        if rng.random() < 0.5:
            d = max(64, d // 64 * 64)
        out = "e4m3" if way != "train" and rng.random() < 0.5 else "io"
        return dict(op="norm", dir=way, rows=rows, d=d, io=io, out=out,
                    res=rng.choice(("f32", "bf16", "none")))
    D = _log_int(rng, 48, 4096)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)
    if way == "step":
        b, T = _log_int(rng, 1, 256), 1
    else:
        b, T = rng.randint(1, 8), _log_int(rng, 1, 8192)
    ragged, sliced = way != "step" and rng.random() < 0.3, rng.random() < 0.4
    if op == "conv":
        while b * T * D > 8 * 2048 * 2048:
            T //= 2
        return dict(op="conv", dir=way, b=b, T=T, D=D, W=rng.randint(2, 4), io=io,
                    ragged=ragged, sliced=sliced)
    G = rng.choice((1, 1, 2))
    D = D // G * G
    N = rng.choice((1, 7, 8, 16, 16, 16, 24, 32, 64))
    most = 2 ** 28 if way == "train" else 2 ** 29
    while b * T * D * N > most:
        if T > 1:
            T //= 2
        else:
            b //= 2
    return dict(op="scan", dir=way, b=b, T=T, D=D, N=N, G=G, io=io, gate=rng.random() < 0.7,
                ragged=ragged, sliced=sliced)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    c = case
    io = _TYPES[c["io"]]

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    s = {"case": dict(case)}
    if c["op"] == "norm":
        rows, d = c["rows"], c["d"]
        res = None if c["res"] == "none" else _TYPES[c["res"]]
        s["weight"] = 1.0 + randn(d, std=0.2)
        s["eps"] = 1e-6
        if c["dir"] == "train":
            s["r"] = randn(rows, d, std=2.0, dtype=res or io)
            s["dy"] = randn(rows, d, dtype=io)
            s["dres"] = randn(rows, d, dtype=res) if res else None
        else:
            s["x"] = randn(rows, d, dtype=io)
            s["residual"] = randn(rows, d, std=2.0, dtype=res) if res else None
        return s

    b, T, D = c["b"], c["T"], c["D"]
    lead = (b,) if c["dir"] == "step" else (b, T)
    if c["ragged"]:
        s["seqlens"] = torch.randint(0, T + 1, (b,), generator=g, device=dev, dtype=torch.int32)
    else:
        s["seqlens"] = None
    if c["op"] == "conv":
        W = c["W"]
        # sliced: x is one half of a wider projection's rows
        x = randn(*lead, 2 * D if c["sliced"] else D, dtype=io)
        s["x"] = x[..., :D]
        s["weight"] = randn(D, W, std=1 / math.sqrt(W))
        s["bias"] = randn(D, std=0.1)
        s["state"] = randn(b, W - 1, D, dtype=io)
        if c["dir"] == "train":
            s["dy"] = randn(b, T, D, dtype=io)
        return s

    N, G = c["N"], c["G"]
    if c["sliced"]:
        # x and z are the halves of one projection, B and C lie behind each other in another
        xz = randn(*lead, 2 * D, dtype=io)
        bc = randn(*lead, 2 * G * N, dtype=io)
        s["x"], z = xz[..., :D], xz[..., D:]
        s["B"] = bc[..., :G * N].unflatten(-1, (G, N))
        s["C"] = bc[..., G * N:].unflatten(-1, (G, N))
    else:
        s["x"], z = randn(*lead, D, dtype=io), randn(*lead, D, dtype=io)
        s["B"], s["C"] = randn(*lead, G, N, dtype=io), randn(*lead, G, N, dtype=io)
    s["z"] = z if c["gate"] else None
    s["dt"] = randn(*lead, D, std=0.5, dtype=io)
    # steps of 0.001 to 0.1 after the softplus, decay rates of 1 to N with a spread
    step = torch.exp(torch.rand(D, generator=g, device=dev) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    rate = torch.arange(1, N + 1, device=dev, dtype=torch.float32)
    s["A"] = -rate * torch.exp(randn(D, N, std=0.1))
    s["D"] = 1.0 + randn(D, std=0.1)
    s["h"] = randn(b, D, N)
    if c["dir"] == "train":
        s["dy"] = randn(b, T, D, dtype=io)
        s["dhT"] = randn(b, D, N)
    return s


# ---------------------------------------------------------------- the library's calls

def _own_conv(m3, s):
    c = s["case"]
    if "plan" not in s:             # buffers that a program keeps from call to call
        dims = m3.ConvDims(c["b"], c["D"], c["W"], m3.io_dtype_of(s["x"].dtype))
        if c["dir"] == "train":
            s["plan"] = (dims, m3.alloc_conv_grads(dims, c["T"]),
                         m3.alloc_conv_bwd_workspace(dims, c["T"]))
        else:
            s["plan"] = (dims, torch.empty(s["x"].shape, dtype=s["x"].dtype, device="cuda"), None)
    dims, out, ws = s["plan"]
    if c["dir"] == "train":
        m3.m3_conv_bwd(dims, c["T"], s["x"], s["weight"], s["bias"], s["state"], s["dy"], out, ws,
                       seqlens=s["seqlens"], flags=m3.M3_FLAG_SILU)
        return {k: out[k] for k in ("dx", "dweight", "dbias", "dstate")}
    if c["dir"] == "step":
        m3.m3_conv_step(dims, s["x"], s["weight"], s["bias"], s["state"], out,
                        flags=m3.M3_FLAG_SILU)
    else:
        m3.m3_conv_fwd(dims, c["T"], s["x"], s["weight"], s["bias"], s["state"], out,
                       seqlens=s["seqlens"], flags=m3.M3_FLAG_SILU)
    return {"y": out, "state": s["state"]}


def _own_scan(m3, s):
    c = s["case"]
    if "plan" not in s:
        dims = m3.SelDims(c["b"], c["D"], c["G"], c["N"], m3.io_dtype_of(s["x"].dtype))
        if c["dir"] == "train":
            s["plan"] = (dims, m3.alloc_sel_grads(dims, c["T"], gate=c["gate"]),
                         m3.alloc_sel_bwd_workspace(dims, c["T"]))
        else:
            ws = m3.alloc_sel_workspace(dims, c["T"]) if c["dir"] == "prompt" else None
            s["plan"] = (dims, torch.empty(s["x"].shape, dtype=s["x"].dtype, device="cuda"), ws)
    dims, out, ws = s["plan"]
    args = [s[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h")]
    if c["dir"] == "train":
        m3.m3_sel_bwd(dims, c["T"], *args, s["dy"], s["dhT"], out, ws, seqlens=s["seqlens"],
                      flags=m3.M3_FLAG_DT_SOFTPLUS)
        return {k: v for k, v in out.items() if v is not None}
    if c["dir"] == "step":
        m3.m3_sel_step(dims, *args, out, flags=m3.M3_FLAG_DT_SOFTPLUS)
    else:
        m3.m3_sel_fwd(dims, c["T"], *args, out, ws, seqlens=s["seqlens"],
                      flags=m3.M3_FLAG_DT_SOFTPLUS)
    return {"y": out, "h": s["h"]}


def _own_norm(m3, s):
    c = s["case"]
    if c["dir"] == "train":
        r, dres = s["r"], s["dres"]
        if "plan" not in s:
            dims = m3.NormDims(c["rows"], c["d"], m3.io_dtype_of(s["dy"].dtype),
                               m3.io_dtype_of(r.dtype))
            s["plan"] = (dims, torch.empty_like(s["dy"]),
                         torch.empty_like(r) if dres is not None else None,
                         torch.empty_like(s["weight"]), m3.alloc_norm_bwd_workspace(dims))
        dims, dx, dr, dw, ws = s["plan"]
        m3.m3_norm_bwd(dims, r, s["weight"], s["eps"], s["dy"], dres, dx, dr, dw, ws)
        out = {"dx": dx, "dweight": dw}
        return out if dr is None else dict(out, dresidual=dr)
    x, res = s["x"], s["residual"]
    if "plan" not in s:
        dims = m3.NormDims(c["rows"], c["d"], m3.io_dtype_of(x.dtype),
                           m3.io_dtype_of(x.dtype if res is None else res.dtype),
                           m3.M3_OUT_E4M3 if c["out"] == "e4m3" else m3.M3_OUT_IO)
        y = torch.empty(x.shape, device="cuda",
                        dtype=torch.float8_e4m3fn if c["out"] == "e4m3" else x.dtype)
        scales = m3.alloc_norm_scales(dims) if c["out"] == "e4m3" else None
        s["plan"] = (dims, y, scales, None if res is None else torch.empty_like(res))
    dims, y, scales, r = s["plan"]
    m3.m3_norm_fwd(dims, x, res, s["weight"], s["eps"], y, scales, r)
    out = {"y": y} if scales is None else {"y": y, "scales": scales}
    return out if r is None else dict(out, residual=r)


# ---------------------------------------------------------------- plain forms

def _valid(seqlens, b, T, device):
    """[b, T, 1] truth values: the tokens inside each sequence's length."""
    t = torch.arange(T, device=device)
    if seqlens is None:
        return torch.ones(b, T, 1, dtype=torch.bool, device=device)
    return (t[None, :] < seqlens[:, None])[..., None]


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _conv_inputs(s):
    """The carried tokens before the sequence's, in 32 bits: [b, W-1+T, D]."""
    x = s["x"] if s["x"].dim() == 3 else s["x"][:, None]
    return torch.cat([s["state"], x], 1).float()


def _conv_sum(s, xp, T):
    w = s["weight"]
    return sum(xp[:, k:k + T] * w[:, k] for k in range(w.shape[1])) + s["bias"]


def _plain_conv(s):
    c, T, W = s["case"], s["case"]["T"], s["case"]["W"]
    xp = _conv_inputs(s)
    valid = _valid(s["seqlens"], c["b"], T, xp.device)
    pre = _conv_sum(s, xp, T)
    sig = _sigmoid(pre)
    if c["dir"] == "train":
        g = torch.where(valid, s["dy"].float() * sig * (1 + pre * (1 - sig)), 0.0)
        dxp = torch.zeros_like(xp)
        for k in range(W):
            dxp[:, k:k + T] += g * s["weight"][:, k]
        dw = torch.stack([(g * xp[:, k:k + T]).sum((0, 1), dtype=torch.float64)
                          for k in range(W)], 1)
        return {"dx": dxp[:, W - 1:].to(s["x"].dtype), "dweight": dw.float(),
                "dbias": g.sum((0, 1), dtype=torch.float64).float(), "dstate": dxp[:, :W - 1]}
    y = torch.where(valid, pre * sig, 0.0).to(s["x"].dtype)
    ends = valid.sum(1)                                   # [b, 1]: tokens of each sequence
    at = ends + torch.arange(W - 1, device=xp.device)     # [b, W-1] places of the carried tokens
    carried = torch.gather(xp, 1, at[..., None].expand(-1, -1, c["D"]))
    s["state"].copy_(carried)
    return {"y": y.view(s["x"].shape), "state": s["state"]}


def _running(decay, value):
    """v_t + d_t v_{t-1} + d_t d_{t-1} v_{t-2} + ... over axis 1, by doubling the reach (both
    arguments are overwritten)."""
    reach = 1
    while reach < value.shape[1]:
        value[:, reach:] += decay[:, reach:] * value[:, :-reach]
        decay[:, reach:] = decay[:, reach:] * decay[:, :-reach]
        reach *= 2
    return value


def _scan_terms(s):
    c = s["case"]
    wide = (lambda v: v[:, None].float()) if c["dir"] == "step" else (lambda v: v.float())
    x, v = wide(s["x"]), wide(s["dt"]) + s["dt_bias"]
    per = c["D"] // c["G"]
    # each channel reads its group's B and C
    B, C = (wide(s[k]).repeat_interleave(per, 2) for k in ("B", "C"))
    valid = _valid(s["seqlens"], c["b"], c["T"], x.device)
    delta = torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))
    delta = torch.where(valid, delta, 0.0)
    decay = torch.exp(delta[..., None] * s["A"])
    return x, v, B, C, valid, delta, decay, wide


def _states(s, x, B, delta, decay):
    value = (delta * x)[..., None] * B
    value[:, 0] += decay[:, 0] * s["h"]
    return _running(decay.clone(), value)


def _plain_scan(s):
    c = s["case"]
    io = s["x"].dtype
    x, v, B, C, valid, delta, decay, wide = _scan_terms(s)
    h = _states(s, x, B, delta, decay)
    if c["dir"] != "train":
        y = (h * C).sum(-1) + s["D"] * x
        if c["gate"]:
            z = wide(s["z"])
            y = y * z * _sigmoid(z)
        y = torch.where(valid, y, 0.0).to(io)
        s["h"].copy_(h[:, -1])
        return {"y": y.view(s["x"].shape), "h": s["h"]}
    dy = torch.where(valid, wide(s["dy"]), 0.0)
    grads = {}
    if c["gate"]:
        z = wide(s["z"])
        sig = _sigmoid(z)
        pre = (h * C).sum(-1) + s["D"] * x
        grads["dz"] = torch.where(valid, dy * pre * sig * (1 + z * (1 - sig)), 0.0).to(io)
        dy = dy * z * sig
    per = (c["b"], c["T"], c["G"], c["D"] // c["G"], c["N"])
    grads["dC"] = (h * dy[..., None]).view(per).sum(3).to(io)
    before = torch.cat([s["h"][:, None], h[:, :-1]], 1)      # the state each token starts from
    del h
    # the adjoint of each token's state, from the last token back
    adj = C * dy[..., None]
    adj[:, -1] += s["dhT"]
    later = torch.cat([decay[:, 1:], torch.ones_like(decay[:, :1])], 1)
    adj = _running(later.flip(1), adj.flip(1)).flip(1)
    del later
    grads["dB"] = (adj * (delta * x)[..., None]).view(per).sum(3).to(io)
    through_b = (adj * B).sum(-1)
    grads["dh"] = decay[:, 0] * adj[:, 0]
    rate = adj * decay * before                               # d loss / d (delta A)
    del adj, decay, before
    ddelta = x * through_b + (rate * s["A"]).sum(-1)
    ddt = torch.where(valid, ddelta * _sigmoid(v), 0.0)
    grads["dx"] = torch.where(valid, delta * through_b + s["D"] * dy, 0.0).to(io)
    grads["ddt"] = ddt.to(io)
    grads["ddt_bias"] = ddt.sum((0, 1), dtype=torch.float64).float()
    grads["dA"] = (rate * delta[..., None]).sum((0, 1), dtype=torch.float64).float()
    grads["dD"] = (dy * x).sum((0, 1), dtype=torch.float64).float()
    return grads


def _plain_norm(s):
    c = s["case"]
    if c["dir"] == "train":
        r, dy, w = s["r"].float(), s["dy"].float(), s["weight"]
        rstd = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + s["eps"])
        unit = r * rstd
        dyw = dy * w
        dr = rstd * (dyw - unit * (dyw * unit).mean(-1, keepdim=True))
        if s["dres"] is not None:
            dr = dr + s["dres"].float()
        out = {"dx": dr.to(s["dy"].dtype),
               "dweight": (dy * unit).sum(0, dtype=torch.float64).float()}
        return out if s["dres"] is None else dict(out, dresidual=dr.to(s["dres"].dtype))
    x, out = s["x"], {}
    r = x.float()
    if s["residual"] is not None:
        out["residual"] = (r + s["residual"].float()).to(s["residual"].dtype)
        r = out["residual"].float()           # the norm is of the residual as it is kept
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    if c["out"] == "io":
        return dict(out, y=y.to(x.dtype))
    groups = -(-c["d"] // SCALE_GROUP)
    padded = torch.zeros(c["rows"], groups * SCALE_GROUP, device=x.device)
    padded[:, :c["d"]] = y.abs()
    amax = padded.view(c["rows"], groups, SCALE_GROUP).amax(-1)
    scales = torch.clamp(amax, min=AMAX_FLOOR) / E4M3_MAX
    q = y / scales.repeat_interleave(SCALE_GROUP, 1)[:, :c["d"]]
    return dict(out, y=q.to(torch.float8_e4m3fn), scales=scales)


def run(state):
    op = state["case"]["op"]
    if own:
        from state_space_model_06_b200 import m3
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[op](m3, state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[op](state)


def work(case):
    c = case
    e = 2 if c["io"] == "bf16" else 4
    if c["op"] == "norm":
        rows, d = c["rows"], c["d"]
        r = {"f32": 4, "bf16": 2, "none": 0}[c["res"]]
        if c["dir"] == "train":
            kept = r or e
            return {"bytes": rows * d * (kept + e + r + e + r) + 8 * d, "flops": 12 * rows * d}
        y = 1 + 4 / SCALE_GROUP if c["out"] == "e4m3" else e
        return {"bytes": rows * d * (e + 2 * r + y) + 4 * d, "flops": 6 * rows * d}
    b, T, D = c["b"], c["T"], c["D"]
    if c["op"] == "conv":
        W = c["W"]
        kept = b * (W - 1) * D
        if c["dir"] == "train":
            return {"bytes": 3 * b * T * D * e + kept * (e + 4) + 8 * D * (W + 1),
                    "flops": b * T * D * (6 * W + 10)}
        return {"bytes": 2 * b * T * D * e + 2 * kept * e + 4 * D * (W + 1),
                "flops": b * T * D * (2 * W + 5)}
    N, G = c["N"], c["G"]
    cells = b * T * D
    weights = 4 * (D * N + 2 * D)
    gate = 1 if c["gate"] else 0
    if c["dir"] == "train":
        # x, dt, dy, (z) and their gradients; B, C twice; h, dhT and dh
        return {"bytes": cells * e * (5 + 2 * gate) + 4 * b * T * G * N * e + 12 * b * D * N
                + 2 * weights, "flops": 24 * cells * N}
    return {"bytes": cells * e * (3 + gate) + 2 * b * T * G * N * e + 8 * b * D * N + weights,
            "flops": 7 * cells * N}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _f64(v):
    return None if v is None else v.double()


def _inside(s, b, t):
    if s["seqlens"] is None:
        return torch.ones(b, 1, dtype=torch.float64, device="cuda")
    return (t < s["seqlens"]).double()[:, None]


def _exact_conv(s):
    c = s["case"]
    b, T, D, W = c["b"], c["T"], c["D"], c["W"]
    if b * T * D > 1 << 28:
        return None
    x = _f64(s["x"]).reshape(b, T, D)
    old, w, bias = _f64(s["state"]), _f64(s["weight"]), _f64(s["bias"])
    lens = s["seqlens"] if s["seqlens"] is not None else torch.full((b,), T, device="cuda")
    lens = lens.tolist()
    grads = c["dir"] == "train"
    y, state = torch.zeros_like(x), old.clone()
    dx, dstate = torch.zeros_like(x), torch.zeros_like(old)
    dw, dbias = torch.zeros_like(w), torch.zeros_like(bias)
    for i in range(b):                    # one sequence after the other, at its own length
        n = lens[i]
        seq = torch.cat([old[i], x[i, :n]])
        state[i] = seq[n:]
        if not n:
            continue
        pre = bias + (seq.unfold(0, W, 1) * w).sum(-1)           # [n, D, W] windows
        gate = torch.sigmoid(pre)
        if not grads:
            y[i, :n] = pre * gate
            continue
        g = _f64(s["dy"][i, :n]) * (gate + pre * gate * (1 - gate))
        dseq = torch.zeros_like(seq)
        for k in range(W):
            dseq[k:k + n] += g * w[:, k]
            dw[:, k] += (g * seq[k:k + n]).sum(0)
        dbias += g.sum(0)
        dstate[i], dx[i, :n] = dseq[:W - 1], dseq[W - 1:]
    if grads:
        return {"dx": dx, "dweight": dw, "dbias": dbias, "dstate": dstate}
    return {"y": y.reshape(s["x"].shape), "state": state}


def _exact_scan(s):
    c = s["case"]
    b, T, D, N, G = (c[k] for k in ("b", "T", "D", "N", "G"))
    train = c["dir"] == "train"
    x, dt, z = (None if s[k] is None else _f64(s[k]).reshape(b, T, D) for k in ("x", "dt", "z"))
    B, C = (_f64(s[k]).reshape(b, T, G, 1, N) for k in ("B", "C"))
    A, skip = _f64(s["A"]).view(G, D // G, N), _f64(s["D"])
    v = dt + _f64(s["dt_bias"])
    delta = torch.logaddexp(v, torch.zeros_like(v))
    h = _f64(s["h"]).view(b, G, D // G, N)
    out = torch.zeros_like(x)
    kept = [h]
    grp = lambda q: q.view(b, G, D // G, 1)  # noqa: E731
    for t in range(T):
        on = _inside(s, b, t)
        step = grp(delta[:, t] * on)
        h = torch.exp(step * A) * h + step * grp(x[:, t]) * B[:, t]
        out[:, t] = ((h * C[:, t]).sum(-1).view(b, D) + skip * x[:, t]) * on
        if train:
            kept.append(h)
    if not train:
        y = out if z is None else out * z * torch.sigmoid(z)
        return {"y": y.view(s["x"].shape), "h": h.reshape(b, D, N)}
    dy = _f64(s["dy"])
    got = {k: torch.zeros_like(x) for k in ("dx", "ddt")}
    got["dB"], got["dC"] = torch.zeros_like(B), torch.zeros_like(C)
    if z is not None:
        got["dz"] = torch.zeros_like(x)
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(skip), torch.zeros_like(skip)
    lam = _f64(s["dhT"]).view(b, G, D // G, N)
    for t in range(T - 1, -1, -1):
        on = _inside(s, b, t)
        e = dy[:, t] * on
        if z is not None:
            sg = torch.sigmoid(z[:, t])
            got["dz"][:, t] = e * out[:, t] * sg * (1 + z[:, t] * (1 - sg))
            e = e * z[:, t] * sg
        step = grp(delta[:, t] * on)
        a = torch.exp(step * A)
        lam = lam + C[:, t] * grp(e)
        got["dC"][:, t] = (kept[t + 1] * grp(e)).sum(2, keepdim=True)
        got["dB"][:, t] = (lam * step * grp(x[:, t])).sum(2, keepdim=True)
        lb = (lam * B[:, t]).sum(-1).view(b, D)
        q = lam * a * kept[t]
        got["dx"][:, t] = step.reshape(b, D) * lb + skip * e
        dd = (x[:, t] * lb + (q * A).sum(-1).view(b, D)) * on
        got["ddt"][:, t] = dd * torch.sigmoid(v[:, t])
        dA += (q * step).sum(0)
        dD += (e * x[:, t]).sum(0)
        dbias += got["ddt"][:, t].sum(0)
        lam = lam * a
    got["dB"], got["dC"] = got["dB"].view(b, T, G, N), got["dC"].view(b, T, G, N)
    return dict(got, dA=dA.view(D, N), dD=dD, ddt_bias=dbias, dh=lam.reshape(b, D, N))


def _exact_norm(s):
    c = s["case"]
    w = _f64(s["weight"])
    if c["dir"] == "train":
        r, dy = _f64(s["r"]), _f64(s["dy"])
        rms = torch.sqrt(r.square().mean(1) + s["eps"])[:, None]
        dot = (dy * w * r).sum(1, keepdim=True) / c["d"]
        dr = dy * w / rms - r * dot / rms ** 3
        dw = (dy * r / rms).sum(0)
        if s["dres"] is None:
            return {"dx": dr, "dweight": dw}
        dr = dr + _f64(s["dres"])
        return {"dx": dr, "dweight": dw, "dresidual": dr}
    r, out = _f64(s["x"]), {}
    if s["residual"] is not None:
        r = r + _f64(s["residual"])
        out["residual"] = r
        r = r.to(s["residual"].dtype).double()
    y = r * w / torch.sqrt(r.square().mean(1) + s["eps"])[:, None]
    if c["out"] == "io":
        return dict(out, y=y)
    d = c["d"]
    scales = torch.stack([torch.linalg.vector_norm(y[:, k:k + SCALE_GROUP], math.inf, dim=1)
                          for k in range(0, d, SCALE_GROUP)], 1)
    scales = scales.clamp(min=AMAX_FLOOR) / E4M3_MAX
    per = torch.arange(d, device=y.device) // SCALE_GROUP
    # the nearest e4m3 value of each: 4 significant bits, steps of 2^-9 at the smallest
    q = y / scales[:, per]
    exponent = torch.frexp(q.abs().clamp(min=2.0 ** -6)).exponent
    unit = torch.ldexp(torch.ones_like(q), exponent - 4)
    return dict(out, y=torch.round(q / unit) * unit, scales=scales)


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s)
