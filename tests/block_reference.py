"""Plain 64-bit forms of the block operators on the CPU (torch.float64), one token after the
other, and bounds of what 32-bit kernels may be off by.

``absolute=True`` computes a formula with every factor replaced by its absolute value: the
result bounds the sum of the absolute values of all terms, which is what rounding errors are
relative to."""
import torch

F64 = torch.float64
U32 = 2.0 ** -24                    # half a step of fp32
# ex2.approx is good to 2 ulp (2^-22); its argument's rounding adds |log2 a| 2^-24, which the
# callers count by the size of the exponent
EX2 = 2.0 ** -22


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def lengths(seqlens, b, T):
    return [T] * b if seqlens is None else [min(max(int(n), 0), T) for n in seqlens.tolist()]


def silu(v):
    return v * torch.sigmoid(v)


# ---------------------------------------------------------------- convolution

def conv(x, weight, bias, state, lens, act):
    """x [b, T, C], weight [C, W], state [b, W-1, C]: y, the new state."""
    b, T, C = x.shape
    W = weight.shape[1]
    y, new = [], []
    for i in range(b):
        u = torch.cat([state[i], x[i, :lens[i]]])
        pre = torch.zeros(lens[i], C, dtype=F64)
        for k in range(W):
            pre = pre + u[k:k + lens[i]] * weight[:, k]
        if bias is not None:
            pre = pre + bias
        out = silu(pre) if act else pre
        y.append(torch.cat([out, torch.zeros(T - lens[i], C, dtype=F64)]))
        new.append(u[lens[i]:])
    return torch.stack(y), torch.stack(new)


def conv_bwd(x, weight, bias, state, lens, act, dy, absolute=False):
    """Gradients by the formula: dx, dweight, dbias, dstate."""
    b, T, C = x.shape
    W = weight.shape[1]
    m = torch.abs if absolute else (lambda v: v)
    dx, dstate = torch.zeros_like(x), torch.zeros_like(state)
    dw, db = torch.zeros_like(weight), torch.zeros(C, dtype=F64)
    for i in range(b):
        n = lens[i]
        u = torch.cat([state[i], x[i, :n]])
        pre = torch.zeros(n, C, dtype=F64)
        for k in range(W):
            pre = pre + u[k:k + n] * weight[:, k]
        if bias is not None:
            pre = pre + bias
        g = m(dy[i, :n])
        if act:
            s = torch.sigmoid(pre)
            g = g * (m(s) + m(pre * s * (1 - s)))
        du = torch.zeros_like(u)
        for k in range(W):
            du[k:k + n] += g * m(weight[:, k])
            dw[:, k] += (g * m(u[k:k + n])).sum(0)
        db += g.sum(0)
        dstate[i], dx[i, :n] = du[:W - 1], du[W - 1:]
    return dict(dx=dx, dweight=dw, dbias=db, dstate=dstate)


# ---------------------------------------------------------------- selective scan

def _delta(dt, bias, softplus):
    v = dt if bias is None else dt + bias
    return torch.logaddexp(v, torch.zeros_like(v)) if softplus else v


def scan(x, dt, A, B, C, D, z, bias, h, lens, softplus, absolute=False):
    """x, dt, z [b, T, ch]; B, C [b, T, G, N]; h [b, ch, N]: y (0 past a length), h_T."""
    b, T, ch = x.shape
    per = ch // B.shape[2]
    m = torch.abs if absolute else (lambda v: v)
    delta = _delta(dt, bias, softplus)
    ys = []
    h = m(h)
    on = torch.tensor([[t < n for t in range(T)] for n in lens], dtype=torch.bool).view(b, T)
    for t in range(T):
        Bt, Ct = (m(v[:, t]).repeat_interleave(per, 1) for v in (B, C))
        d, live = delta[:, t, :, None], on[:, t, None]
        nh = torch.exp(d * A) * h + m(d) * m(x[:, t, :, None]) * Bt
        h = torch.where(live[..., None], nh, h)
        y = (Ct * h).sum(-1)
        if D is not None:
            y = y + m(D) * m(x[:, t])
        if z is not None:
            y = y * m(silu(z[:, t]))
        ys.append(torch.where(live, y, torch.zeros_like(y)))
    return (torch.stack(ys, 1) if T else torch.zeros_like(x)), h


def scan_bwd(x, dt, A, B, C, D, z, bias, h0, lens, softplus, dy, dhT, absolute=False):
    """Gradients by the formula, from the last token back."""
    b, T, ch = x.shape
    G, N = B.shape[2], B.shape[3]
    per = ch // G
    m = torch.abs if absolute else (lambda v: v)
    delta = _delta(dt, bias, softplus)
    dsp = torch.sigmoid(dt if bias is None else dt + bias) if softplus else torch.ones_like(dt)
    hs = [m(h0)]
    on = torch.tensor([[t < n for t in range(T)] for n in lens], dtype=F64).view(b, T)
    for t in range(T):
        Bt = m(B[:, t]).repeat_interleave(per, 1)
        d = (delta[:, t] * on[:, t, None])[..., None]
        hs.append(torch.exp(d * A) * hs[-1] + m(d) * m(x[:, t, :, None]) * Bt)
    lam = torch.zeros_like(h0) if dhT is None else m(dhT)
    g = {k: torch.zeros_like(v) for k, v in dict(dx=x, ddt=x, dB=B, dC=C, dA=A).items()}
    g["dz"] = torch.zeros_like(x)
    g["dD"], g["ddt_bias"] = torch.zeros(ch, dtype=F64), torch.zeros(ch, dtype=F64)
    for t in reversed(range(T)):
        o = on[:, t, None]
        Bt, Ct = (m(v[:, t]).repeat_interleave(per, 1) for v in (B, C))
        e = m(dy[:, t]) * o
        if z is not None:
            sg = torch.sigmoid(z[:, t])
            y = (Ct * hs[t + 1]).sum(-1) + (0 if D is None else m(D) * m(x[:, t]))
            g["dz"][:, t] = e * y * (m(sg) + m(z[:, t] * sg * (1 - sg))
                                     if absolute else sg * (1 + z[:, t] * (1 - sg)))
            e = e * m(z[:, t] * sg)
        d = (delta[:, t] * o)[..., None]
        a = torch.exp(d * A)
        lam = lam + Ct * e[..., None]
        g["dC"][:, t] = (hs[t + 1] * e[..., None]).view(b, G, per, N).sum(2)
        g["dB"][:, t] = (lam * m(d) * m(x[:, t, :, None])).view(b, G, per, N).sum(2)
        lb = (lam * Bt).sum(-1)
        q = lam * a * hs[t]
        g["dx"][:, t] = m(d[..., 0]) * lb + (0 if D is None else m(D) * e)
        dd = m(x[:, t]) * lb * o + (q * m(A)).sum(-1) * o
        g["ddt"][:, t] = dd * dsp[:, t]
        g["dA"] += (q * m(d)).sum(0)
        g["dD"] += (e * m(x[:, t])).sum(0)
        lam = lam * a
    g["ddt_bias"] = g["ddt"].sum((0, 1))
    g["dh"] = lam
    return g


def scan_bounds(T, N, ch, A, dt, bias, softplus):
    """Relative error (to the sum of absolute terms) of a path through the recurrence in 32 bits.

    A path is a product of at most T decays with a handful of other factors, added up over at
    most T + N + ch terms (the sums are trees or short chains: at most T + N + 64 roundings in a
    row).  Each decay is off by EX2 for the exponential, a rounding for the product with the
    state, and by |delta A| times the relative error of delta A for its argument; over a path the
    last adds up to |log P| times that error, and P |log P| <= 1/e, so it is counted once with
    the largest single exponent.  delta is off by 4 roundings and by the rounding of dt + bias
    times the slope of log softplus, at most 1: |dt + bias| U32."""
    v = f64(dt) if bias is None else f64(dt) + f64(bias)
    rel_delta = 6 * U32 + float(v.abs().max()) * U32 + 2.0 ** -21
    return T * (EX2 + 2 * U32) + (T + N + 64) * U32 + 4 * rel_delta + 16 * U32


# ---------------------------------------------------------------- norm

def norm(x, residual, weight, eps, res_dtype):
    """y, r (rounded to res_dtype where there is a residual)."""
    r = x if residual is None else (x + residual).to(res_dtype).to(F64)
    y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    return (y if weight is None else y * weight), r


def norm_bwd(r, weight, eps, dy, dres, absolute=False):
    m = torch.abs if absolute else (lambda v: v)
    rstd = 1 / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    u = m(r) * rstd
    g = m(dy) if weight is None else m(dy) * m(weight)
    back = u * (g * u).mean(-1, keepdim=True)
    dr = rstd * (g + back if absolute else g - back)
    if dres is not None:
        dr = dr + m(dres)
    return dr, (m(dy) * u).sum(0)
