"""The plain 64-bit forms of the block operators against differentiation of their forward
formulas (automatic and by differences), and the one-token and ragged cases of each."""
import pytest
import torch

import block_reference as ref

F64 = torch.float64


def rnd(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, dtype=F64) * std


def conv_case(seed, b=2, T=5, C=3, W=4):
    g = torch.Generator().manual_seed(seed)
    return dict(x=rnd(g, b, T, C), weight=rnd(g, C, W), bias=rnd(g, C),
                state=rnd(g, b, W - 1, C)), rnd(g, b, T, C)


def scan_case(seed, b=2, T=5, ch=4, G=2, N=3):
    g = torch.Generator().manual_seed(seed)
    c = dict(x=rnd(g, b, T, ch), dt=rnd(g, b, T, ch), A=-torch.exp(rnd(g, ch, N, std=0.3)),
             B=rnd(g, b, T, G, N), C=rnd(g, b, T, G, N), D=rnd(g, ch), z=rnd(g, b, T, ch),
             bias=rnd(g, ch), h=rnd(g, b, ch, N))
    return c, rnd(g, b, T, ch), rnd(g, b, ch, N)


def differences(f, v, eps=1e-6):
    out = torch.zeros_like(v)
    for i in range(v.numel()):
        hi, lo = v.clone(), v.clone()
        hi.view(-1)[i] += eps
        lo.view(-1)[i] -= eps
        out.view(-1)[i] = (f(hi) - f(lo)) / (2 * eps)
    return out


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("lens", [[5, 5], [3, 0]])
def test_conv_gradients(act, lens):
    c, dy = conv_case(1)
    got = ref.conv_bwd(*c.values(), lens, act, dy)
    for k, n in zip(c, ("dx", "dweight", "dbias", "dstate")):
        num = differences(lambda v: (ref.conv(*dict(c, **{k: v}).values(), lens, act)[0]
                                     * dy).sum(), c[k])
        assert torch.allclose(got[n], num, atol=1e-7), n


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lens", [[5, 5], [2, 0]])
def test_scan_gradients(gate, softplus, lens):
    c, dy, dhT = scan_case(2)
    if not gate:
        c["z"] = None
    if not softplus:
        c["dt"], c["bias"] = c["dt"].abs(), c["bias"].abs()
    got = ref.scan_bwd(*c.values(), lens, softplus, dy, dhT)

    def loss(**kw):
        y, h = ref.scan(*dict(c, **kw).values(), lens, softplus)
        return (y * dy).sum() + (h * dhT).sum()

    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", bias="ddt_bias",
                 h="dh")
    for k, n in names.items():
        if c[k] is None:
            continue
        num = differences(lambda v: loss(**{k: v}), c[k])
        assert torch.allclose(got[n], num, atol=1e-6), n
        leaf = c[k].clone().requires_grad_()
        auto, = torch.autograd.grad(loss(**{k: leaf}), leaf)
        assert torch.allclose(got[n], auto, atol=1e-12), n


def test_norm_gradients():
    g = torch.Generator().manual_seed(3)
    x, w, dy, dres = rnd(g, 3, 7), rnd(g, 7), rnd(g, 3, 7), rnd(g, 3, 7)
    dr, dw = ref.norm_bwd(x, w, 1e-3, dy, dres)
    loss = lambda x, w: (ref.norm(x, None, w, 1e-3, F64)[0] * dy).sum() + (x * dres).sum()
    assert torch.allclose(dr, differences(lambda v: loss(v, w), x), atol=1e-7)
    assert torch.allclose(dw, differences(lambda v: loss(x, v), w), atol=1e-7)


def test_calls_chain():
    """A sequence in pieces, the last one token by token, is the whole sequence."""
    c, _ = conv_case(4, T=9)
    y, s = ref.conv(*c.values(), [9, 9], True)
    st, parts = c["state"], []
    for lo, hi in ((0, 1), (1, 6), (6, 7), (7, 8), (8, 9)):
        p, st = ref.conv(c["x"][:, lo:hi], c["weight"], c["bias"], st, [hi - lo] * 2, True)
        parts.append(p)
    assert torch.allclose(torch.cat(parts, 1), y, atol=1e-13) and torch.equal(st, s)
    c, _, _ = scan_case(5, T=6)
    y, h = ref.scan(*c.values(), [6, 6], True)
    hh, parts = c["h"], []
    for lo, hi in ((0, 4), (4, 5), (5, 6)):
        cut = {k: v[:, lo:hi] if k in ("x", "dt", "B", "C", "z") else v for k, v in c.items()}
        p, hh = ref.scan(*dict(cut, h=hh).values(), [hi - lo] * 2, True)
        parts.append(p)
    assert torch.allclose(torch.cat(parts, 1), y, atol=1e-14) and torch.allclose(hh, h, atol=1e-14)


def test_scan_closed_form():
    """Constant coefficients: h_t is a geometric sum."""
    T, a, d = 7, -0.5, 0.3
    one = lambda *s: torch.ones(s, dtype=F64)
    y, h = ref.scan(one(1, T, 1), one(1, T, 1) * d, one(1, 1) * a, one(1, T, 1, 1),
                    one(1, T, 1, 1), None, None, None, one(1, 1, 1) * 2, [T], False)
    q = torch.exp(torch.tensor(a * d, dtype=F64))
    want = 2 * q ** T + d * (1 - q ** T) / (1 - q)
    assert torch.allclose(h.view(()), want) and torch.allclose(y[0, -1, 0], want)
