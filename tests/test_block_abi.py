"""Host-side validation of the block operators' entry points (CPU only): every argument is
checked before anything is launched, and the packed structs have the header's layouts."""
import ctypes
import os
import subprocess

import pytest
import torch

from state_space_model_06_b200 import m3

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, WS = 0x10000, 0x100000         # addresses that no check looks behind
F32, BF16 = m3.M3_F32, m3.M3_BF16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m3.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return m3.load_library()


def rows(ptr=P, bs=64 * 16, ts=16):
    return bytes(m3.m3_rows(ptr, bs, ts))


def test_packed_layouts_match_the_header(tmp_path):
    """What the binding packs has the sizes and offsets of the C structs."""
    rows = m3._PACK_ROWS.__self__.size
    packs = dict(m3_rows=rows, m3_conv_dims=m3._PACK_CONV_DIMS.__self__.size,
                 m3_conv_grads=rows + m3._PACK_CONV_PARAMS.__self__.size,
                 m3_sel_dims=m3._PACK_SEL_DIMS.__self__.size,
                 m3_sel_inputs=5 * rows + m3._PACK_POINTERS.__self__.size,
                 m3_sel_grads=5 * rows + m3._PACK_POINTERS.__self__.size,
                 m3_norm_dims=m3._PACK_NORM_DIMS.__self__.size)
    src = tmp_path / "layout.c"
    lines = []
    for name in packs:
        ct = getattr(m3, name)
        lines.append('printf("%%zu", sizeof(%s));' % name)
        lines += ['printf(" %%zu", offsetof(%s, %s));' % (name, f[0]) for f in ct._fields_]
        lines.append('printf("\\n");')
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "m3.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    out = subprocess.check_output([str(exe)]).decode().splitlines()
    for line, (name, size) in zip(out, packs.items()):
        ct = getattr(m3, name)
        want = [int(v) for v in line.split()]
        assert want == [ctypes.sizeof(ct)] + [getattr(ct, f[0]).offset for f in ct._fields_], name
        assert size == want[0], name


# ---------------------------------------------------------------- convolution

def conv(lib, fn="fwd", dims=(2, 16, 4, BF16), T=64, x=rows(P + 0x8000), w=P, bias=P, state=P, y=rows(),
         flags=0, seqlens=None):
    d = bytes(m3.m3_conv_dims(*dims))
    if fn == "step":
        return lib.m3_conv_step(d, x, w, bias, state, y, flags, None)
    return lib.m3_conv_fwd(d, T, x, w, bias, seqlens, state, y, flags, None)


@pytest.mark.parametrize("fn", ["fwd", "step"])
@pytest.mark.parametrize("kw,status", [
    (dict(dims=(0, 16, 4, BF16)), m3.M3_ERR_SHAPE),
    (dict(dims=(2, 0, 4, BF16)), m3.M3_ERR_SHAPE),
    (dict(dims=(2, 16, 0, BF16)), m3.M3_ERR_SHAPE),
    (dict(dims=(2, 16, 9, BF16)), m3.M3_ERR_UNSUPPORTED),
    (dict(dims=(2, 16, 4, 5)), m3.M3_ERR_DTYPE),
    (dict(x=None), m3.M3_ERR_NULL),
    (dict(x=rows(0)), m3.M3_ERR_NULL),
    (dict(y=rows(0)), m3.M3_ERR_NULL),
    (dict(w=0), m3.M3_ERR_NULL),
    (dict(state=0), m3.M3_ERR_NULL),
    (dict(w=P + 2), m3.M3_ERR_ALIGN),
    (dict(bias=P + 1), m3.M3_ERR_ALIGN),
    (dict(x=rows(P + 1)), m3.M3_ERR_ALIGN),
    (dict(state=P + 1), m3.M3_ERR_ALIGN),
    (dict(x=rows(bs=-16)), m3.M3_ERR_SHAPE),
    (dict(y=rows(bs=8)), m3.M3_ERR_SHAPE),            # batch rows overlap
    (dict(flags=m3.M3_FLAG_DT_SOFTPLUS), m3.M3_ERR_UNSUPPORTED),
    (dict(flags=m3.M3_FLAG_DEBUG_CHECKS), m3.M3_ERR_UNSUPPORTED),
])
def test_conv_refusals(lib, fn, kw, status):
    assert conv(lib, fn, **kw) == status


def test_conv_prompt_refusals(lib):
    assert conv(lib, T=-1) == m3.M3_ERR_SHAPE
    assert conv(lib, T=(1 << 30) + 1) == m3.M3_ERR_UNSUPPORTED
    assert conv(lib, x=rows(ts=-16)) == m3.M3_ERR_SHAPE
    assert conv(lib, y=rows(ts=8)) == m3.M3_ERR_SHAPE           # token rows overlap
    assert conv(lib, y=rows(bs=32, ts=16)) == m3.M3_ERR_SHAPE   # sequences overlap
    assert conv(lib, y=rows(bs=0, ts=16)) == m3.M3_ERR_SHAPE
    assert conv(lib, seqlens=P + 2) == m3.M3_ERR_ALIGN
    assert conv(lib, x=rows(), y=rows()) == m3.M3_ERR_UNSUPPORTED       # in place
    assert conv(lib, T=0, x=None, y=None) == m3.M3_OK           # no tokens: nothing to do


def test_conv_backward_refusals(lib):
    d = m3.ConvDims(2, 16, 4, BF16)
    need = m3.m3_conv_bwd_workspace_bytes(d, 64)
    assert need >= 4 * 2 * 5 * 16

    Q, R = P + 0x8000, P + 0x10000

    def bwd(dx=(P, 1024, 16), dw=P, db=P, ds=P, dy=rows(Q), ws=WS, nb=need, bias=P, T=64):
        g = bytes(m3.m3_conv_grads(m3.m3_rows(*dx), dw, db, ds))
        return lib.m3_conv_bwd(bytes(d.c()), T, rows(R), P, bias, None, P, dy, g, ws, nb, 0, None)

    assert bwd(dw=0) == m3.M3_ERR_NULL
    assert bwd(db=0) == m3.M3_ERR_NULL
    assert bwd(dx=(0, 1024, 16)) == m3.M3_ERR_NULL
    assert bwd(dx=(P, 16, 16)) == m3.M3_ERR_SHAPE
    assert bwd(dx=(Q, 1024, 16)) == m3.M3_ERR_UNSUPPORTED        # dx over dy
    assert bwd(dx=(R, 1024, 16)) == m3.M3_ERR_UNSUPPORTED        # dx over x
    assert bwd(dy=rows(0)) == m3.M3_ERR_NULL
    assert bwd(ds=P + 2) == m3.M3_ERR_ALIGN
    assert bwd(ws=0) == m3.M3_ERR_WORKSPACE
    assert bwd(ws=WS + 16) == m3.M3_ERR_WORKSPACE
    assert bwd(nb=need - 1) == m3.M3_ERR_WORKSPACE
    assert bwd(T=-2) == m3.M3_ERR_SHAPE


# ---------------------------------------------------------------- selective scan

def sel_in(z=0, seqlens=0, A=P, D=P, bias=P, x=(P, 1024, 16), B=(P, 512, 8)):
    r = m3.m3_rows
    return bytes(m3.m3_sel_inputs(r(*x), r(P, 1024, 16), r(*B), r(P, 512, 8), r(z, 1024, 16), A, D,
                                  bias, seqlens))


def sel(lib, fn="fwd", dims=(2, 16, 1, 8, BF16), T=64, inp=None, h=P, y=rows(), ws=WS, nb=1 << 20,
        flags=0):
    d = bytes(m3.m3_sel_dims(*dims))
    inp = sel_in() if inp is None else inp
    if fn == "step":
        return lib.m3_sel_step(d, inp, h, y, flags, None)
    return lib.m3_sel_fwd(d, T, inp, h, y, ws, nb, flags, None)


@pytest.mark.parametrize("fn", ["fwd", "step"])
@pytest.mark.parametrize("kw,status", [
    (dict(dims=(2, 16, 3, 8, BF16)), m3.M3_ERR_SHAPE),        # groups do not divide channels
    (dict(dims=(2, 16, 1, 0, BF16)), m3.M3_ERR_SHAPE),
    (dict(dims=(2, 16, 1, 257, BF16)), m3.M3_ERR_UNSUPPORTED),
    (dict(dims=(2, 16, 1, 8, 2)), m3.M3_ERR_DTYPE),
    (dict(h=0), m3.M3_ERR_NULL),
    (dict(inp=sel_in(A=0)), m3.M3_ERR_NULL),
    (dict(inp=sel_in(x=(0, 1024, 16))), m3.M3_ERR_NULL),
    (dict(inp=sel_in(B=(P + 1, 512, 8))), m3.M3_ERR_ALIGN),
    (dict(inp=sel_in(z=P + 1)), m3.M3_ERR_ALIGN),
    (dict(inp=sel_in(D=P + 2)), m3.M3_ERR_ALIGN),
    (dict(h=P + 2), m3.M3_ERR_ALIGN),
    (dict(inp=sel_in(x=(P, -1, 16))), m3.M3_ERR_SHAPE),
    (dict(y=rows(bs=8)), m3.M3_ERR_SHAPE),
    (dict(y=rows(0)), m3.M3_ERR_NULL),
    (dict(flags=m3.M3_FLAG_SILU), m3.M3_ERR_UNSUPPORTED),
    (dict(flags=1 << 12), m3.M3_ERR_UNSUPPORTED),
])
def test_sel_refusals(lib, fn, kw, status):
    assert sel(lib, fn, **kw) == status


def test_sel_call_refusals(lib):
    assert sel(lib, T=-1) == m3.M3_ERR_SHAPE
    assert sel(lib, T=(1 << 30) + 1) == m3.M3_ERR_UNSUPPORTED
    assert sel(lib, ws=WS + 8) == m3.M3_ERR_WORKSPACE
    assert sel(lib, T=0, inp=b"") == m3.M3_OK
    assert sel(lib, "step", inp=sel_in(seqlens=P)) == m3.M3_ERR_UNSUPPORTED
    d = m3.SelDims(1, 64, 1, 16, BF16)
    # a long sequence of few channels is segmented: two states a segment and more
    assert m3.m3_sel_workspace_bytes(d, 8192) > m3.m3_sel_workspace_bytes(d, 32) == 256
    with pytest.raises(m3.M3Error):
        m3.m3_sel_workspace_bytes(d, -1)


def test_sel_backward_refusals(lib):
    d = m3.SelDims(2, 16, 1, 8, BF16)
    need = m3.m3_sel_bwd_workspace_bytes(d, 64)

    def bwd(T=64, inp=None, dz=P, dB=(P, 512, 8), dA=P, dD=P, db=P, dh=P, dhT=None, ws=WS, nb=need,
            flags=0):
        r = m3.m3_rows
        g = bytes(m3.m3_sel_grads(r(P, 1024, 16), r(P, 1024, 16), r(*dB), r(P, 512, 8),
                                  r(dz, 1024, 16), dA, dD, db, dh))
        return lib.m3_sel_bwd(bytes(d.c()), T, sel_in(z=P) if inp is None else inp, P, rows(), dhT, g,
                              ws, nb, flags, None)

    assert bwd(dz=0) == m3.M3_ERR_NULL                  # the gate is on
    assert bwd(dA=0) == m3.M3_ERR_NULL
    assert bwd(dD=0) == m3.M3_ERR_NULL
    assert bwd(db=0) == m3.M3_ERR_NULL
    assert bwd(dB=(P, 4, 8)) == m3.M3_ERR_SHAPE
    assert bwd(dhT=P + 1) == m3.M3_ERR_ALIGN
    assert bwd(ws=0) == m3.M3_ERR_WORKSPACE
    assert bwd(nb=need - 256) == m3.M3_ERR_WORKSPACE
    assert bwd(flags=m3.M3_FLAG_FORCE_SIMT) == m3.M3_ERR_UNSUPPORTED
    assert bwd(T=-1) == m3.M3_ERR_SHAPE


# ---------------------------------------------------------------- norm

def norm(lib, dims=(4, 64, BF16, F32, m3.M3_OUT_IO), x=(P, 64), res=(P, 64), w=P, eps=1e-6,
         y=(P, 64), scales=P, ro=(P, 64)):
    return lib.m3_norm_fwd(bytes(m3.m3_norm_dims(*dims)), *x, *res, w, eps, *y, scales, *ro, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dims=(-1, 64, BF16, F32, 0)), m3.M3_ERR_SHAPE),
    (dict(dims=(4, 0, BF16, F32, 0)), m3.M3_ERR_SHAPE),
    (dict(dims=(4, 32769, BF16, F32, 0)), m3.M3_ERR_UNSUPPORTED),
    (dict(dims=(4, 64, 9, F32, 0)), m3.M3_ERR_DTYPE),
    (dict(dims=(4, 64, BF16, F32, 7)), m3.M3_ERR_DTYPE),
    (dict(res=(0, 0)), m3.M3_ERR_DTYPE),              # no residual: res_dtype is x's
    (dict(eps=-1e-6), m3.M3_ERR_SHAPE),
    (dict(eps=float("nan")), m3.M3_ERR_SHAPE),
    (dict(eps=float("inf")), m3.M3_ERR_SHAPE),
    (dict(x=(0, 64)), m3.M3_ERR_NULL),
    (dict(y=(0, 64)), m3.M3_ERR_NULL),
    (dict(x=(P, 63)), m3.M3_ERR_SHAPE),
    (dict(x=(P + 1, 64)), m3.M3_ERR_ALIGN),
    (dict(res=(P + 2, 64)), m3.M3_ERR_ALIGN),
    (dict(w=P + 2), m3.M3_ERR_ALIGN),
    (dict(dims=(4, 64, BF16, F32, m3.M3_OUT_E4M3), scales=0), m3.M3_ERR_NULL),
    (dict(dims=(0, 64, BF16, F32, 0), x=(0, 0), y=(0, 0)), m3.M3_OK),
])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


def test_norm_backward_refusals(lib):
    d = m3.NormDims(4, 64, BF16, F32)
    need = m3.m3_norm_bwd_workspace_bytes(d)

    def bwd(r=(P, 64), w=P, dy=(P, 64), dx=(P, 64), dw=P, ws=WS, nb=need, eps=1e-6):
        return lib.m3_norm_bwd(bytes(d.c()), *r, w, eps, *dy, 0, 0, *dx, 0, 0, dw, ws, nb, None)

    assert bwd(r=(0, 64)) == m3.M3_ERR_NULL
    assert bwd(dy=(0, 64)) == m3.M3_ERR_NULL
    assert bwd(dx=(P, 8)) == m3.M3_ERR_SHAPE
    assert bwd(dw=0) == m3.M3_ERR_NULL
    assert bwd(ws=0) == m3.M3_ERR_WORKSPACE
    assert bwd(nb=need - 1) == m3.M3_ERR_WORKSPACE
    assert bwd(eps=-1.0) == m3.M3_ERR_SHAPE


# ---------------------------------------------------------------- the binding's checks

def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(2, 3, 16, dtype=torch.bfloat16)
    with pytest.raises(m3.M3Error) as e:
        m3.m3_conv_fwd(m3.ConvDims(2, 16, 4), 3, x, torch.zeros(16, 4), None,
                       torch.zeros(2, 3, 16, dtype=torch.bfloat16), x)
    assert e.value.status == m3.M3_ERR_UNSUPPORTED


class Fake:
    """A tensor's outside, on a CUDA device that this machine does not have."""

    def __init__(self, t, device=0):
        self.t, self.dev = t, device
        self.dtype, self.shape, self.device = t.dtype, t.shape, f"cuda:{device}"

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("change,status", [
    (dict(x=torch.zeros(2, 3, 16)), m3.M3_ERR_DTYPE),
    (dict(x=torch.zeros(2, 4, 16, dtype=torch.bfloat16)), m3.M3_ERR_SHAPE),
    (dict(x=torch.zeros(2, 3, 32, dtype=torch.bfloat16)[..., ::2]), m3.M3_ERR_SHAPE),
    (dict(weight=torch.zeros(4, 16).t()), m3.M3_ERR_SHAPE),
    (dict(state=torch.zeros(2, 2, 16, dtype=torch.bfloat16)), m3.M3_ERR_SHAPE),
    (dict(state=torch.zeros(2, 3, 16)), m3.M3_ERR_DTYPE),
    (dict(seqlens=torch.zeros(2, dtype=torch.int64)), m3.M3_ERR_DTYPE),
])
def test_binding_checks_tensors_against_dims(lib, change, status):
    args = dict(x=torch.zeros(2, 3, 16, dtype=torch.bfloat16), weight=torch.zeros(16, 4),
                bias=None, state=torch.zeros(2, 3, 16, dtype=torch.bfloat16),
                y=torch.zeros(2, 3, 16, dtype=torch.bfloat16), seqlens=None)
    args.update(change)
    args = {k: None if v is None else Fake(v) for k, v in args.items()}
    with pytest.raises(m3.M3Error) as e:
        m3.m3_conv_fwd(m3.ConvDims(2, 16, 4), 3, **args)
    assert e.value.status == status


def test_binding_refuses_several_devices(lib):
    x = torch.zeros(2, 3, 16, dtype=torch.bfloat16)
    with pytest.raises(m3.M3Error) as e:
        m3.m3_conv_fwd(m3.ConvDims(2, 16, 4), 3, Fake(x), Fake(torch.zeros(16, 4), 1), None,
                       Fake(x), Fake(x))
    assert e.value.status == m3.M3_ERR_UNSUPPORTED
