"""Thin ctypes binding of the C ABI in ``include/m3.h`` (libm3.so, built in-tree).

The functions keep the C names and only marshal arguments: torch tensors become
device pointers, dims become an ``m3_dims`` struct, the current torch stream is
passed as the cudaStream_t.  Every step of the computation runs in the CUDA
kernels of libm3.so; there is no fallback of any kind -- if the library is
missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass, replace

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libm3.so")

M3_OK, M3_ERR_NULL, M3_ERR_SHAPE, M3_ERR_DTYPE, M3_ERR_ALIGN, M3_ERR_UNSUPPORTED, \
    M3_ERR_WORKSPACE, M3_ERR_LAUNCH, M3_ERR_TIMEOUT, M3_ERR_CUDA, M3_ERR_RANGE = range(11)
M3_F32, M3_BF16 = 0, 1
M3_FLAG_THETA_IS_ANGLE = 1
M3_FLAG_FORCE_SIMT = 2
M3_FLAG_TEST_STALL = 4
M3_FLAG_DEBUG_CHECKS = 8
M3_FLAG_SILU = 16
M3_FLAG_DT_SOFTPLUS = 32
M3_OUT_IO, M3_OUT_E4M3 = 0, 1

EXPORTED = ("m3_state_bytes", "m3_state_init", "m3_scan_workspace_bytes", "m3_scan_fwd",
            "m3_decode_step", "m3_query_status", "m3_scan_fwd_noalloc", "m3_scan_fwd_gated",
            "m3_decode_step_gated", "m3_scan_workspace_bytes_ex", "m3_scan_fwd_ex",
            "m3_decode_step_ex", "m3_scan_bwd_workspace_bytes", "m3_scan_bwd",
            "m3_scan_bwd_workspace_bytes_ex", "m3_scan_bwd_ex",
            "m3_conv_fwd", "m3_conv_step", "m3_conv_bwd_workspace_bytes", "m3_conv_bwd",
            "m3_sel_workspace_bytes", "m3_sel_fwd", "m3_sel_step", "m3_sel_bwd_workspace_bytes",
            "m3_sel_bwd", "m3_norm_fwd", "m3_norm_bwd_workspace_bytes", "m3_norm_bwd",
            "m3_status_string")


class M3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {m3_status_string(status)} (status {status})")


class m3_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("nheads", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32)]


class m3_state(ctypes.Structure):
    _fields_ = [("h", ctypes.c_void_p), ("x_prev", ctypes.c_void_p), ("B_prev", ctypes.c_void_p)]


class m3_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "dB", "dC", "ddt", "dA", "dlam", "dtheta",
                                               "dD", "dh0", "dx_prev", "dB_prev")]


class m3_extra_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dz", "dB_bias", "dC_bias", "dx_expand",
                                                "dz_expand")]


class m3_extras(ctypes.Structure):
    _fields_ = [("z", ctypes.c_void_p), ("B_bias", ctypes.c_void_p), ("C_bias", ctypes.c_void_p),
                ("bc_norm_eps", ctypes.c_float), ("x_expand", ctypes.c_void_p),
                ("z_expand", ctypes.c_void_p)]


class m3_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class m3_conv_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "channels", "width", "io_dtype")]


class m3_conv_grads(ctypes.Structure):
    _fields_ = [("dx", m3_rows), ("dweight", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("dstate", ctypes.c_void_p)]


class m3_sel_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "channels", "ngroups", "dstate",
                                              "io_dtype")]


class m3_sel_inputs(ctypes.Structure):
    _fields_ = [(n, m3_rows) for n in ("x", "dt", "B", "C", "z")] + \
        [(n, ctypes.c_void_p) for n in ("A", "D", "dt_bias", "seqlens")]


class m3_sel_grads(ctypes.Structure):
    _fields_ = [(n, m3_rows) for n in ("dx", "ddt", "dB", "dC", "dz")] + \
        [(n, ctypes.c_void_p) for n in ("dA", "dD", "ddt_bias", "dh")]


class m3_norm_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "width", "io_dtype", "res_dtype", "out")]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libm3.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library not built: {path} (run __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        vp, u32, i32, sz = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int32, ctypes.c_size_t
        dp = ctypes.POINTER(m3_dims)
        sp = ctypes.POINTER(m3_state)
        szp = ctypes.POINTER(ctypes.c_size_t)
        lib.m3_state_bytes.argtypes = [dp, szp, szp, szp]
        lib.m3_state_init.argtypes = [dp, sp, vp, vp]
        lib.m3_scan_workspace_bytes.argtypes = [dp, i32, i32, szp]
        lib.m3_scan_fwd.argtypes = [dp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, sp, vp, vp, sz,
                                    u32, vp]
        lib.m3_decode_step.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, sp, vp, u32, vp]
        lib.m3_scan_fwd_gated.argtypes = [dp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sp,
                                          vp, vp, sz, u32, vp]
        lib.m3_decode_step_gated.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sp, vp,
                                             u32, vp]
        ep = ctypes.POINTER(m3_extras)
        lib.m3_scan_workspace_bytes_ex.argtypes = [dp, i32, i32, ep, szp]
        lib.m3_scan_fwd_ex.argtypes = [dp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, ep, sp, vp,
                                       vp, sz, u32, vp]
        lib.m3_decode_step_ex.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, ep, sp, vp, u32, vp]
        lib.m3_scan_fwd_noalloc.argtypes = [dp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, sp, vp,
                                            u32, vp]
        lib.m3_scan_bwd_workspace_bytes.argtypes = [dp, i32, szp]
        lib.m3_scan_bwd.argtypes = [dp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sp, vp, vp,
                                    ctypes.POINTER(m3_grads), vp, sz, u32, vp]
        lib.m3_scan_bwd_workspace_bytes_ex.argtypes = [dp, i32, ep, szp]
        lib.m3_scan_bwd_ex.argtypes = [dp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sp, ep, vp, vp,
                                       ctypes.POINTER(m3_grads), ctypes.POINTER(m3_extra_grads),
                                       vp, sz, u32, vp]
        # block operators: structs are passed as packed bytes (see _PACK_ROWS)
        i64, f32 = ctypes.c_int64, ctypes.c_float
        lib.m3_conv_fwd.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, u32, vp]
        lib.m3_conv_step.argtypes = [vp, vp, vp, vp, vp, vp, u32, vp]
        lib.m3_conv_bwd_workspace_bytes.argtypes = [vp, i32, szp]
        lib.m3_conv_bwd.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp]
        lib.m3_sel_workspace_bytes.argtypes = [vp, i32, szp]
        lib.m3_sel_fwd.argtypes = [vp, i32, vp, vp, vp, vp, sz, u32, vp]
        lib.m3_sel_step.argtypes = [vp, vp, vp, vp, u32, vp]
        lib.m3_sel_bwd_workspace_bytes.argtypes = [vp, i32, szp]
        lib.m3_sel_bwd.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, sz, u32, vp]
        lib.m3_norm_fwd.argtypes = [vp, vp, i64, vp, i64, vp, f32, vp, i64, vp, vp, i64, vp]
        lib.m3_norm_bwd_workspace_bytes.argtypes = [vp, szp]
        lib.m3_norm_bwd.argtypes = [vp, vp, i64, vp, f32, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp,
                                    sz, vp]
        lib.m3_query_status.argtypes = [vp, vp]
        lib.m3_status_string.argtypes = [ctypes.c_int]
        lib.m3_status_string.restype = ctypes.c_char_p
        for name in EXPORTED[:-1]:
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


@dataclass
class Dims:
    batch: int
    nheads: int
    ngroups: int
    headdim: int
    dstate: int
    rank: int = 1
    io_dtype: int = M3_BF16

    def c(self) -> m3_dims:
        return m3_dims(self.batch, self.nheads, self.ngroups, self.headdim, self.dstate,
                       self.rank, self.io_dtype)


def io_dtype_of(t: torch.dtype) -> int:
    return {torch.bfloat16: M3_BF16, torch.float32: M3_F32}[t]


def torch_dtype_of(io: int) -> torch.dtype:
    return {M3_BF16: torch.bfloat16, M3_F32: torch.float32}[io]


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != M3_OK:
        raise M3Error(status, where)


def m3_status_string(status: int) -> str:
    return load_library().m3_status_string(int(status)).decode()


class State:
    """Caller-owned resumable state (h fp32, previous token's x and B in io dtype)."""

    def __init__(self, dims: Dims, device="cuda"):
        io = torch_dtype_of(dims.io_dtype)
        self.dims = dims
        self.h = torch.zeros(dims.batch, dims.nheads, dims.dstate, dims.headdim,
                             dtype=torch.float32, device=device)
        self.x_prev = torch.zeros(dims.batch, dims.nheads, dims.rank, dims.headdim, dtype=io,
                                  device=device)
        self.B_prev = torch.zeros(dims.batch, dims.ngroups, dims.rank, dims.dstate, dtype=io,
                                  device=device)

    def c(self) -> m3_state:
        return m3_state(self.h.data_ptr(), self.x_prev.data_ptr(), self.B_prev.data_ptr())

    def rows(self, lo: int, hi: int) -> "State":
        """Batch rows [lo, hi) of this state (the same memory), for a call on a slice of
        the batch: every tensor of the state leads with the batch axis."""
        v = State.__new__(State)
        v.dims = replace(self.dims, batch=hi - lo)
        v.h, v.x_prev, v.B_prev = self.h[lo:hi], self.x_prev[lo:hi], self.B_prev[lo:hi]
        return v


def m3_state_bytes(dims: Dims):
    h, x, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().m3_state_bytes(ctypes.byref(dims.c()), ctypes.byref(h), ctypes.byref(x),
                                         ctypes.byref(b)), "m3_state_bytes")
    return h.value, x.value, b.value


def m3_state_init(dims: Dims, state: State, h0=None, stream=None):
    st = state.c()
    _check(load_library().m3_state_init(ctypes.byref(dims.c()), ctypes.byref(st), _ptr(h0),
                                        _stream(stream)), "m3_state_init")


def m3_scan_workspace_bytes(dims: Dims, seqlen: int, chunk: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().m3_scan_workspace_bytes(ctypes.byref(dims.c()), int(seqlen), int(chunk),
                                                  ctypes.byref(n)), "m3_scan_workspace_bytes")
    return n.value


def m3_scan_fwd(dims: Dims, seqlen: int, chunk: int, x, B, C, dt, A, lam, theta, D,
                state: State, y, workspace, flags: int = 0, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = state.c()
    _check(load_library().m3_scan_fwd(
        ctypes.byref(dims.c()), int(seqlen), int(chunk), _ptr(x), _ptr(B), _ptr(C), _ptr(dt),
        _ptr(A), _ptr(lam), _ptr(theta), _ptr(D), ctypes.byref(st), _ptr(y), _ptr(workspace),
        ws_bytes, int(flags), _stream(stream)), "m3_scan_fwd")


def m3_scan_fwd_noalloc(dims: Dims, seqlen: int, chunk: int, x, B, C, dt, A, lam, theta, D,
                        state: State, y, flags: int = 0, stream=None):
    """Prefill for callers that cannot allocate device memory: no workspace argument;
    the library lends its own fixed scratch (see include/m3.h)."""
    st = state.c()
    _check(load_library().m3_scan_fwd_noalloc(
        ctypes.byref(dims.c()), int(seqlen), int(chunk), _ptr(x), _ptr(B), _ptr(C), _ptr(dt),
        _ptr(A), _ptr(lam), _ptr(theta), _ptr(D), ctypes.byref(st), _ptr(y), int(flags),
        _stream(stream)), "m3_scan_fwd_noalloc")


def m3_scan_fwd_gated(dims: Dims, seqlen: int, chunk: int, x, B, C, dt, A, lam, theta, D, z,
                      state: State, y, workspace, flags: int = 0, stream=None):
    """Prefill with the fused output gate y * SiLU(z) (z in the layout and dtype of y)."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = state.c()
    _check(load_library().m3_scan_fwd_gated(
        ctypes.byref(dims.c()), int(seqlen), int(chunk), _ptr(x), _ptr(B), _ptr(C), _ptr(dt),
        _ptr(A), _ptr(lam), _ptr(theta), _ptr(D), _ptr(z), ctypes.byref(st), _ptr(y),
        _ptr(workspace), ws_bytes, int(flags), _stream(stream)), "m3_scan_fwd_gated")


@dataclass
class Extras:
    """Optional fused parts (see m3_extras in include/m3.h): output gate z, BC biases
    B_bias / C_bias [H][N] fp32, BCNorm epsilon (0: off), MIMO lightweight expansion
    weights x_expand / z_expand [H][R][P] fp32 (x, z then hold [..][H][P])."""
    z: object = None
    B_bias: object = None
    C_bias: object = None
    bc_norm_eps: float = 0.0
    x_expand: object = None
    z_expand: object = None

    def c(self) -> m3_extras:
        return m3_extras(_ptr(self.z), _ptr(self.B_bias), _ptr(self.C_bias),
                         float(self.bc_norm_eps), _ptr(self.x_expand), _ptr(self.z_expand))


def _ex_ref(ex):
    return ctypes.byref(ex.c()) if ex is not None else None


def m3_scan_workspace_bytes_ex(dims: Dims, seqlen: int, chunk: int, ex) -> int:
    n = ctypes.c_size_t()
    _check(load_library().m3_scan_workspace_bytes_ex(ctypes.byref(dims.c()), int(seqlen),
                                                     int(chunk), _ex_ref(ex), ctypes.byref(n)),
           "m3_scan_workspace_bytes_ex")
    return n.value


def m3_scan_fwd_ex(dims: Dims, seqlen: int, chunk: int, x, B, C, dt, A, lam, theta, D, ex,
                   state: State, y, workspace, flags: int = 0, stream=None):
    """Prefill with the optional fused parts in ``ex`` (an Extras, or None)."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = state.c()
    _check(load_library().m3_scan_fwd_ex(
        ctypes.byref(dims.c()), int(seqlen), int(chunk), _ptr(x), _ptr(B), _ptr(C), _ptr(dt),
        _ptr(A), _ptr(lam), _ptr(theta), _ptr(D), _ex_ref(ex), ctypes.byref(st), _ptr(y),
        _ptr(workspace), ws_bytes, int(flags), _stream(stream)), "m3_scan_fwd_ex")


def m3_decode_step_ex(dims: Dims, x, B, C, dt, A, lam, theta, D, ex, state: State, y,
                      flags: int = 0, stream=None):
    """Decode step with the optional fused parts in ``ex`` (an Extras, or None)."""
    st = state.c()
    _check(load_library().m3_decode_step_ex(
        ctypes.byref(dims.c()), _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(A), _ptr(lam),
        _ptr(theta), _ptr(D), _ex_ref(ex), ctypes.byref(st), _ptr(y), int(flags),
        _stream(stream)), "m3_decode_step_ex")


def alloc_workspace_ex(dims: Dims, seqlen: int, chunk: int, ex, device="cuda") -> torch.Tensor:
    """A workspace tensor of the size m3_scan_fwd_ex needs with these extras."""
    n = m3_scan_workspace_bytes_ex(dims, seqlen, chunk, ex)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def m3_decode_step_gated(dims: Dims, x, B, C, dt, A, lam, theta, D, z, state: State, y,
                         flags: int = 0, stream=None):
    """Decode step with the fused output gate y * SiLU(z)."""
    st = state.c()
    _check(load_library().m3_decode_step_gated(
        ctypes.byref(dims.c()), _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(A), _ptr(lam),
        _ptr(theta), _ptr(D), _ptr(z), ctypes.byref(st), _ptr(y), int(flags), _stream(stream)),
        "m3_decode_step_gated")


def m3_decode_step(dims: Dims, x, B, C, dt, A, lam, theta, D, state: State, y, flags: int = 0,
                   stream=None):
    st = state.c()
    _check(load_library().m3_decode_step(
        ctypes.byref(dims.c()), _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(A), _ptr(lam),
        _ptr(theta), _ptr(D), ctypes.byref(st), _ptr(y), int(flags), _stream(stream)),
        "m3_decode_step")


def m3_query_status(workspace, stream=None) -> int:
    """Synchronise the stream and return the device-side status word (M3_OK, M3_ERR_TIMEOUT or
    M3_ERR_RANGE)."""
    return int(load_library().m3_query_status(_ptr(workspace), _stream(stream)))


def alloc_workspace(dims: Dims, seqlen: int, chunk: int, device="cuda") -> torch.Tensor:
    """A workspace tensor of the size m3_scan_fwd needs (256-byte aligned by torch)."""
    n = m3_scan_workspace_bytes(dims, seqlen, chunk)
    return torch.zeros(n, dtype=torch.uint8, device=device)


GRAD_NAMES = ("dx", "dB", "dC", "ddt", "dA", "dlam", "dtheta", "dD", "dh0", "dx_prev", "dB_prev")


def alloc_grads(dims: Dims, seqlen: int, device="cuda") -> dict:
    """fp32 gradient tensors of m3_scan_bwd, in its layouts."""
    b, H, G, P, N, R, T = (dims.batch, dims.nheads, dims.ngroups, dims.headdim, dims.dstate,
                           dims.rank, seqlen)
    f = dict(dtype=torch.float32, device=device)
    return dict(dx=torch.empty(b, T, H, R, P, **f), dB=torch.empty(b, T, G, R, N, **f),
                dC=torch.empty(b, T, G, R, N, **f), ddt=torch.empty(b, T, H, **f),
                dA=torch.empty(b, T, H, **f), dlam=torch.empty(b, T, H, **f),
                dtheta=torch.empty(b, T, G, N // 2, **f), dD=torch.empty(H, **f),
                dh0=torch.empty(b, H, N, P, **f), dx_prev=torch.empty(b, H, R, P, **f),
                dB_prev=torch.empty(b, G, R, N, **f))


def m3_scan_bwd_workspace_bytes(dims: Dims, seqlen: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().m3_scan_bwd_workspace_bytes(ctypes.byref(dims.c()), int(seqlen),
                                                      ctypes.byref(n)),
           "m3_scan_bwd_workspace_bytes")
    return n.value


def alloc_bwd_workspace(dims: Dims, seqlen: int, device="cuda") -> torch.Tensor:
    return torch.zeros(m3_scan_bwd_workspace_bytes(dims, seqlen), dtype=torch.uint8,
                       device=device)


def m3_scan_bwd(dims: Dims, seqlen: int, x, B, C, dt, A, lam, theta, D, state0: State, dy,
                dhT, grads: dict, workspace, flags: int = 0, stream=None):
    """Backward pass of m3_scan_fwd: gradients into ``grads`` (see alloc_grads); state0 is
    the state the forward call started from (read only); dhT may be None."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = state0.c()
    g = m3_grads(*(_ptr(grads.get(k)) for k in GRAD_NAMES))
    _check(load_library().m3_scan_bwd(
        ctypes.byref(dims.c()), int(seqlen), _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(A),
        _ptr(lam), _ptr(theta), _ptr(D), ctypes.byref(st), _ptr(dy), _ptr(dhT), ctypes.byref(g),
        _ptr(workspace), ws_bytes, int(flags), _stream(stream)), "m3_scan_bwd")


EXTRA_GRAD_NAMES = ("dz", "dB_bias", "dC_bias", "dx_expand", "dz_expand")


def alloc_extra_grads(dims: Dims, seqlen: int, ex, device="cuda") -> dict:
    """fp32 gradient tensors of the parts of ``ex`` (an Extras) that are on."""
    b, H, P, N, R, T = dims.batch, dims.nheads, dims.headdim, dims.dstate, dims.rank, seqlen
    f = dict(dtype=torch.float32, device=device)
    out = {}
    if ex.z is not None:
        out["dz"] = torch.empty((b, T, H, P) if ex.z_expand is not None else (b, T, H, R, P), **f)
    if ex.B_bias is not None:
        out["dB_bias"] = torch.empty(H, N, **f)
    if ex.C_bias is not None:
        out["dC_bias"] = torch.empty(H, N, **f)
    if ex.x_expand is not None:
        out["dx_expand"] = torch.empty(H, R, P, **f)
    if ex.z_expand is not None:
        out["dz_expand"] = torch.empty(H, R, P, **f)
    return out


def m3_scan_bwd_workspace_bytes_ex(dims: Dims, seqlen: int, ex) -> int:
    n = ctypes.c_size_t()
    _check(load_library().m3_scan_bwd_workspace_bytes_ex(ctypes.byref(dims.c()), int(seqlen),
                                                         _ex_ref(ex), ctypes.byref(n)),
           "m3_scan_bwd_workspace_bytes_ex")
    return n.value


def alloc_bwd_workspace_ex(dims: Dims, seqlen: int, ex, device="cuda") -> torch.Tensor:
    return torch.zeros(m3_scan_bwd_workspace_bytes_ex(dims, seqlen, ex), dtype=torch.uint8,
                       device=device)


def m3_scan_bwd_ex(dims: Dims, seqlen: int, x, B, C, dt, A, lam, theta, D, state0: State, ex,
                   dy, dhT, grads: dict, extra_grads: dict, workspace, flags: int = 0,
                   stream=None):
    """Backward pass of m3_scan_fwd_ex: gradients into ``grads`` (alloc_grads; dx is
    [b][T][H][P] with x_expand) and ``extra_grads`` (alloc_extra_grads)."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = state0.c()
    g = m3_grads(*(_ptr(grads.get(k)) for k in GRAD_NAMES))
    xg = m3_extra_grads(*(_ptr(extra_grads.get(k)) for k in EXTRA_GRAD_NAMES))
    _check(load_library().m3_scan_bwd_ex(
        ctypes.byref(dims.c()), int(seqlen), _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(A),
        _ptr(lam), _ptr(theta), _ptr(D), ctypes.byref(st), _ex_ref(ex), _ptr(dy), _ptr(dhT),
        ctypes.byref(g), ctypes.byref(xg), _ptr(workspace), ws_bytes, int(flags),
        _stream(stream)), "m3_scan_bwd_ex")


# ---------------------------------------------------------------------------------------------
# Block operators: short causal convolution, selective scan, residual RMS norm.  Activations may
# be views (a half of a projection's output): their strides go to the library.  The tensors of a
# call must agree with its dims in shape and type; a mismatch raises M3Error before anything is
# launched (the library sees addresses only).  A call runs on its tensors' device, on that
# device's current stream unless ``stream`` is given.

_F32 = torch.float32
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_TYPE_OF = {M3_F32: torch.float32, M3_BF16: torch.bfloat16}


@dataclass
class ConvDims:
    batch: int
    channels: int
    width: int
    io_dtype: int = M3_BF16

    def c(self) -> m3_conv_dims:
        return m3_conv_dims(self.batch, self.channels, self.width, self.io_dtype)


@dataclass
class SelDims:
    batch: int
    channels: int
    ngroups: int
    dstate: int
    io_dtype: int = M3_BF16

    def c(self) -> m3_sel_dims:
        return m3_sel_dims(self.batch, self.channels, self.ngroups, self.dstate, self.io_dtype)


@dataclass
class NormDims:
    rows: int
    width: int
    io_dtype: int = M3_BF16
    res_dtype: int = M3_BF16
    out: int = M3_OUT_IO

    def c(self) -> m3_norm_dims:
        return m3_norm_dims(self.rows, self.width, self.io_dtype, self.res_dtype, self.out)


# A call's structs go to the library as packed bytes, in the layouts of include/m3.h (the ctypes
# structures above describe them field by field): single-token calls are short, and building
# ctypes structures would take longer than the kernel.
_PACK_CONV_DIMS = struct.Struct("4i").pack
_PACK_SEL_DIMS = struct.Struct("5i").pack
_PACK_NORM_DIMS = struct.Struct("5i").pack
_PACK_ROWS = struct.Struct("Pqq").pack
_PACK_CONV_PARAMS = struct.Struct("PPP").pack      # behind dx: m3_conv_grads
_PACK_POINTERS = struct.Struct("PPPP").pack        # behind five rows: m3_sel_inputs, m3_sel_grads
_NO_ROWS = _PACK_ROWS(0, 0, 0)


def _bad(status, name, t, what):
    raise M3Error(status, f"{name}: got {t.dtype} {tuple(t.shape)} on {t.device}, strides "
                          f"{t.stride()}; expected {what}")


def _device(t, name):
    """The index of a call's device: that of its first tensor."""
    if t is None:
        raise M3Error(M3_ERR_NULL, name)
    dev = t.get_device()
    if dev < 0:
        _bad(M3_ERR_UNSUPPORTED, name, t, "a CUDA tensor")
    return dev


def _must_be(t, shape, dtype, dev, name, contiguous):
    """Raises what is wrong with a tensor (a last axis of one element may have any stride)."""
    if t.dtype is not dtype:
        _bad(M3_ERR_DTYPE, name, t, dtype)
    if t.shape != shape:
        _bad(M3_ERR_SHAPE, name, t, shape)
    if t.get_device() != dev:
        _bad(M3_ERR_UNSUPPORTED, name, t, f"device {dev}")
    if not contiguous:
        _bad(M3_ERR_SHAPE, name, t, "contiguous rows")


def _rows(t, shape, dtype, dev, name):
    """An activation of this shape ([batch, T, width] or [batch, width]) as a packed m3_rows."""
    if t is None:
        return _NO_ROWS
    st = t.stride()
    if st[-1] != 1 or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _must_be(t, shape, dtype, dev, name, st[-1] == 1 or shape[-1] == 1)
    return _PACK_ROWS(t.data_ptr(), st[0], st[1])


def _group_rows(t, shape, dtype, dev, name):
    """The same of B or C ([.., groups, states]): the groups of a row lie behind each other."""
    if t is None:
        return _NO_ROWS
    st, n = t.stride(), shape[-1]
    _must_be(t, shape, dtype, dev, name,
             (st[-1] == 1 or n == 1) and (st[-2] == n or shape[-2] == 1))
    return _PACK_ROWS(t.data_ptr(), st[0], st[1])


def _packed(t, shape, dtype, dev, name):
    """A packed tensor's address (None: 0)."""
    if t is None:
        return 0
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != dev):
        _must_be(t, shape, dtype, dev, name, t.is_contiguous())
    return t.data_ptr()


def _matrix(t, shape, dtypes, dev, name):
    """A [rows, width] tensor's address and row stride."""
    if t is None:
        return 0, 0
    st = t.stride()
    if st[-1] != 1 or t.dtype not in dtypes or t.shape != shape or t.get_device() != dev:
        _must_be(t, shape, t.dtype if t.dtype in dtypes else dtypes[0], dev, name,
                 st[-1] == 1 or shape[-1] == 1)
    return t.data_ptr(), st[0]


def _workspace(t, dev, name):
    if t is None:
        return None, 0
    if not t.is_contiguous():
        _bad(M3_ERR_WORKSPACE, name, t, "a contiguous workspace")
    if t.get_device() != dev:
        _bad(M3_ERR_UNSUPPORTED, name, t, f"device {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _run(name, dev, stream, *args):
    """Call the library on device ``dev``: on its current stream, or on ``stream``."""
    fn = getattr(_lib or load_library(), name)
    if stream is None:
        stream = _raw_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if dev == _current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        raise M3Error(status, name)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _io_type(dims, name):
    t = _TYPE_OF.get(dims.io_dtype)
    if t is None:
        raise M3Error(M3_ERR_DTYPE, name)
    return t


def m3_conv_fwd(dims: ConvDims, seqlen: int, x, weight, bias, state, y, seqlens=None,
                flags: int = 0, stream=None):
    """Short causal convolution of x [b, T, C] into y, carrying ``state`` [b, W-1, C] (updated in
    place).  ``bias`` and ``seqlens`` (int32 [b]) may be None; flags: M3_FLAG_SILU."""
    name, b, C, W = "m3_conv_fwd", dims.batch, dims.channels, dims.width
    io, dev = _io_type(dims, name), _device(x, name)
    shape = (b, seqlen, C)
    _run(name, dev, stream, _PACK_CONV_DIMS(b, C, W, dims.io_dtype), seqlen,
         _rows(x, shape, io, dev, name), _packed(weight, (C, W), _F32, dev, name),
         _packed(bias, (C,), _F32, dev, name), _packed(seqlens, (b,), torch.int32, dev, name),
         _packed(state, (b, W - 1, C), io, dev, name), _rows(y, shape, io, dev, name), flags)


def m3_conv_step(dims: ConvDims, x, weight, bias, state, y, flags: int = 0, stream=None):
    """One token of every sequence: x, y [b, C]."""
    name, b, C, W = "m3_conv_step", dims.batch, dims.channels, dims.width
    io, dev = _io_type(dims, name), _device(x, name)
    shape = (b, C)
    _run(name, dev, stream, _PACK_CONV_DIMS(b, C, W, dims.io_dtype),
         _rows(x, shape, io, dev, name), _packed(weight, (C, W), _F32, dev, name),
         _packed(bias, (C,), _F32, dev, name), _packed(state, (b, W - 1, C), io, dev, name),
         _rows(y, shape, io, dev, name), flags)


def m3_conv_bwd_workspace_bytes(dims: ConvDims, seqlen: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().m3_conv_bwd_workspace_bytes(ctypes.byref(dims.c()), int(seqlen),
                                                      ctypes.byref(n)),
           "m3_conv_bwd_workspace_bytes")
    return n.value


def alloc_conv_bwd_workspace(dims: ConvDims, seqlen: int, device="cuda") -> torch.Tensor:
    return torch.empty(m3_conv_bwd_workspace_bytes(dims, seqlen), dtype=torch.uint8, device=device)


def alloc_conv_grads(dims: ConvDims, seqlen: int, device="cuda") -> dict:
    """Gradient tensors of m3_conv_bwd."""
    b, C, W = dims.batch, dims.channels, dims.width
    f = dict(dtype=_F32, device=device)
    return dict(dx=torch.empty(b, seqlen, C, dtype=torch_dtype_of(dims.io_dtype), device=device),
                dweight=torch.empty(C, W, **f), dbias=torch.empty(C, **f),
                dstate=torch.empty(b, W - 1, C, **f))


def m3_conv_bwd(dims: ConvDims, seqlen: int, x, weight, bias, state0, dy, grads: dict, workspace,
                seqlens=None, flags: int = 0, stream=None):
    """Backward of m3_conv_fwd into ``grads`` (see alloc_conv_grads; dbias is needed with a bias,
    dstate may be absent); ``state0`` is the state that the forward call started from."""
    name, b, C, W = "m3_conv_bwd", dims.batch, dims.channels, dims.width
    io, dev = _io_type(dims, name), _device(x, name)
    shape, get = (b, seqlen, C), grads.get
    _run(name, dev, stream, _PACK_CONV_DIMS(b, C, W, dims.io_dtype), seqlen,
         _rows(x, shape, io, dev, name), _packed(weight, (C, W), _F32, dev, name),
         _packed(bias, (C,), _F32, dev, name), _packed(seqlens, (b,), torch.int32, dev, name),
         _packed(state0, (b, W - 1, C), io, dev, name), _rows(dy, shape, io, dev, name),
         _rows(get("dx"), shape, io, dev, name) + _PACK_CONV_PARAMS(
             _packed(get("dweight"), (C, W), _F32, dev, name),
             _packed(get("dbias"), (C,), _F32, dev, name),
             _packed(get("dstate"), (b, W - 1, C), _F32, dev, name)),
         *_workspace(workspace, dev, name), flags)


def _sel_inputs(dims, lead, x, dt, A, B, C, D, z, dt_bias, seqlens, dev, name):
    """The call's dims and m3_sel_inputs, packed; lead is (b, T) or (b,)."""
    io, b, ch, G, N = _io_type(dims, name), dims.batch, dims.channels, dims.ngroups, dims.dstate
    wide, gn = (*lead, ch), (*lead, G, N)
    return _PACK_SEL_DIMS(b, ch, G, N, dims.io_dtype), (
        _rows(x, wide, io, dev, name) + _rows(dt, wide, io, dev, name)
        + _group_rows(B, gn, io, dev, name) + _group_rows(C, gn, io, dev, name)
        + _rows(z, wide, io, dev, name) + _PACK_POINTERS(
            _packed(A, (ch, N), _F32, dev, name), _packed(D, (ch,), _F32, dev, name),
            _packed(dt_bias, (ch,), _F32, dev, name),
            _packed(seqlens, (b,), torch.int32, dev, name)))


def m3_sel_workspace_bytes(dims: SelDims, seqlen: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().m3_sel_workspace_bytes(ctypes.byref(dims.c()), int(seqlen),
                                                 ctypes.byref(n)), "m3_sel_workspace_bytes")
    return n.value


def alloc_sel_workspace(dims: SelDims, seqlen: int, device="cuda") -> torch.Tensor:
    return torch.empty(m3_sel_workspace_bytes(dims, seqlen), dtype=torch.uint8, device=device)


def m3_sel_fwd(dims: SelDims, seqlen: int, x, dt, A, B, C, D, z, dt_bias, h, y, workspace,
               seqlens=None, flags: int = 0, stream=None):
    """Selective scan of x [b, T, D] into y, carrying h [b, D, N] fp32 (updated in place).
    dt, z like x; B, C [b, T, G, N]; A [D, N] fp32; D, dt_bias [D] fp32.  D, z, dt_bias, seqlens
    (int32 [b]) and workspace may be None; flags: M3_FLAG_DT_SOFTPLUS."""
    name, b, ch = "m3_sel_fwd", dims.batch, dims.channels
    dev, lead = _device(x, name), (b, seqlen)
    packed = _sel_inputs(dims, lead, x, dt, A, B, C, D, z, dt_bias, seqlens, dev, name)
    _run(name, dev, stream, packed[0], seqlen, packed[1],
         _packed(h, (b, ch, dims.dstate), _F32, dev, name),
         _rows(y, (b, seqlen, ch), _TYPE_OF[dims.io_dtype], dev, name),
         *_workspace(workspace, dev, name), flags)


def m3_sel_step(dims: SelDims, x, dt, A, B, C, D, z, dt_bias, h, y, flags: int = 0, stream=None):
    """One token of every sequence: x, dt, z, y [b, D]; B, C [b, G, N]."""
    name, b, ch = "m3_sel_step", dims.batch, dims.channels
    dev = _device(x, name)
    packed = _sel_inputs(dims, (b,), x, dt, A, B, C, D, z, dt_bias, None, dev, name)
    _run(name, dev, stream, *packed, _packed(h, (b, ch, dims.dstate), _F32, dev, name),
         _rows(y, (b, ch), _TYPE_OF[dims.io_dtype], dev, name), flags)


def m3_sel_bwd_workspace_bytes(dims: SelDims, seqlen: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().m3_sel_bwd_workspace_bytes(ctypes.byref(dims.c()), int(seqlen),
                                                     ctypes.byref(n)),
           "m3_sel_bwd_workspace_bytes")
    return n.value


def alloc_sel_bwd_workspace(dims: SelDims, seqlen: int, device="cuda") -> torch.Tensor:
    return torch.empty(m3_sel_bwd_workspace_bytes(dims, seqlen), dtype=torch.uint8, device=device)


def alloc_sel_grads(dims: SelDims, seqlen: int, gate: bool = True, device="cuda") -> dict:
    """Gradient tensors of m3_sel_bwd (dz with the gate alone)."""
    b, T, D, G, N = dims.batch, seqlen, dims.channels, dims.ngroups, dims.dstate
    io = dict(dtype=torch_dtype_of(dims.io_dtype), device=device)
    f = dict(dtype=_F32, device=device)
    out = dict(dx=torch.empty(b, T, D, **io), ddt=torch.empty(b, T, D, **io),
               dB=torch.empty(b, T, G, N, **io), dC=torch.empty(b, T, G, N, **io),
               dA=torch.empty(D, N, **f), dD=torch.empty(D, **f), ddt_bias=torch.empty(D, **f),
               dh=torch.empty(b, D, N, **f))
    if gate:
        out["dz"] = torch.empty(b, T, D, **io)
    return out


def m3_sel_bwd(dims: SelDims, seqlen: int, x, dt, A, B, C, D, z, dt_bias, h0, dy, dhT,
               grads: dict, workspace, seqlens=None, flags: int = 0, stream=None):
    """Backward of m3_sel_fwd into ``grads`` (see alloc_sel_grads; dh may be absent); ``h0`` is
    the state that the forward call started from, ``dhT`` [b, D, N] fp32 may be None."""
    name, b, ch, G, N = "m3_sel_bwd", dims.batch, dims.channels, dims.ngroups, dims.dstate
    dev, lead, get = _device(x, name), (b, seqlen), grads.get
    packed = _sel_inputs(dims, lead, x, dt, A, B, C, D, z, dt_bias, seqlens, dev, name)
    io, wide, gn, hs = _TYPE_OF[dims.io_dtype], (b, seqlen, ch), (b, seqlen, G, N), (b, ch, N)
    _run(name, dev, stream, packed[0], seqlen, packed[1], _packed(h0, hs, _F32, dev, name),
         _rows(dy, wide, io, dev, name), _packed(dhT, hs, _F32, dev, name),
         _rows(get("dx"), wide, io, dev, name) + _rows(get("ddt"), wide, io, dev, name)
         + _group_rows(get("dB"), gn, io, dev, name) + _group_rows(get("dC"), gn, io, dev, name)
         + _rows(get("dz"), wide, io, dev, name) + _PACK_POINTERS(
             _packed(get("dA"), (ch, N), _F32, dev, name), _packed(get("dD"), (ch,), _F32, dev, name),
             _packed(get("ddt_bias"), (ch,), _F32, dev, name),
             _packed(get("dh"), hs, _F32, dev, name)),
         *_workspace(workspace, dev, name), flags)


def _norm_types(dims, name):
    if dims.io_dtype not in _TYPE_OF or dims.res_dtype not in _TYPE_OF:
        raise M3Error(M3_ERR_DTYPE, name)
    return (_TYPE_OF[dims.io_dtype],), (_TYPE_OF[dims.res_dtype],)


def alloc_norm_scales(dims: NormDims, device="cuda") -> torch.Tensor:
    """The scales of an e4m3 output: one for each 128 values of a row."""
    return torch.empty(dims.rows, (dims.width + 127) // 128, dtype=_F32, device=device)


def m3_norm_fwd(dims: NormDims, x, residual, weight, eps: float, y, scales=None,
                residual_out=None, stream=None):
    """r = x + residual (kept in ``residual_out``), y = r / rms(r) * weight.  With M3_OUT_E4M3, y
    is float8_e4m3fn (or uint8) and ``scales`` [rows, ceil(width / 128)] fp32.  residual, weight
    and residual_out may be None."""
    name, rows, width = "m3_norm_fwd", dims.rows, dims.width
    io, res = _norm_types(dims, name)
    dev, shape = _device(x, name), (rows, width)
    e4m3 = dims.out == M3_OUT_E4M3
    _run(name, dev, stream,
         _PACK_NORM_DIMS(rows, width, dims.io_dtype, dims.res_dtype, dims.out),
         *_matrix(x, shape, io, dev, name), *_matrix(residual, shape, res, dev, name),
         _packed(weight, (width,), _F32, dev, name), eps,
         *_matrix(y, shape, _E4M3 if e4m3 else io, dev, name),
         _packed(scales, (rows, (width + 127) // 128), _F32, dev, name),
         *_matrix(residual_out, shape, res, dev, name))


def m3_norm_bwd_workspace_bytes(dims: NormDims) -> int:
    n = ctypes.c_size_t()
    _check(load_library().m3_norm_bwd_workspace_bytes(ctypes.byref(dims.c()), ctypes.byref(n)),
           "m3_norm_bwd_workspace_bytes")
    return n.value


def alloc_norm_bwd_workspace(dims: NormDims, device="cuda") -> torch.Tensor:
    return torch.empty(m3_norm_bwd_workspace_bytes(dims), dtype=torch.uint8, device=device)


def m3_norm_bwd(dims: NormDims, r, weight, eps: float, dy, dres, dx, dresidual, dweight, workspace,
                stream=None):
    """Backward of m3_norm_fwd: ``r`` is its residual_out (x without a residual), ``dres`` the
    gradient of residual_out or None.  dr goes to ``dx`` in the io type and to ``dresidual``
    (None: not wanted) in the residual's."""
    name, rows, width = "m3_norm_bwd", dims.rows, dims.width
    io, res = _norm_types(dims, name)
    dev, shape = _device(dy, name), (rows, width)
    _run(name, dev, stream,
         _PACK_NORM_DIMS(rows, width, dims.io_dtype, dims.res_dtype, dims.out),
         *_matrix(r, shape, res, dev, name), _packed(weight, (width,), _F32, dev, name), eps,
         *_matrix(dy, shape, io, dev, name), *_matrix(dres, shape, res, dev, name),
         *_matrix(dx, shape, io, dev, name), *_matrix(dresidual, shape, res, dev, name),
         _packed(dweight, (width,), _F32, dev, name), *_workspace(workspace, dev, name))
