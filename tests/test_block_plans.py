"""The block operators under the plans that large calls get: segments of several tiles in the
selective scan, long runs in the convolution, many turns of a block in the norm's backward.  Many
short sequences (or rows) reach them at sizes that a 64-bit reference can follow.  The plans are
restated here and held against the library's workspace sizes, so that no case can fall back to a
simpler plan unnoticed."""
import pytest
import torch

import block_reference as ref
import test_block_gpu as tb
from block_reference import U32, f64, half_step
from state_space_model_06_b200 import m3

BF, F32 = torch.bfloat16, torch.float32


def round256(n):
    return -(-n // 256) * 256


def ends(b, T, marks):
    """Lengths that end at every mark in turn, among them 0, 1 and beyond both sides."""
    marks = [T, 0, 1, T + 9, -3] + list(marks)
    return torch.tensor([marks[i % len(marks)] for i in range(b)], dtype=torch.int32).cuda()


def lay(t, wide):
    """The same values in rows that start on 16 bytes, or off them."""
    if wide:
        return t.contiguous()
    out = torch.empty(*t.shape[:2], t[0, 0].numel() + 1, dtype=t.dtype, device=t.device)
    out = out[..., 1:].unflatten(-1, t.shape[2:]) if t.dim() > 3 else out[..., 1:]
    return out.copy_(t)


def cells(b, T, ch, G, N, io, marks, wide, seed):
    """Inputs of a scan, with NaN behind the lengths, and the same in 64 bits with zeros there."""
    c, _, _ = tb.scan_inputs((b, T, ch, G, N, io, "z D bias softplus"), seed)
    for k in ("x", "dt", "B", "C", "z"):
        c[k] = lay(c[k], wide)
    sl = ends(b, T, marks)
    past = torch.arange(T).cuda()[None] >= sl[:, None]
    for k in ("x", "dt", "B", "C", "z"):
        c[k].masked_fill_(past.view(b, T, *[1] * (c[k].dim() - 2)), float("nan"))
    r = {k: f64(v) for k, v in c.items()}
    for k in ("x", "dt", "B", "C", "z"):
        r[k].nan_to_num_(nan=0.0)
    return c, r, sl


# ---------------------------------------------------------------- scan, backward

# states: tokens of a tile, channels of a block, padded states
BWD_SHAPE = {4: (32, 64, 4), 8: (32, 64, 8), 16: (32, 64, 16), 24: (32, 32, 32), 40: (32, 16, 64),
             72: (16, 16, 128), 200: (16, 8, 256)}


def bwd_plan(b, T, ch, G, N, m=None):
    """Tiles of a segment (or m of them), segments, and the workspace's bytes."""
    tile, CB, NP = BWD_SHAPE[N]
    blocks, ntile = -(-(ch // G) // CB) * G, -(-T // tile)
    if m is None:
        m = 4
        while m > 1 and blocks * b * -(-ntile // m) < 148 * 12:
            m //= 2
    nseg, states = -(-ntile // m), ch * N
    sizes = [b * ntile * states, b * ntile * ch] + [b * nseg * states] * 3 + \
        [b * nseg * 2 * ch, b * T * blocks * 2 * NP]
    return m, nseg, sum(round256(4 * n) for n in sizes)


def bwd_serves(b, T, ch, G, N):
    """The size that serves every length up to T: that of T itself, or of the longest with fewer
    tiles a segment."""
    tile = BWD_SHAPE[N][0]
    longest = {}
    for n in range(1, -(-T // tile) + 1):
        longest[bwd_plan(b, n * tile, ch, G, N)[0]] = min(n * tile, T)
    return max(bwd_plan(b, t, ch, G, N)[2] for t in longest.values())


SCAN_BWD = [  # b, tiles' worth of tokens and a few more, ch, G, N, io, wide rows, tiles a segment
    (890, 4, 8, 1, 4, BF, True, 4),
    (600, 4, 5, 1, 4, F32, False, 2),
    (890, 4, 4, 1, 8, F32, True, 4),
    (600, 4, 8, 1, 8, BF, True, 2),
    (890, 4, 8, 1, 16, BF, True, 4),
    (890, 4, 7, 1, 16, BF, False, 4),
    (600, 4, 4, 1, 16, F32, True, 2),
    (450, 4, 6, 2, 16, F32, False, 4),
    (450, 6, 16, 2, 16, BF, True, 4),       # segments of 4 and 3 tiles
    (890, 4, 4, 1, 24, F32, True, 4),
    (600, 4, 8, 1, 24, BF, True, 2),
    (890, 4, 3, 1, 40, BF, False, 4),
    (600, 4, 4, 1, 40, F32, True, 2),
    (890, 4, 8, 1, 72, BF, True, 4),
    (600, 4, 3, 1, 72, F32, False, 2),
    (890, 4, 4, 1, 200, F32, True, 4),
    (600, 4, 5, 1, 200, BF, False, 2),
]


def bwd_tokens(case):
    b, tiles, ch, G, N, io, wide, m = case
    return BWD_SHAPE[N][0] * tiles + 5


@pytest.mark.parametrize("case", SCAN_BWD)
def test_scan_bwd_plan(case):
    """The case gets the segments that it is listed for, by the library's own workspace size."""
    b, _, ch, G, N, io, _, want = case
    T = bwd_tokens(case)
    m, nseg, size = bwd_plan(b, T, ch, G, N)
    assert m == want and nseg >= 2
    d = m3.SelDims(b, ch, G, N, m3.io_dtype_of(io))
    assert m3.m3_sel_bwd_workspace_bytes(d, T) == bwd_serves(b, T, ch, G, N) >= size
    # no other number of tiles a segment would have this size: the call refuses less (here) and
    # takes as much (on the GPU)
    assert all(size != bwd_plan(b, T, ch, G, N, k)[2] for k in (1, 2, 4) if k != m)
    P, rows = 0x10000, lambda w: m3.m3_rows(0x10000, T * w, w)
    inputs = bytes(m3.m3_sel_inputs(*[rows(w) for w in (ch, ch, G * N, G * N, ch)], P, P, P, 0))
    grads = bytes(m3.m3_sel_grads(*[rows(w) for w in (ch, ch, G * N, G * N, ch)], P, P, P, P))
    assert m3.load_library().m3_sel_bwd(bytes(d.c()), T, inputs, P, bytes(rows(ch)), P, grads, P,
                                        size - 1, 0, None) == m3.M3_ERR_WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("case", SCAN_BWD)
def test_scan_bwd_over_several_tiles(case):
    """Segments of two and four tiles, the last one shorter, with lengths that end in each of
    them; and the same calls' outputs."""
    b, _, ch, G, N, io, wide, _ = case
    T, tile = bwd_tokens(case), BWD_SHAPE[N][0]
    m, nseg, size = bwd_plan(b, T, ch, G, N)
    marks = [k * tile + o for k in range(-(-T // tile)) for o in (0, 1, 7, tile - 1)]
    c, r, sl = cells(b, T, ch, G, N, io, [v for v in marks if 1 < v < T], wide, 31)
    g = torch.Generator().manual_seed(32)
    dy, dhT = tb.rnd(g, b, T, ch, dtype=io), tb.rnd(g, b, ch, N)
    rdy = f64(dy)
    past = torch.arange(T)[None] >= sl.cpu()[:, None]
    dy.masked_fill_(past.cuda()[..., None], float("inf"))
    rdy.masked_fill_(past[..., None], 0.0)
    dy = lay(dy, wide)
    lens = ref.lengths(sl, b, T)
    want = ref.scan_bwd(*r.values(), lens, True, rdy, f64(dhT))
    mag = ref.scan_bwd(*r.values(), lens, True, rdy, f64(dhT), absolute=True)
    rel = 2 * ref.scan_bounds(T, N, ch, r["A"], r["dt"], r["bias"], True) + 2.0 ** -19
    # roundings in a row of a parameter's sum: a segment's tokens, a warp's share of the segments
    # (eight warps at least), the lanes and the warps
    rows = m * tile + b * nseg / 8 + 5 + 32
    d = m3.SelDims(b, ch, G, N, m3.io_dtype_of(io))
    gr = {k: tb.nan_like(v) for k, v in m3.alloc_sel_grads(d, T).items()}
    if not wide:
        for k in ("dx", "ddt", "dz"):
            gr[k] = lay(gr[k], False)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    m3.m3_sel_bwd(d, T, c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["bias"],
                  c["h"], dy, dhT, gr, ws, seqlens=sl, flags=m3.M3_FLAG_DT_SOFTPLUS)
    for k, v in gr.items():
        sums = U32 * (ch if k in ("dB", "dC") else rows if k in ("dA", "dD", "ddt_bias") else 0)
        tol = (rel + sums) * mag[k] + 1e-37
        if k in ("dx", "ddt", "dB", "dC", "dz"):
            tol = tol + half_step(io) * want[k].abs()
        tb.near(v, want[k], tol, k)


# ---------------------------------------------------------------- scan, segmented prompts

# states: channels of a block in one piece, and in segments
FWD_SHAPE = {4: (64, 64), 8: (64, 64), 16: (32, 64), 24: (32, 32), 40: (32, 32), 72: (16, 16),
             200: (16, 16)}


def fwd_plan(b, T, ch, G, N):
    """Tiles (of 32 tokens) of a segment, segments, and the bytes that serve every length up to
    T."""
    one, many = (b * G * -(-(ch // G) // CB) for CB in FWD_SHAPE[N])
    tiles = -(-T // 32)
    n = min(148 * 14 // many, tiles) if one <= 148 * 3 and tiles > 4 else 1
    per = -(-tiles // n)
    return per, -(-tiles // per), round256(4 * b * n * ch * (N + 1)) if n > 1 else 256


SCAN_FWD = [  # b, T, ch, G, N, io, wide rows
    (400, 349, 8, 1, 4, BF, True),          # segments of 3, 3, 3 and 2 tiles
    (400, 349, 4, 1, 8, F32, True),
    (400, 349, 8, 1, 16, BF, True),
    (400, 349, 3, 1, 16, F32, False),
    (100, 352, 4, 4, 24, F32, False),       # four groups of one channel
    (50, 330, 64, 8, 24, BF, True),
    (100, 349, 4, 4, 40, BF, False),
    (100, 349, 16, 4, 72, F32, True),
    (100, 349, 4, 4, 200, BF, False),
]


@pytest.mark.parametrize("case", SCAN_FWD)
def test_scan_fwd_plan(case):
    b, T, ch, G, N, io, _ = case
    per, n, size = fwd_plan(b, T, ch, G, N)
    assert per >= 2 and n >= 2
    assert m3.m3_sel_workspace_bytes(m3.SelDims(b, ch, G, N, m3.io_dtype_of(io)), T) == size


@pytest.mark.gpu
@pytest.mark.parametrize("case", SCAN_FWD)
def test_scan_fwd_over_several_tiles(case):
    """Segments of several tiles, with lengths that end in each tile of one and at its edges."""
    b, T, ch, G, N, io, wide = case
    per, n, size = fwd_plan(b, T, ch, G, N)
    marks = [k * 32 + o for k in range(-(-T // 32)) for o in (0, 1, 13)]
    c, r, sl = cells(b, T, ch, G, N, io, [v for v in marks if 1 < v < T], wide, 33)
    lens = ref.lengths(sl, b, T)
    want_y, want_h = ref.scan(*r.values(), lens, True)
    mag_y, mag_h = ref.scan(*r.values(), lens, True, absolute=True)
    rel = ref.scan_bounds(T, N, ch, r["A"], r["dt"], r["bias"], True)
    d = m3.SelDims(b, ch, G, N, m3.io_dtype_of(io))
    y, h = lay(tb.nan_like(c["x"]), wide), c["h"].clone()
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    m3.m3_sel_fwd(d, T, c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["bias"], h, y,
                  ws, seqlens=sl, flags=m3.M3_FLAG_DT_SOFTPLUS)
    tb.near(h, want_h, rel * mag_h + 1e-37, "h")
    tb.near(y, want_y, half_step(io) * want_y.abs() + (rel + 2.0 ** -20) * mag_y + 1e-37, "y")


# ---------------------------------------------------------------- convolution

def conv_run(b, T, C, slots):
    """Tokens of a run: the least time in whole rounds of blocks."""
    cost = lambda s: -(-(b * -(-C // 512) * -(-T // s)) // slots) * (s + 8)
    return min(range(8, 129, 8), key=cost)


CONV = [  # b, T, C, W, io, options: wide rows with C a multiple of 16 bytes, else narrow ones
    (290, 230, 64, 4, BF, "silu bias"),
    (290, 230, 20, 4, F32, "silu bias"),
    (290, 230, 21, 4, BF, "silu bias"),
    (290, 230, 12, 3, F32, "bias"),
    (290, 231, 16, 8, BF, "silu"),
    (290, 233, 8, 8, F32, "silu bias"),
    (290, 229, 9, 2, F32, "silu bias odd"),
    (290, 232, 8, 1, BF, "silu bias"),
]


@pytest.mark.parametrize("case", CONV)
def test_conv_plan(case):
    """Runs of several turns of the ring, forward (four groups of four tokens) and backward."""
    b, T, C, W, io, _ = case
    assert conv_run(b, T, C, 148 * 7) >= 48
    s = conv_run(b, T, C, 148 * 4)
    assert s >= 48
    # these fit one round of blocks, where the size that serves every length is that of the runs
    assert b * -(-T // s) <= 148 * 4 and 148 * 4 // b == -(-T // s)
    assert m3.m3_conv_bwd_workspace_bytes(m3.ConvDims(b, C, W, m3.io_dtype_of(io)), T) == \
        round256(4 * b * -(-T // s) * (W + 1) * C)


def conv_lengths(b, T):
    """Ends before, at and behind the ring's turns and the groups of four."""
    return ends(b, T, [2, 3, 4, 5, 11, 15, 16, 17, 18, 19, 47, 55, 56, 57, 63, 64, 71, 72, 73, 74,
                       75, 76, 79, 100, 112, 144, 145, 168, 190, 200, T - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("case", CONV)
def test_conv_fwd_long_runs(case):
    b, T, C, W, io, _ = case
    x, w, bias, state, _, act = tb.conv_inputs(case, 41)
    sl = conv_lengths(b, T)
    x.masked_fill_((torch.arange(T).cuda()[None] >= sl[:, None])[..., None], float("nan"))
    lens = ref.lengths(sl, b, T)
    y, new = ref.conv(*(f64(v) for v in (x, w, bias, state)), lens, act)
    tol = tb.conv_tol(case, (x, w, bias, state), lens, act, y)
    out = tb.nan_like(torch.empty(b, T, C, dtype=io, device="cuda"))
    m3.m3_conv_fwd(m3.ConvDims(b, C, W, m3.io_dtype_of(io)), T, x, w, bias, state, out, seqlens=sl,
                   flags=m3.M3_FLAG_SILU if act else 0)
    tb.near(out, y, tol, "y")
    assert torch.equal(f64(state), new)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CONV)
def test_conv_bwd_long_runs(case):
    b, T, C, W, io, _ = case
    x, w, bias, state, _, act = tb.conv_inputs(case, 42)
    dy = tb.rnd(torch.Generator().manual_seed(43), b, T, C, dtype=io)
    sl = conv_lengths(b, T)
    past = (torch.arange(T).cuda()[None] >= sl[:, None])[..., None]
    x.masked_fill_(past, float("nan"))
    dy.masked_fill_(past, float("inf"))
    lens = ref.lengths(sl, b, T)
    args = [f64(v) for v in (x, w, bias, state)]
    want = ref.conv_bwd(*args, lens, act, f64(dy))
    mag = ref.conv_bwd(*args, lens, act, f64(dy), absolute=True)
    d = m3.ConvDims(b, C, W, m3.io_dtype_of(io))
    gr = {k: tb.nan_like(v) for k, v in m3.alloc_conv_grads(d, T).items()}
    m3.m3_conv_bwd(d, T, x, w, bias, state, dy, gr, m3.alloc_conv_bwd_workspace(d, T), seqlens=sl,
                   flags=m3.M3_FLAG_SILU if act else 0)
    # the activation's slope moves with pre's error: |act''| <= 1/2 on (W + 3) U32 |terms|
    pre = args[1].abs().sum(1).max() * max(float(args[0].nan_to_num().abs().max()),
                                           float(args[3].abs().max()) if args[3].numel() else 0.0)
    pre = float(pre) + (0.0 if bias is None else float(args[2].abs().max()))
    rel = (W + 6) * U32 + (2.0 ** -19 + 0.5 * (W + 3) * U32 * pre * 8 if act else 0)
    s = conv_run(b, T, C, 148 * 4)
    for k in ("dx", "dweight", "dbias", "dstate"):
        if k == "dbias" and bias is None:
            continue
        tol = rel * mag[k] + 1e-37
        if k == "dx":
            tol = tol + half_step(io) * want[k].abs()
        elif k != "dstate":      # a run's tokens, a warp's share of the runs, the warps
            tol = tol + (s + b * -(-T // s) / 8 + 32) * U32 * mag[k]
        tb.near(gr[k], want[k], tol, k)


# ---------------------------------------------------------------- one workspace for several lengths

def sizes(f, lengths):
    out = [f(T) for T in lengths]
    assert out == sorted(out)
    return dict(zip(lengths, out))


@pytest.mark.parametrize("b,ch,N", [(1, 2048, 16), (4, 4096, 16), (8, 1024, 24), (2, 64, 40),
                                    (300, 4, 4), (37, 100, 200)])
def test_a_workspace_serves_shorter_calls(b, ch, N):
    """The size for a length is enough for every shorter one."""
    d = m3.SelDims(b, ch, 1, N)
    have = sizes(lambda T: m3.m3_sel_bwd_workspace_bytes(d, T), range(16, 6000, 16))
    for T in range(16, 6000, 112):
        assert have[T] == bwd_serves(b, T, ch, 1, N)
    sizes(lambda T: m3.m3_sel_workspace_bytes(d, T), range(0, 20000, 32))
    for W, io in ((4, m3.M3_BF16), (7, m3.M3_F32)):
        d = m3.ConvDims(b, ch, W, io)
        have, most = sizes(lambda T: m3.m3_conv_bwd_workspace_bytes(d, T), range(8, 20000, 8)), 0
        for T in have:
            most = max(most, -(-T // conv_run(b, T, ch, 148 * 4)))
            assert have[T] == max(round256(4 * b * most * (W + 1) * ch), 256)
        assert m3.m3_conv_bwd_workspace_bytes(d, 0) == 256


@pytest.mark.gpu
def test_conv_bwd_in_a_longer_calls_workspace():
    b, C, W, T = 2, 64, 4, 2368              # one run more than half of 2376's would need
    case = (b, T, C, W, F32, "silu bias")
    x, w, bias, state, _, _ = tb.conv_inputs(case, 44)
    dy = tb.rnd(torch.Generator().manual_seed(45), b, T, C)
    d = m3.ConvDims(b, C, W, m3.M3_F32)
    assert conv_run(b, T, C, 148 * 4) < conv_run(b, T + 8, C, 148 * 4)
    out = []
    for n in (T, T + 8):
        gr = {k: tb.nan_like(v) for k, v in m3.alloc_conv_grads(d, T).items()}
        m3.m3_conv_bwd(d, T, x, w, bias, state, dy, gr, m3.alloc_conv_bwd_workspace(d, n),
                       flags=m3.M3_FLAG_SILU)
        out.append(gr)
    for k in out[0]:
        assert torch.equal(out[0][k], out[1][k]), k


@pytest.mark.gpu
def test_scan_in_a_longer_calls_workspace():
    """Forward in as many segments as with a workspace of its own (the same bits), backward."""
    for b, T, longer, ch, G, call in ((100, 160, 192, 4, 4, "fwd"), (300, 320, 352, 64, 1, "bwd")):
        c, _, sp = tb.scan_inputs((b, T, ch, G, 4, F32, "z D bias softplus"), 46)
        d = m3.SelDims(b, ch, G, 4, m3.M3_F32)
        short, long = (fwd_plan(b, n, ch, G, 4)[1] if call == "fwd" else bwd_plan(b, n, ch, G, 4)[2]
                       for n in (T, longer))
        assert short > long
        out = []
        for n in (T, longer):
            h = c["h"].clone()
            args = [c[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "bias")]
            if call == "fwd":
                y = tb.nan_like(c["x"])
                m3.m3_sel_fwd(d, T, *args, h, y, m3.alloc_sel_workspace(d, n),
                              flags=m3.M3_FLAG_DT_SOFTPLUS)
                out.append(dict(y=y, h=h))
            else:
                gr = {k: tb.nan_like(v) for k, v in m3.alloc_sel_grads(d, T).items()}
                m3.m3_sel_bwd(d, T, *args, h, c["x"], None, gr, m3.alloc_sel_bwd_workspace(d, n),
                              flags=m3.M3_FLAG_DT_SOFTPLUS)
                out.append(gr)
        for k in out[0]:
            assert torch.equal(out[0][k], out[1][k]), (call, k)


# ---------------------------------------------------------------- norm, backward

NORM_BWD = [  # rows, width, io, residual, options: threads a row 32 to 1024, two and four vectors
    (6001, 250, BF, F32, "w"),
    (5001, 500, F32, F32, "w"),
    (2501, 1000, BF, BF, "w"),
    (1300, 2048, BF, F32, "w"),
    (800, 4096, F32, BF, "w strided"),
    (400, 8192, BF, F32, "w"),
    (400, 16384, BF, BF, "w"),
    (310, 16390, F32, F32, "w"),
    (310, 32768, BF, F32, "w"),
]


def norm_blocks(rows, width):
    t = 32
    while t < 1024 and t * 8 < width:
        t *= 2
    groups = -(-rows // max(128 // t, 1))
    return groups, min(groups, 148 * (1024 // max(t, 128)))


@pytest.mark.parametrize("case", NORM_BWD)
def test_norm_bwd_plan(case):
    """Every block takes two turns or more, and some one more than others."""
    rows, width, io, res, _ = case
    groups, blocks = norm_blocks(rows, width)
    # rows that share a block's turn are the spare ones' case too
    assert groups > blocks and groups % blocks
    d = m3.NormDims(rows, width, m3.io_dtype_of(io), m3.io_dtype_of(res))
    assert m3.m3_norm_bwd_workspace_bytes(d) == round256(4 * blocks * width)


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("case", NORM_BWD)
def test_norm_bwd_many_turns(case, inplace):
    tb.test_norm_bwd(case, inplace)
