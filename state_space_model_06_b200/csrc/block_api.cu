// block_api.cu -- C ABI of the block operators (m3_conv_*, m3_sel_*, m3_norm_*): host-side
// validation and dispatch.  Everything is checked before anything is launched.
#include <cmath>
#include <cstring>

#include "block_internal.h"

using namespace m3;

namespace {

bool at_least(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t esize(int io) { return io == M3_BF16 ? 2 : 4; }
bool io_known(int io) { return io == M3_F32 || io == M3_BF16; }

m3_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return M3_OK;
    return e == cudaErrorNotSupported ? M3_ERR_UNSUPPORTED : M3_ERR_LAUNCH;
}

// Geometry of one call's rows.  step: one token a sequence (token strides unused).
struct Geo {
    int64_t batch, T;
    size_t e;
    bool step;
};

m3_status check_in(const m3_rows& r, const Geo& g) {
    if (!r.ptr) return M3_ERR_NULL;
    if (!at_least(r.ptr, g.e)) return M3_ERR_ALIGN;
    if (r.batch_stride < 0 || (!g.step && r.token_stride < 0)) return M3_ERR_SHAPE;
    return M3_OK;
}

// Output rows must not overlap: one of the two axes lies inside the other.
m3_status check_out(const m3_rows& r, const Geo& g, int64_t width) {
    m3_status st = check_in(r, g);
    if (st != M3_OK) return st;
    const int64_t T = g.step ? 1 : g.T, bs = r.batch_stride, ts = r.token_stride;
    if (T > 1 && ts < width) return M3_ERR_SHAPE;
    if (g.batch > 1 && bs < width) return M3_ERR_SHAPE;
    if (T > 1 && g.batch > 1) {
        // span / stride compared by division: no product of strides and counts can overflow
        const bool tokens_inside = (bs - width) / ts >= T - 1;
        const bool batch_inside = (ts - width) / bs >= g.batch - 1;
        if (!tokens_inside && !batch_inside) return M3_ERR_SHAPE;
    }
    return M3_OK;
}

// Whether every row starts on 16 bytes.
bool wide_rows(const m3_rows& r, const Geo& g) {
    const int64_t per = 16 / (int64_t)g.e;
    return at_least(r.ptr, 16) && (g.batch == 1 || r.batch_stride % per == 0) &&
           (g.step || g.T == 1 || r.token_stride % per == 0);
}

View view(const m3_rows& r) { return View{r.ptr, r.batch_stride, r.token_stride}; }
template <typename O>
void set_out(O& o, const m3_rows& r) {
    o.p = r.ptr;
    o.bs = r.batch_stride;
    o.ts = r.token_stride;
}

constexpr int64_t kMaxBlocks = 2147483647;   // a one-dimensional grid
constexpr int32_t kMaxTokens = 1 << 30;      // token numbers and a run more stay in 32 bits

// ------------------------------------------------------------------ convolution

m3_status conv_dims_ok(const m3_conv_dims* d) {
    if (!d) return M3_ERR_NULL;
    if (!io_known(d->io_dtype)) return M3_ERR_DTYPE;
    if (d->batch < 1 || d->channels < 1 || d->width < 1) return M3_ERR_SHAPE;
    if (d->width > 8 || d->channels > 1 << 24) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

// Tokens of a run.  A block's time is about its tokens and eight more (the filter, and the W - 1
// tokens read again at its start), and `slots` blocks run at a time: of 8, 16, .. 128 tokens the
// run that takes the least time in whole rounds of blocks.  At least 8, so that only the first run
// reaches back into the state.
int64_t conv_columns(const m3_conv_dims* d) { return (int64_t)d->batch * ((d->channels + 511) / 512); }
int64_t conv_cost(int64_t columns, int64_t T, int s, int slots) {
    return (columns * ((T + s - 1) / s) + slots - 1) / slots * (s + 8);
}
void conv_runs(const m3_conv_dims* d, int32_t T, int slots, int* seg, int* nseg) {
    const int64_t columns = conv_columns(d);
    int64_t best = 0;
    for (int s = 8; s <= 128; s += 8) {
        const int64_t cost = conv_cost(columns, T, s, slots);
        if (s == 8 || cost < best) {
            best = cost;
            *seg = s;
            *nseg = (int)(((int64_t)T + s - 1) / s);
        }
    }
}
// Blocks that the GPU holds in bf16 with up to four taps.  fp32 holds six an SM forward (32 KiB of
// shared memory each), and more taps four forward and two backward: their rounds are longer than
// they are counted here.
constexpr int kConvFwdSlots = 148 * 7, kConvBwdSlots = 148 * 4;

// Bytes of the shares of `nseg` runs a sequence.
size_t conv_bytes(const m3_conv_dims* d, int64_t nseg) {
    const size_t n = sizeof(float) * (size_t)d->batch * nseg * (d->width + 1) * d->channels;
    return n < 256 ? 256 : (n + 255) / 256 * 256;
}
// The most runs of any length up to T (the choice above goes up and down with T).  Runs of s tokens
// make n of them where they are chosen at the longest such length, min(n s, T): the other choices
// cost the most there.  They cannot be chosen where s + 8 for each s tokens cost more than runs of
// 128 in their whole rounds: beyond 136 (1 + slots / columns) / (8 / s - 8 / 128) tokens.
int64_t conv_most_runs(const m3_conv_dims* d, int32_t T, int slots) {
    const int64_t columns = conv_columns(d);
    auto chosen = [&](int s, int64_t t) {
        const int64_t cost = conv_cost(columns, t, s, slots);
        for (int k = 8; k <= 120; k += 8) {      // the nearest first: they cost least
            if (s + k <= 128 && conv_cost(columns, t, s + k, slots) < cost) return false;
            if (s - k >= 8 && conv_cost(columns, t, s - k, slots) <= cost) return false;
        }
        return true;
    };
    int64_t best = ((int64_t)T + 127) / 128;
    for (int s = 8; s < 128; s += 8) {
        const double end = 136. * (1. + slots / (double)columns) / (8. / s - 0.0625) + s;
        int64_t n = ((end < T ? (int64_t)end : T) + s - 1) / s;
        while (n > best) {
            if (chosen(s, n * s < T ? n * s : T))
                best = n;
            else      // nor are fewer runs of as many rounds, for which the others cost no more
                n = ((columns * n + slots - 1) / slots - 1) * slots / columns;
        }
    }
    return best;
}

m3_status conv_common(const m3_conv_dims* d, const Geo& g, const m3_rows* x, const float* weight,
                      const float* bias, const int32_t* seqlens, const void* state, uint32_t flags) {
    if (flags & ~M3_FLAG_SILU) return M3_ERR_UNSUPPORTED;
    if (!x || !weight || (d->width > 1 && !state)) return M3_ERR_NULL;
    m3_status st = check_in(*x, g);
    if (st != M3_OK) return st;
    if (!at_least(weight, 4) || (bias && !at_least(bias, 4)) || (seqlens && !at_least(seqlens, 4)) ||
        !at_least(state, g.e))
        return M3_ERR_ALIGN;
    return M3_OK;
}

void conv_args(ConvArgs* a, const m3_conv_dims* d, int32_t T, const m3_rows* x, const float* weight,
               const float* bias, const int32_t* seqlens, const void* state, uint32_t flags) {
    std::memset(a, 0, sizeof(*a));
    a->x = view(*x);
    a->weight = weight;
    a->bias = bias;
    a->seqlens = seqlens;
    a->state = const_cast<void*>(state);
    a->batch = d->batch;
    a->T = T;
    a->C = d->channels;
    a->W = d->width;
    a->silu = flags & M3_FLAG_SILU;
}

// Four neighbouring channels are one access in every tensor.
bool conv_wide(const m3_conv_dims* d, const float* weight, const void* state) {
    return d->channels % (16 / (int)esize(d->io_dtype)) == 0 && at_least(state, 16) &&
           at_least(weight, 16);
}

}  // namespace

extern "C" {

m3_status m3_conv_fwd(const m3_conv_dims* d, int32_t T, const m3_rows* x, const float* weight,
                      const float* bias, const int32_t* seqlens, void* state, const m3_rows* y,
                      uint32_t flags, void* stream) {
    m3_status st = conv_dims_ok(d);
    if (st != M3_OK) return st;
    if (T < 0) return M3_ERR_SHAPE;
    if (T > kMaxTokens) return M3_ERR_UNSUPPORTED;
    if (flags & ~M3_FLAG_SILU) return M3_ERR_UNSUPPORTED;
    if (T == 0) return M3_OK;
    const Geo g{d->batch, T, esize(d->io_dtype), false};
    if ((st = conv_common(d, g, x, weight, bias, seqlens, state, flags)) != M3_OK) return st;
    if (!y) return M3_ERR_NULL;
    if ((st = check_out(*y, g, d->channels)) != M3_OK) return st;
    if (y->ptr == x->ptr) return M3_ERR_UNSUPPORTED;      // a run reads tokens of the one before
    ConvArgs a;
    conv_args(&a, d, T, x, weight, bias, seqlens, state, flags);
    set_out(a.y, *y);
    conv_runs(d, T, kConvFwdSlots, &a.seg, &a.nseg);
    if ((int64_t)a.batch * a.nseg > kMaxBlocks) return M3_ERR_UNSUPPORTED;
    a.wide = conv_wide(d, weight, state) && wide_rows(*x, g) && wide_rows(*y, g);
    return status_of(launch_conv(a, ConvCall::fwd, d->io_dtype, static_cast<cudaStream_t>(stream)));
}

m3_status m3_conv_step(const m3_conv_dims* d, const m3_rows* x, const float* weight,
                       const float* bias, void* state, const m3_rows* y, uint32_t flags,
                       void* stream) {
    m3_status st = conv_dims_ok(d);
    if (st != M3_OK) return st;
    const Geo g{d->batch, 1, esize(d->io_dtype), true};
    if ((st = conv_common(d, g, x, weight, bias, nullptr, state, flags)) != M3_OK) return st;
    if (!y) return M3_ERR_NULL;
    if ((st = check_out(*y, g, d->channels)) != M3_OK) return st;
    if ((int64_t)d->batch * d->channels / 128 + 1 > kMaxBlocks) return M3_ERR_UNSUPPORTED;
    ConvArgs a;
    conv_args(&a, d, 1, x, weight, bias, nullptr, state, flags);
    set_out(a.y, *y);
    a.wide = conv_wide(d, weight, state) && wide_rows(*x, g) && wide_rows(*y, g);
    return status_of(launch_conv(a, ConvCall::step, d->io_dtype, static_cast<cudaStream_t>(stream)));
}

m3_status m3_conv_bwd_workspace_bytes(const m3_conv_dims* d, int32_t T, size_t* bytes) {
    m3_status st = conv_dims_ok(d);
    if (st != M3_OK) return st;
    if (!bytes) return M3_ERR_NULL;
    if (T < 0) return M3_ERR_SHAPE;
    if (T > kMaxTokens) return M3_ERR_UNSUPPORTED;
    *bytes = conv_bytes(d, conv_most_runs(d, T, kConvBwdSlots));
    return M3_OK;
}

m3_status m3_conv_bwd(const m3_conv_dims* d, int32_t T, const m3_rows* x, const float* weight,
                      const float* bias, const int32_t* seqlens, const void* state0,
                      const m3_rows* dy, const m3_conv_grads* gr, void* ws, size_t ws_bytes,
                      uint32_t flags, void* stream) {
    m3_status st = conv_dims_ok(d);
    if (st != M3_OK) return st;
    if (T < 0) return M3_ERR_SHAPE;
    if (T > kMaxTokens) return M3_ERR_UNSUPPORTED;
    if (flags & ~M3_FLAG_SILU) return M3_ERR_UNSUPPORTED;
    if (!gr || !gr->dweight || (bias && !gr->dbias)) return M3_ERR_NULL;
    if (!at_least(gr->dweight, 4) || (gr->dbias && !at_least(gr->dbias, 4)) ||
        (gr->dstate && !at_least(gr->dstate, 4)))
        return M3_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t C = d->channels, W = d->width;
    if (T == 0) {
        cudaError_t e = cudaMemsetAsync(gr->dweight, 0, C * W * sizeof(float), s);
        if (e == cudaSuccess && bias) e = cudaMemsetAsync(gr->dbias, 0, C * sizeof(float), s);
        if (e == cudaSuccess && gr->dstate && W > 1)
            e = cudaMemsetAsync(gr->dstate, 0, (size_t)d->batch * (W - 1) * C * sizeof(float), s);
        return e == cudaSuccess ? M3_OK : M3_ERR_CUDA;
    }
    const Geo g{d->batch, T, esize(d->io_dtype), false};
    if ((st = conv_common(d, g, x, weight, bias, seqlens, state0, flags)) != M3_OK) return st;
    if (!dy) return M3_ERR_NULL;
    if ((st = check_in(*dy, g)) != M3_OK) return st;
    if ((st = check_out(gr->dx, g, d->channels)) != M3_OK) return st;
    if (gr->dx.ptr == x->ptr || gr->dx.ptr == dy->ptr) return M3_ERR_UNSUPPORTED;
    ConvArgs a;
    conv_args(&a, d, T, x, weight, bias, seqlens, state0, flags);
    conv_runs(d, T, kConvBwdSlots, &a.seg, &a.nseg);
    if (!ws || !at_least(ws, 256) || ws_bytes < conv_bytes(d, a.nseg)) return M3_ERR_WORKSPACE;
    a.dy = view(*dy);
    set_out(a.dx, gr->dx);
    a.dweight = gr->dweight;
    a.dbias = bias ? gr->dbias : nullptr;
    a.dstate = gr->dstate;
    a.part = static_cast<float*>(ws);
    if ((int64_t)a.batch * a.nseg > kMaxBlocks) return M3_ERR_UNSUPPORTED;
    a.wide = conv_wide(d, weight, state0) && wide_rows(*x, g) && wide_rows(*dy, g) && wide_rows(gr->dx, g);
    return status_of(launch_conv(a, ConvCall::bwd, d->io_dtype, s));
}

}  // extern "C"

namespace {

// ------------------------------------------------------------------ selective scan

m3_status sel_dims_ok(const m3_sel_dims* d) {
    if (!d) return M3_ERR_NULL;
    if (!io_known(d->io_dtype)) return M3_ERR_DTYPE;
    if (d->batch < 1 || d->channels < 1 || d->ngroups < 1 || d->dstate < 1) return M3_ERR_SHAPE;
    if (d->channels % d->ngroups) return M3_ERR_SHAPE;
    if (d->dstate > 256 || d->channels > 1 << 24) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

m3_status sel_common(const m3_sel_dims* d, const Geo& g, const m3_sel_inputs* in, const void* h) {
    if (!in || !in->A || !h) return M3_ERR_NULL;
    m3_status st;
    for (const m3_rows* r : {&in->x, &in->dt, &in->B, &in->C})
        if ((st = check_in(*r, g)) != M3_OK) return st;
    if (in->z.ptr && (st = check_in(in->z, g)) != M3_OK) return st;
    if (!at_least(in->A, 4) || !at_least(h, 4) || (in->D && !at_least(in->D, 4)) ||
        (in->dt_bias && !at_least(in->dt_bias, 4)) || (in->seqlens && !at_least(in->seqlens, 4)))
        return M3_ERR_ALIGN;
    return M3_OK;
}

void sel_args(SelArgs* a, const m3_sel_dims* d, int32_t T, const m3_sel_inputs* in, const float* h,
              uint32_t flags) {
    std::memset(a, 0, sizeof(*a));
    a->x = view(in->x);
    a->dt = view(in->dt);
    a->B = view(in->B);
    a->C = view(in->C);
    a->z = view(in->z);
    a->A = in->A;
    a->Dskip = in->D;
    a->dt_bias = in->dt_bias;
    a->seqlens = in->seqlens;
    a->h = const_cast<float*>(h);
    a->batch = d->batch;
    a->T = T;
    a->D = d->channels;
    a->G = d->ngroups;
    a->N = d->dstate;
    a->softplus = flags & M3_FLAG_DT_SOFTPLUS;
}

// Whether every row of x, dt and z, and every group's part of it, starts on 16 bytes and is a
// multiple of 16 bytes long: tiles then come by asynchronous 16-byte copies.
bool sel_wide(const m3_sel_dims* d, const Geo& g, const m3_sel_inputs* in) {
    return d->channels / d->ngroups % (16 / (int)g.e) == 0 && wide_rows(in->x, g) &&
           wide_rows(in->dt, g) && (!in->z.ptr || wide_rows(in->z, g));
}
// The same of B and C.
bool sel_wide_bc(const m3_sel_dims* d, const Geo& g, const m3_sel_inputs* in) {
    return d->dstate % (16 / (int)g.e) == 0 && wide_rows(in->B, g) && wide_rows(in->C, g);
}

// An upper bound of the blocks of any launch over (tile, segment, batch) or over the states.
bool sel_grid_ok(const SelArgs& a) {
    const double cells = (double)a.batch * a.D * a.nseg;
    const double rows = (double)a.batch * a.T * a.G * 2 * a.N;
    return cells < 2147483647.0 && rows / 256 < 2147483646.0 &&
           (double)a.batch * a.D * a.N / 64 < 2147483646.0;
}

}  // namespace

extern "C" {

m3_status m3_sel_workspace_bytes(const m3_sel_dims* d, int32_t T, size_t* bytes) {
    m3_status st = sel_dims_ok(d);
    if (st != M3_OK) return st;
    if (!bytes) return M3_ERR_NULL;
    if (T < 0) return M3_ERR_SHAPE;
    if (T > kMaxTokens) return M3_ERR_UNSUPPORTED;
    const size_t n = T ? sel_fwd_most(d->batch, T, d->channels, d->ngroups, d->dstate) : 0;
    *bytes = n < 256 ? 256 : (n + 255) / 256 * 256;
    return M3_OK;
}

m3_status m3_sel_fwd(const m3_sel_dims* d, int32_t T, const m3_sel_inputs* in, float* h,
                     const m3_rows* y, void* ws, size_t ws_bytes, uint32_t flags, void* stream) {
    m3_status st = sel_dims_ok(d);
    if (st != M3_OK) return st;
    if (T < 0) return M3_ERR_SHAPE;
    if (T > kMaxTokens) return M3_ERR_UNSUPPORTED;
    if (flags & ~M3_FLAG_DT_SOFTPLUS) return M3_ERR_UNSUPPORTED;
    if (ws && !at_least(ws, 256)) return M3_ERR_WORKSPACE;
    if (T == 0) return M3_OK;
    const Geo g{d->batch, T, esize(d->io_dtype), false};
    if ((st = sel_common(d, g, in, h)) != M3_OK) return st;
    if (!y) return M3_ERR_NULL;
    if ((st = check_out(*y, g, d->channels)) != M3_OK) return st;
    SelArgs a;
    sel_args(&a, d, T, in, h, flags);
    set_out(a.y, *y);
    a.wide = sel_wide(d, g, in) && wide_rows(*y, g);
    a.wide_bc = sel_wide_bc(d, g, in);
    a.nseg = sel_fwd_segments(a.batch, T, a.D, a.G, a.N, &a.seg);
    if (a.nseg > 1 && (!ws || ws_bytes < sel_fwd_workspace(a.batch, T, a.D, a.G, a.N))) a.nseg = 1;
    if (a.nseg == 1) a.seg = T;
    a.hseg = static_cast<float*>(ws);
    a.dsum = a.hseg + (size_t)a.batch * a.nseg * a.D * a.N;
    if (!sel_grid_ok(a)) return M3_ERR_UNSUPPORTED;
    return status_of(launch_sel_fwd(a, d->io_dtype, static_cast<cudaStream_t>(stream)));
}

m3_status m3_sel_step(const m3_sel_dims* d, const m3_sel_inputs* in, float* h, const m3_rows* y,
                      uint32_t flags, void* stream) {
    m3_status st = sel_dims_ok(d);
    if (st != M3_OK) return st;
    if (flags & ~M3_FLAG_DT_SOFTPLUS) return M3_ERR_UNSUPPORTED;
    const Geo g{d->batch, 1, esize(d->io_dtype), true};
    if ((st = sel_common(d, g, in, h)) != M3_OK) return st;
    if (in->seqlens) return M3_ERR_UNSUPPORTED;
    if (!y) return M3_ERR_NULL;
    if ((st = check_out(*y, g, d->channels)) != M3_OK) return st;
    SelArgs a;
    sel_args(&a, d, 1, in, h, flags);
    set_out(a.y, *y);
    a.nseg = 1;
    if ((double)a.batch * a.D / 16 > 2147483646.0) return M3_ERR_UNSUPPORTED;
    a.wide = a.N % 4 == 0 && at_least(h, 16) && at_least(in->A, 16);
    // four neighbouring states of B and C are one access, and the batch fits a grid's second axis
    const size_t quad = 4 * g.e;
    a.step_rows = a.batch <= 65535 && at_least(in->B.ptr, quad) && at_least(in->C.ptr, quad) &&
                  (a.batch == 1 || (in->B.batch_stride % 4 == 0 && in->C.batch_stride % 4 == 0));
    return status_of(launch_sel_step(a, d->io_dtype, static_cast<cudaStream_t>(stream)));
}

m3_status m3_sel_bwd_workspace_bytes(const m3_sel_dims* d, int32_t T, size_t* bytes) {
    m3_status st = sel_dims_ok(d);
    if (st != M3_OK) return st;
    if (!bytes) return M3_ERR_NULL;
    if (T < 0) return M3_ERR_SHAPE;
    if (T > kMaxTokens) return M3_ERR_UNSUPPORTED;
    SelArgs a;
    std::memset(&a, 0, sizeof(a));
    a.batch = d->batch; a.T = T; a.D = d->channels; a.G = d->ngroups; a.N = d->dstate;
    const size_t n = sel_bwd_most(a);
    *bytes = n < 256 ? 256 : n;
    return M3_OK;
}

m3_status m3_sel_bwd(const m3_sel_dims* d, int32_t T, const m3_sel_inputs* in, const float* h0,
                     const m3_rows* dy, const float* dhT, const m3_sel_grads* gr, void* ws,
                     size_t ws_bytes, uint32_t flags, void* stream) {
    m3_status st = sel_dims_ok(d);
    if (st != M3_OK) return st;
    if (T < 0) return M3_ERR_SHAPE;
    if (T > kMaxTokens) return M3_ERR_UNSUPPORTED;
    if (flags & ~M3_FLAG_DT_SOFTPLUS) return M3_ERR_UNSUPPORTED;
    if (!in || !gr || !gr->dA || (in->D && !gr->dD) || (in->dt_bias && !gr->ddt_bias))
        return M3_ERR_NULL;
    for (const float* f : {dhT, (const float*)gr->dA, (const float*)gr->dD,
                           (const float*)gr->ddt_bias, (const float*)gr->dh})
        if (f && !at_least(f, 4)) return M3_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t D = d->channels, N = d->dstate, hb = sizeof(float) * (size_t)d->batch * D * N;
    if (T == 0) {
        cudaError_t e = cudaMemsetAsync(gr->dA, 0, D * N * sizeof(float), s);
        if (e == cudaSuccess && in->D) e = cudaMemsetAsync(gr->dD, 0, D * sizeof(float), s);
        if (e == cudaSuccess && in->dt_bias)
            e = cudaMemsetAsync(gr->ddt_bias, 0, D * sizeof(float), s);
        if (e == cudaSuccess && gr->dh && gr->dh != dhT)
            e = dhT ? cudaMemcpyAsync(gr->dh, dhT, hb, cudaMemcpyDeviceToDevice, s)
                    : cudaMemsetAsync(gr->dh, 0, hb, s);
        return e == cudaSuccess ? M3_OK : M3_ERR_CUDA;
    }
    const Geo g{d->batch, T, esize(d->io_dtype), false};
    if ((st = sel_common(d, g, in, h0)) != M3_OK) return st;
    if (!dy) return M3_ERR_NULL;
    if ((st = check_in(*dy, g)) != M3_OK) return st;
    const int64_t bn = (int64_t)d->ngroups * d->dstate;
    if ((st = check_out(gr->dx, g, d->channels)) != M3_OK ||
        (st = check_out(gr->ddt, g, d->channels)) != M3_OK ||
        (st = check_out(gr->dB, g, bn)) != M3_OK || (st = check_out(gr->dC, g, bn)) != M3_OK ||
        (in->z.ptr && (st = check_out(gr->dz, g, d->channels)) != M3_OK))
        return st;
    SelArgs a;
    sel_args(&a, d, T, in, h0, flags);
    const size_t need = sel_bwd_plan(&a, static_cast<char*>(ws));
    if (!ws || !at_least(ws, 256) || ws_bytes < need) return M3_ERR_WORKSPACE;
    if (!sel_grid_ok(a)) return M3_ERR_UNSUPPORTED;
    a.dy = view(*dy);
    set_out(a.dx, gr->dx);
    set_out(a.ddt, gr->ddt);
    set_out(a.dB, gr->dB);
    set_out(a.dC, gr->dC);
    set_out(a.dz, gr->dz);
    a.wide = sel_wide(d, g, in) && wide_rows(*dy, g) && wide_rows(gr->dx, g) &&
             wide_rows(gr->ddt, g) && (!in->z.ptr || wide_rows(gr->dz, g));
    a.wide_bc = sel_wide_bc(d, g, in);
    a.dhT = dhT;
    a.dA = gr->dA;
    a.dD = in->D ? gr->dD : nullptr;
    a.ddt_bias = in->dt_bias ? gr->ddt_bias : nullptr;
    a.dh = gr->dh;
    return status_of(launch_sel_bwd(a, d->io_dtype, s));
}

}  // extern "C"

namespace {

// ------------------------------------------------------------------ norm

m3_status norm_dims_ok(const m3_norm_dims* d) {
    if (!d) return M3_ERR_NULL;
    if (!io_known(d->io_dtype) || !io_known(d->res_dtype)) return M3_ERR_DTYPE;
    if (d->out != M3_OUT_IO && d->out != M3_OUT_E4M3) return M3_ERR_DTYPE;
    if (d->rows < 0 || d->width < 1) return M3_ERR_SHAPE;
    if (d->width > 32768) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

// A [rows][width] tensor of e-byte elements, or an absent optional one (ok).
m3_status check_mat(const void* p, int64_t stride, const m3_norm_dims* d, size_t e, bool needed) {
    if (!p) return needed ? M3_ERR_NULL : M3_OK;
    if (!at_least(p, e)) return M3_ERR_ALIGN;
    if (d->rows > 1 && stride < d->width) return M3_ERR_SHAPE;
    return M3_OK;
}

// Rows of vectors of 8 values: 16-byte aligned (e4m3: 8 bytes).
bool wide_mat(const void* p, int64_t stride, const m3_norm_dims* d, size_t e) {
    const size_t a = e == 1 ? 8 : 16;
    return !p || (at_least(p, a) && (d->rows == 1 || stride * (int64_t)e % (int64_t)a == 0));
}

}  // namespace

extern "C" {

m3_status m3_norm_fwd(const m3_norm_dims* d, const void* x, int64_t xs, const void* res, int64_t rs,
                      const float* weight, float eps, void* y, int64_t ys, float* scales,
                      void* res_out, int64_t ros, void* stream) {
    m3_status st = norm_dims_ok(d);
    if (st != M3_OK) return st;
    if (!(eps >= 0.f) || std::isinf(eps)) return M3_ERR_SHAPE;
    if (!res && d->res_dtype != d->io_dtype) return M3_ERR_DTYPE;
    if (d->rows == 0) return M3_OK;
    const size_t e = esize(d->io_dtype), er = esize(d->res_dtype);
    const size_t ey = d->out == M3_OUT_E4M3 ? 1 : e;
    if ((st = check_mat(x, xs, d, e, true)) != M3_OK || (st = check_mat(res, rs, d, er, false)) != M3_OK ||
        (st = check_mat(y, ys, d, ey, true)) != M3_OK ||
        (st = check_mat(res_out, ros, d, er, false)) != M3_OK)
        return st;
    if (d->out == M3_OUT_E4M3 && !scales) return M3_ERR_NULL;
    if ((weight && !at_least(weight, 4)) || (scales && !at_least(scales, 4))) return M3_ERR_ALIGN;
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.xs = xs; a.res = res; a.rs = rs; a.weight = weight; a.eps = eps;
    a.y = y; a.ys = ys; a.scales = scales; a.res_out = res_out; a.ros = ros;
    a.rows = d->rows; a.d = d->width;
    a.wide = d->width % 8 == 0 && wide_mat(x, xs, d, e) && wide_mat(res, rs, d, er) &&
             wide_mat(y, ys, d, ey) && wide_mat(res_out, ros, d, er) && wide_mat(weight, 0, d, 4);
    return status_of(launch_norm_fwd(a, d->io_dtype, d->res_dtype, d->out,
                                     static_cast<cudaStream_t>(stream)));
}

m3_status m3_norm_bwd_workspace_bytes(const m3_norm_dims* d, size_t* bytes) {
    m3_status st = norm_dims_ok(d);
    if (st != M3_OK) return st;
    if (!bytes) return M3_ERR_NULL;
    const size_t n = sizeof(float) * (size_t)norm_bwd_blocks(d->rows, d->width) * d->width;
    *bytes = n < 256 ? 256 : (n + 255) / 256 * 256;
    return M3_OK;
}

m3_status m3_norm_bwd(const m3_norm_dims* d, const void* r, int64_t rs, const float* weight,
                      float eps, const void* dy, int64_t dys, const void* dres, int64_t drs,
                      void* dx, int64_t dxs, void* dresidual, int64_t dros, float* dweight,
                      void* ws, size_t ws_bytes, void* stream) {
    m3_status st = norm_dims_ok(d);
    if (st != M3_OK) return st;
    if (!(eps >= 0.f) || std::isinf(eps)) return M3_ERR_SHAPE;
    if (weight && !dweight) return M3_ERR_NULL;
    if ((weight && !at_least(weight, 4)) || (dweight && !at_least(dweight, 4))) return M3_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d->rows == 0) {
        if (weight && cudaMemsetAsync(dweight, 0, sizeof(float) * d->width, s) != cudaSuccess)
            return M3_ERR_CUDA;
        return M3_OK;
    }
    const size_t e = esize(d->io_dtype), er = esize(d->res_dtype);
    if ((st = check_mat(r, rs, d, er, true)) != M3_OK || (st = check_mat(dy, dys, d, e, true)) != M3_OK ||
        (st = check_mat(dres, drs, d, er, false)) != M3_OK ||
        (st = check_mat(dx, dxs, d, e, true)) != M3_OK ||
        (st = check_mat(dresidual, dros, d, er, false)) != M3_OK)
        return st;
    size_t need;
    m3_norm_bwd_workspace_bytes(d, &need);
    if (weight && (!ws || !at_least(ws, 256) || ws_bytes < need)) return M3_ERR_WORKSPACE;
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = r; a.xs = rs; a.weight = weight; a.eps = eps; a.dy = dy; a.dys = dys;
    a.dres = dres; a.drs = drs; a.dx = dx; a.dxs = dxs; a.dresidual = dresidual; a.dros = dros;
    a.dweight = weight ? dweight : nullptr;
    a.part = weight ? static_cast<float*>(ws) : nullptr;
    a.rows = d->rows; a.d = d->width;
    a.blocks = norm_bwd_blocks(d->rows, d->width);
    a.wide = d->width % 8 == 0 && wide_mat(r, rs, d, er) && wide_mat(dy, dys, d, e) &&
             wide_mat(dres, drs, d, er) && wide_mat(dx, dxs, d, e) &&
             wide_mat(dresidual, dros, d, er) && wide_mat(weight, 0, d, 4);
    return status_of(launch_norm_bwd(a, d->io_dtype, d->res_dtype, s));
}

}  // extern "C"
