// conv.cu -- short causal convolution over the tokens, one filter a channel (m3_conv_*).
//
// y_t = act(bias + sum_k w[k] u_{t-W+1+k}).  A thread owns four neighbouring channels and walks a
// run of tokens; the W - 1 tokens before the current one stay in registers, so every x is read
// once from memory but for the W - 1 tokens at the start of a run.
//
// Memory bounds it.  Prompt, 8 x 4096 tokens of 4096 channels, W 4, SiLU, bf16: 106 us, one call
// after another (5.1 TB/s; 82 us at the copy rate), 94 alone in a graph; there the first forms took
// 299 us (eight channels and scalar arithmetic: 120 registers, 16 warps an SM) and 164 (packed
// pairs).  Backward, 4 x 2048 tokens: 62 us (58 alone) where the bytes would take 31: 124 registers
// hold 16 warps an SM, and each token's chain (convolution, logistic, three sums) is not covered by
// four warps a sub-partition; alone, five blocks an SM spill (98 us), and two channels a thread,
// with 28 warps, double the copies and addresses (62 us).
#include "block_internal.h"
#include "block_common.cuh"

namespace m3 {

namespace {

// Four channels a thread, as two pairs: a pair of fp32 values takes one FFMA2 for its two taps.
constexpr int V = 4;

template <typename IO>
struct alignas(V * sizeof(IO)) Quad {
    IO v[V];
};

// The n values at p (WIDE: all four, in one access); the rest are zero.
template <typename IO, bool WIDE>
__device__ __forceinline__ Quad<IO> load_quad(const IO* p, int n) {
    if constexpr (WIDE) {
        return *reinterpret_cast<const Quad<IO>*>(p);
    } else {
        Quad<IO> q;
#pragma unroll
        for (int i = 0; i < V; i++) q.v[i] = i < n ? p[i] : from_f<IO>(0.f);
        return q;
    }
}
template <typename IO>
__device__ __forceinline__ void widen(f2 (&f)[2], const Quad<IO>& q) {
    f[0] = pack2(to_f(q.v[0]), to_f(q.v[1]));
    f[1] = pack2(to_f(q.v[2]), to_f(q.v[3]));
}
template <typename IO, bool WIDE>
__device__ __forceinline__ void store_quad(const f2 (&f)[2], IO* p, int n) {
    float v[V];
    unpack2(f[0], v[0], v[1]);
    unpack2(f[1], v[2], v[3]);
    Vec<IO, V>::template store<WIDE>(v, p, n);
}

// Taps and bias of a thread's channels: w[k] as pairs of channels.  The V x W weights lie behind
// each other in memory, so they come as whole 16-byte loads.
template <int W, bool WIDE>
__device__ __forceinline__ void load_filter(const ConvArgs& a, int c0, int n, f2 (&w)[W][2], f2 (&bias)[2]) {
    float f[V * W], bs[V];
    const float* p = a.weight + (long long)c0 * W;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < W; i++) {
            const float4 q = reinterpret_cast<const float4*>(p)[i];
            f[4 * i] = q.x; f[4 * i + 1] = q.y; f[4 * i + 2] = q.z; f[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; i++) f[i] = i < n * W ? p[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; i++) bs[i] = a.bias && i < n ? a.bias[c0 + i] : 0.f;
#pragma unroll
    for (int k = 0; k < W; k++) {
        w[k][0] = pack2(f[k], f[W + k]);
        w[k][1] = pack2(f[2 * W + k], f[3 * W + k]);
    }
    bias[0] = pack2(bs[0], bs[1]);
    bias[1] = pack2(bs[2], bs[3]);
}

template <typename IO>
__device__ __forceinline__ f2 sigmoid2(f2 v) {
    float lo, hi;
    if constexpr (sizeof(IO) == 2) {
        unpack2(mul2(v, pack2(-kLog2e, -kLog2e)), lo, hi);
        unpack2(add2(pack2(ex2(lo), ex2(hi)), pack2(1.f, 1.f)), lo, hi);
        return pack2(rcp(lo), rcp(hi));
    } else {
        unpack2(v, lo, hi);
        return pack2(sigmoid_f<IO>(lo), sigmoid_f<IO>(hi));
    }
}

// The tokens before t0 into win[0 .. W-2].
template <typename IO, int W, bool WIDE>
__device__ __forceinline__ void load_window(const ConvArgs& a, const IO* x, long long ts, const IO* st,
                                            int t0, int len, int n, f2 (&win)[W][2]) {
#pragma unroll
    for (int j = 0; j < W - 1; j++) {
        const int t = t0 - (W - 1) + j;
        win[j][0] = win[j][1] = 0;
        if (t < 0)
            widen(win[j], load_quad<IO, WIDE>(st + (long long)(t + W - 1) * a.C, n));
        else if (t < len)
            widen(win[j], load_quad<IO, WIDE>(x + t * ts, n));
    }
}

// A thread's coming tokens: R tensors, groups of U tokens, D groups on their way.  With wide rows
// they come by asynchronous copies into places that the thread alone reads, so there is nothing
// to wait for but its own copies; loads into registers held up to 3.5 TB/s (the prompt case:
// 152 us alone), as a thread's registers hold only a few tokens and its loads share few scoreboards.
template <typename IO, int R, int D, bool WIDE>
struct Ahead {
    static constexpr int U = 4;
    const IO* p[R];
    long long ts[R];
    Quad<IO>* sm;      // [D][R][U][blockDim]
    int n, left, slot;
    __device__ __forceinline__ void start(int groups) {
        left = groups;
        slot = 0;
        if constexpr (WIDE)
#pragma unroll
            for (int d = 0; d < D - 1; d++) ask(d);
    }
    __device__ __forceinline__ Quad<IO>* at(int d, int r, int u) {
        return sm + ((d * R + r) * U + u) * 128 + threadIdx.x;
    }
    __device__ __forceinline__ void ask(int d) {
        if (left > 0) {
            left--;
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int u = 0; u < U; u++) {
                    cp_async<V * (int)sizeof(IO)>(at(d, r, u), p[r]);
                    p[r] += ts[r];
                }
        }
        cp_async_commit();
    }
    // The next group's values.
    __device__ __forceinline__ void take(Quad<IO> (&q)[R][U]) {
        if constexpr (WIDE) {
            cp_async_wait<D - 2>();
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int u = 0; u < U; u++) q[r][u] = *at(slot, r, u);
            ask(slot == 0 ? D - 1 : slot - 1);      // the place of the group before
            slot = slot == D - 1 ? 0 : slot + 1;
        } else {
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int u = 0; u < U; u++, p[r] += ts[r]) q[r][u] = load_quad<IO, WIDE>(p[r], n);
        }
    }
    // One token more, behind the groups (p points at it once every group has been asked for).
    __device__ __forceinline__ Quad<IO> one(int r) {
        const Quad<IO> q = load_quad<IO, WIDE>(p[r], n);
        p[r] += ts[r];
        return q;
    }
};

// ------------------------------------------------------------------ forward

template <typename IO, int W, bool WIDE>
__global__ void __launch_bounds__(128, W <= 4 ? 7 : 4) conv_fwd_kernel(const ConvArgs a) {
    const int c0 = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c0 >= a.C) return;
    const int n = min(V, a.C - c0);
    const int b = blockIdx.x / a.nseg, seg = blockIdx.x - b * a.nseg;
    const int t0 = seg * a.seg;
    const int t1 = min(t0 + a.seg, a.T);
    const int len = tokens_of(a.seqlens, b, a.T);
    const long long xts = a.x.ts, yts = a.y.ts;
    const IO* x = static_cast<const IO*>(a.x.p) + b * a.x.bs + c0;
    IO* y = static_cast<IO*>(a.y.p) + b * a.y.bs + c0;
    IO* st = static_cast<IO*>(a.state) + (long long)b * (W - 1) * a.C + c0;
    const int te = max(min(t1, len), t0);
    using In = Ahead<IO, 1, 4, WIDE>;
    constexpr int U = In::U;
    __shared__ Quad<IO> sm[WIDE ? 4 * U * 128 : 1];
    In in{{x + t0 * xts}, {xts}, sm, n};
    const int groups = (te - t0) / U;
    in.start(groups);
    IO* py = y + t0 * yts;

    f2 w[W][2], bias[2], win[W][2];      // win[j] holds u_{t-W+1+j}
    load_filter<W, WIDE>(a, c0, n, w, bias);
    load_window<IO, W, WIDE>(a, x, xts, st, t0, len, n, win);
    auto token = [&](const Quad<IO>& q) {
        f2 s[2];
        widen(win[W - 1], q);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            s[i] = bias[i];
#pragma unroll
            for (int k = 0; k < W; k++) s[i] = fma2(w[k][i], win[k][i], s[i]);
            if (a.silu) s[i] = mul2(s[i], sigmoid2<IO>(s[i]));
#pragma unroll
            for (int k = 0; k < W - 1; k++) win[k][i] = win[k + 1][i];
        }
        store_quad<IO, WIDE>(s, py, n);
        py += yts;
    };
    for (int g = 0; g < groups; g++) {
        Quad<IO> q[1][U];
        in.take(q);
#pragma unroll
        for (int u = 0; u < U; u++) token(q[0][u]);
    }
    for (int t = t0 + groups * U; t < te; t++) token(in.one(0));
    cp_async_wait<0>();
    const f2 zero[2] = {0, 0};
    for (int t = te; t < t1; t++) store_quad<IO, WIDE>(zero, y + t * yts, n);

    // The first run alone reads the state, so it also writes the new one: the last W - 1
    // tokens of [state | x], oldest first (place j is u_{len-W+1+j}; each source is at or behind
    // the place that it goes to, and a place is read before a later step writes it).
    if (seg == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; j++) {
            const int t = len - (W - 1) + j;
            const Quad<IO> q = load_quad<IO, WIDE>(t >= 0 ? x + t * xts : st + (long long)(t + W - 1) * a.C, n);
            IO* o = st + (long long)j * a.C;
            if constexpr (WIDE) {
                *reinterpret_cast<Quad<IO>*>(o) = q;
            } else {
#pragma unroll
                for (int i = 0; i < V; i++)
                    if (i < n) o[i] = q.v[i];
            }
        }
    }
}

// ------------------------------------------------------------------ one token

template <typename IO, int W, bool WIDE>
__global__ void __launch_bounds__(64) conv_step_kernel(const ConvArgs a) {
    const int per = (a.C + V - 1) / V;
    const long long id = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (id >= (long long)per * a.batch) return;
    const int b = (int)(id / per), c0 = (int)(id - (long long)b * per) * V;
    const int n = min(V, a.C - c0);
    IO* st = static_cast<IO*>(a.state) + (long long)b * (W - 1) * a.C + c0;
    Quad<IO> q[W];
#pragma unroll
    for (int j = 0; j < W - 1; j++) q[j] = load_quad<IO, WIDE>(st + (long long)j * a.C, n);
    q[W - 1] = load_quad<IO, WIDE>(static_cast<const IO*>(a.x.p) + b * a.x.bs + c0, n);
    f2 w[W][2], s[2];
    load_filter<W, WIDE>(a, c0, n, w, s);
#pragma unroll
    for (int k = 0; k < W; k++) {
        f2 u[2];
        widen(u, q[k]);
        s[0] = fma2(w[k][0], u[0], s[0]);
        s[1] = fma2(w[k][1], u[1], s[1]);
    }
    if (a.silu) {
        s[0] = mul2(s[0], sigmoid2<IO>(s[0]));
        s[1] = mul2(s[1], sigmoid2<IO>(s[1]));
    }
#pragma unroll
    for (int j = 0; j < W - 1; j++) {
        IO* o = st + (long long)j * a.C;
        if constexpr (WIDE) {
            *reinterpret_cast<Quad<IO>*>(o) = q[j + 1];
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (i < n) o[i] = q[j + 1].v[i];
        }
    }
    store_quad<IO, WIDE>(s, static_cast<IO*>(a.y.p) + b * a.y.bs + c0, n);
}

// ------------------------------------------------------------------ backward
//
// g_t = dy_t act'(pre_t);  dx_s = sum_k w[k] g_{s+W-1-k};  dw[k] = sum_t g_t u_{t-W+1+k}.
// A thread walks the tokens t0 .. t1 + W - 2 of its run, recomputing pre from x.  Its own
// tokens' g go into dw; dx_s is complete once g_{s+W-1} is known.  The first run also
// covers s = -(W-1) .. -1, the gradients of the carried tokens.

template <typename IO, int W, bool WIDE>
__global__ void __launch_bounds__(128, W <= 4 ? 4 : 2) conv_bwd_kernel(const ConvArgs a) {
    const int c0 = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c0 >= a.C) return;
    const int n = min(V, a.C - c0);
    const int b = blockIdx.x / a.nseg, seg = blockIdx.x - b * a.nseg;
    const int t0 = seg * a.seg;
    const int t1 = min(t0 + a.seg, a.T);
    const int len = tokens_of(a.seqlens, b, a.T);
    const long long xts = a.x.ts, gts = a.dy.ts, dts = a.dx.ts;
    const IO* x = static_cast<const IO*>(a.x.p) + b * a.x.bs + c0;
    const IO* dy = static_cast<const IO*>(a.dy.p) + b * a.dy.bs + c0;
    IO* dx = static_cast<IO*>(a.dx.p) + b * a.dx.bs + c0;
    const IO* st = static_cast<const IO*>(a.state) + (long long)b * (W - 1) * a.C + c0;

    // the tokens that are looked at: this run's, and W - 1 behind it that only finish its dx
    const int te = max(min(t1 + W - 1, len), t0), last = t1 + W - 1;
    constexpr int D = sizeof(IO) == 2 ? 4 : 3;
    using In = Ahead<IO, 2, D, WIDE>;
    constexpr int U = In::U;
    __shared__ Quad<IO> sm[WIDE ? D * 2 * U * 128 : 1];
    In in{{x + t0 * xts, dy + t0 * gts}, {xts, gts}, sm, n};
    const int groups = max(min(t1, len) - t0, 0) / U;      // whole groups of the run's own tokens
    in.start(groups);
    IO* pd = dx + (t0 - (W - 1)) * dts;
    f2 w[W][2], bias[2], win[W][2], dw[W][2], acc[W][2], db[2] = {0, 0};
    load_filter<W, WIDE>(a, c0, n, w, bias);
    load_window<IO, W, WIDE>(a, x, xts, st, t0, len, n, win);
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
        for (int i = 0; i < 2; i++) dw[k][i] = acc[k][i] = 0;   // acc[j]: dx_{t-W+1+j} so far

    // inside: the token is inside the sequence; mine: it is one of the run's own
    auto token = [&](const Quad<IO>& qx, const Quad<IO>& qg, int t, bool inside, bool mine) {
        f2 g[2] = {0, 0};
        win[W - 1][0] = win[W - 1][1] = 0;
        if (inside) {
            widen(win[W - 1], qx);
            widen(g, qg);
            if (a.silu) {
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    f2 s = bias[i];
#pragma unroll
                    for (int k = 0; k < W; k++) s = fma2(w[k][i], win[k][i], s);
                    // act' = sg + s sg (1 - sg)
                    const f2 sg = sigmoid2<IO>(s), m = fma2(sg, pack2(-1.f, -1.f), pack2(1.f, 1.f));
                    g[i] = mul2(g[i], fma2(mul2(s, sg), m, sg));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const f2 own = mine ? g[i] : 0;
            db[i] = add2(db[i], own);
#pragma unroll
            for (int k = 0; k < W; k++) {
                dw[k][i] = fma2(own, win[k][i], dw[k][i]);
                acc[k][i] = fma2(w[k][i], g[i], acc[k][i]);
            }
        }
        // acc[0] is complete: the gradient of token t - W + 1
        const int s = t - (W - 1);
        if (s >= t0) {
            store_quad<IO, WIDE>(acc[0], pd, n);
        } else if (s < 0 && a.dstate) {      // a carried token
            float v[V];
            unpack2(acc[0][0], v[0], v[1]);
            unpack2(acc[0][1], v[2], v[3]);
            float* o = a.dstate + ((long long)b * (W - 1) + (s + W - 1)) * a.C + c0;
#pragma unroll
            for (int i = 0; i < V; i++)
                if (i < n) o[i] = v[i];
        }
        pd += dts;
#pragma unroll
        for (int i = 0; i < 2; i++) {
#pragma unroll
            for (int k = 0; k < W - 1; k++) {
                win[k][i] = win[k + 1][i];
                acc[k][i] = acc[k + 1][i];
            }
            acc[W - 1][i] = 0;
        }
    };
    for (int k = 0; k < groups; k++) {
        Quad<IO> q[2][U];
        in.take(q);
#pragma unroll
        for (int u = 0; u < U; u++) token(q[0][u], q[1][u], t0 + k * U + u, true, true);
    }
    for (int t = t0 + groups * U; t < last; t++) {
        Quad<IO> qx, qg;
        const bool inside = t < te;
        if (inside) {
            qx = in.one(0);
            qg = in.one(1);
        }
        token(qx, qg, t, inside, t < t1);
    }
    cp_async_wait<0>();
    // shares of this run: [b * nseg + seg][W + 1][C]
    float* part = a.part + (long long)blockIdx.x * (W + 1) * a.C + c0;
#pragma unroll
    for (int k = 0; k <= W; k++) {
        float v[V];
        unpack2(k < W ? dw[k < W ? k : 0][0] : db[0], v[0], v[1]);
        unpack2(k < W ? dw[k < W ? k : 0][1] : db[1], v[2], v[3]);
        Vec<float, V>::template store<WIDE>(v, part + (long long)k * a.C, n);
    }
}

// Sums the shares over the runs: a block per 32 channels and tap (the last one is the bias).
__global__ void __launch_bounds__(1024) conv_bwd_sum_kernel(const float* part, int runs, int W, int C,
                                                            float* dweight, float* dbias) {
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = blockIdx.y;
    const float v = column_sum(part + (long long)k * C + c, runs, (long long)(W + 1) * C, c < C);
    if (threadIdx.x < 32 && c < C) {
        if (k < W)
            dweight[(long long)c * W + k] = v;
        else if (dbias)
            dbias[c] = v;
    }
}

template <typename IO, int W, bool WIDE>
cudaError_t fwd_t(const ConvArgs& a, cudaStream_t s) {
    const dim3 grid(a.batch * a.nseg, (a.C + 128 * V - 1) / (128 * V));
    conv_fwd_kernel<IO, W, WIDE><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, int W, bool WIDE>
cudaError_t step_t(const ConvArgs& a, cudaStream_t s) {
    const long long n = (long long)a.batch * ((a.C + V - 1) / V);
    conv_step_kernel<IO, W, WIDE><<<(unsigned)((n + 63) / 64), 64, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, int W, bool WIDE>
cudaError_t bwd_t(const ConvArgs& a, cudaStream_t s) {
    const dim3 grid(a.batch * a.nseg, (a.C + 128 * V - 1) / (128 * V));
    conv_bwd_kernel<IO, W, WIDE><<<grid, 128, 0, s>>>(a);
    conv_bwd_sum_kernel<<<dim3((a.C + 31) / 32, W + 1), column_threads((long long)a.C * (W + 1)), 0, s>>>(
        a.part, a.batch * a.nseg, W, a.C, a.dweight, a.dbias);
    return cudaGetLastError();
}

template <typename IO, int W>
cudaError_t dispatch(const ConvArgs& a, ConvCall call, cudaStream_t s) {
    switch (call) {
        case ConvCall::fwd: return a.wide ? fwd_t<IO, W, true>(a, s) : fwd_t<IO, W, false>(a, s);
        case ConvCall::step: return a.wide ? step_t<IO, W, true>(a, s) : step_t<IO, W, false>(a, s);
        case ConvCall::bwd: return a.wide ? bwd_t<IO, W, true>(a, s) : bwd_t<IO, W, false>(a, s);
    }
    return cudaErrorNotSupported;
}

template <typename IO>
cudaError_t by_width(const ConvArgs& a, ConvCall call, cudaStream_t s) {
    switch (a.W) {
        case 1: return dispatch<IO, 1>(a, call, s);
        case 2: return dispatch<IO, 2>(a, call, s);
        case 3: return dispatch<IO, 3>(a, call, s);
        case 4: return dispatch<IO, 4>(a, call, s);
        case 5: return dispatch<IO, 5>(a, call, s);
        case 6: return dispatch<IO, 6>(a, call, s);
        case 7: return dispatch<IO, 7>(a, call, s);
        case 8: return dispatch<IO, 8>(a, call, s);
    }
    return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_conv(const ConvArgs& a, ConvCall call, int io_dtype, cudaStream_t s) {
    return io_dtype == M3_BF16 ? by_width<__nv_bfloat16>(a, call, s) : by_width<float>(a, call, s);
}

}  // namespace m3
