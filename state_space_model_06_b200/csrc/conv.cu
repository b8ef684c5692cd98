// conv.cu -- short causal convolution over the tokens, one filter a channel (m3_conv_*).
//
// y_t = act(bias + sum_k w[k] u_{t-W+1+k}).  A thread owns V neighbouring channels and walks a
// run of tokens; the W - 1 tokens before the current one stay in registers, so every x is read
// once from memory but for the W - 1 tokens at the start of a run.
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
__device__ __forceinline__ f2 silu2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(lo * sigmoid_f<IO>(lo), hi * sigmoid_f<IO>(hi));
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

// ------------------------------------------------------------------ forward

template <typename IO, int W, bool WIDE>
__global__ void __launch_bounds__(128) conv_fwd_kernel(const ConvArgs a) {
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
    const int te = min(t1, len);
    constexpr int U = 32 / (int)sizeof(IO) / 2;      // tokens on their way while U others are worked on
    Quad<IO> next[U];
    if (t0 < te)
#pragma unroll
        for (int u = 0; u < U; u++) next[u] = load_quad<IO, WIDE>(x + min(t0 + u, te - 1) * xts, n);

    f2 w[W][2], bias[2], win[W][2];      // win[j] holds u_{t-W+1+j}
    load_filter<W, WIDE>(a, c0, n, w, bias);
    load_window<IO, W, WIDE>(a, x, xts, st, t0, len, n, win);
    for (int t = t0; t < te; t += U) {
        Quad<IO> cur[U];
#pragma unroll
        for (int u = 0; u < U; u++) cur[u] = next[u];
        if (t + U < te)
#pragma unroll
            for (int u = 0; u < U; u++) next[u] = load_quad<IO, WIDE>(x + min(t + U + u, te - 1) * xts, n);
#pragma unroll
        for (int u = 0; u < U; u++) {
            f2 s[2];
            widen(win[W - 1], cur[u]);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                s[i] = bias[i];
#pragma unroll
                for (int k = 0; k < W; k++) s[i] = fma2(w[k][i], win[k][i], s[i]);
                if (a.silu) s[i] = silu2<IO>(s[i]);
#pragma unroll
                for (int k = 0; k < W - 1; k++) win[k][i] = win[k + 1][i];
            }
            if (t + u < te) store_quad<IO, WIDE>(s, y + (t + u) * yts, n);
        }
    }
    const f2 zero[2] = {0, 0};
    for (int t = max(t0, te); t < t1; t++) store_quad<IO, WIDE>(zero, y + t * yts, n);

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
        s[0] = silu2<IO>(s[0]);
        s[1] = silu2<IO>(s[1]);
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
__global__ void __launch_bounds__(128) conv_bwd_kernel(const ConvArgs a) {
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
    const int te = min(t1 + W - 1, len), last = t1 + W - 1;
    constexpr int U = 4;
    Quad<IO> nx[U], ng[U];
    auto request = [&](int t) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            nx[u] = load_quad<IO, WIDE>(x + min(t + u, te - 1) * xts, n);
            ng[u] = load_quad<IO, WIDE>(dy + min(t + u, te - 1) * gts, n);
        }
    };
    if (t0 < te) request(t0);
    f2 w[W][2], bias[2], win[W][2], dw[W][2], acc[W][2], db[2] = {0, 0};
    load_filter<W, WIDE>(a, c0, n, w, bias);
    load_window<IO, W, WIDE>(a, x, xts, st, t0, len, n, win);
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
        for (int i = 0; i < 2; i++) dw[k][i] = acc[k][i] = 0;   // acc[j]: dx_{t-W+1+j} so far

    for (int t = t0; t < last; t += U) {
        Quad<IO> cx[U], cg[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            cx[u] = nx[u];
            cg[u] = ng[u];
        }
        if (t + U < te) request(t + U);
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (t + u < last) {
                f2 g[2] = {0, 0};
                win[W - 1][0] = win[W - 1][1] = 0;
                if (t + u < te) {      // past the length nothing is looked at
                    widen(win[W - 1], cx[u]);
                    widen(g, cg[u]);
                    if (a.silu) {
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            f2 s = bias[i];
#pragma unroll
                            for (int k = 0; k < W; k++) s = fma2(w[k][i], win[k][i], s);
                            float v[2], d[2];
                            unpack2(s, v[0], v[1]);
#pragma unroll
                            for (int j = 0; j < 2; j++) {
                                const float sg = sigmoid_f<IO>(v[j]);
                                d[j] = fmaf(v[j] * sg, 1.f - sg, sg);
                            }
                            g[i] = mul2(g[i], pack2(d[0], d[1]));
                        }
                    }
                }
                const bool mine = t + u < t1;
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
                // acc[0] is complete: the gradient of token t + u - W + 1
                const int s = t + u - (W - 1);
                if (s >= t0) {
                    store_quad<IO, WIDE>(acc[0], dx + s * dts, n);
                } else if (s < 0 && a.dstate) {      // a carried token
                    float v[V];
                    unpack2(acc[0][0], v[0], v[1]);
                    unpack2(acc[0][1], v[2], v[3]);
                    float* o = a.dstate + ((long long)b * (W - 1) + (s + W - 1)) * a.C + c0;
#pragma unroll
                    for (int i = 0; i < V; i++)
                        if (i < n) o[i] = v[i];
                }
#pragma unroll
                for (int i = 0; i < 2; i++) {
#pragma unroll
                    for (int k = 0; k < W - 1; k++) {
                        win[k][i] = win[k + 1][i];
                        acc[k][i] = acc[k + 1][i];
                    }
                    acc[W - 1][i] = 0;
                }
            }
        }
    }
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

// Sums the shares over the runs, in a fixed order: a block per 32 channels and tap, its warps
// taking every eighth run each.
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const float* part, int runs, int W, int C,
                                                           float* dweight, float* dbias) {
    __shared__ float sm[8][33];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
    float s = 0.f;
    if (c < C)
        for (int r = wid; r < runs; r += 8) s += part[((long long)r * (W + 1) + k) * C + c];
    sm[wid][lane] = s;
    __syncthreads();
    if (wid == 0 && c < C) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) v += sm[i][lane];
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
    conv_bwd_sum_kernel<<<dim3((a.C + 31) / 32, W + 1), 256, 0, s>>>(
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
