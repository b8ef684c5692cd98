// conv.cu -- short causal convolution over the tokens, one filter a channel (m3_conv_*).
//
// y_t = act(bias + sum_k w[k] u_{t-W+1+k}).  A thread owns V neighbouring channels and walks a
// run of tokens; the W - 1 tokens before the current one stay in registers, so every x is read
// once from memory but for the W - 1 tokens at the start of a run.
#include "block_internal.h"
#include "block_common.cuh"

namespace m3 {

namespace {

// ------------------------------------------------------------------ forward

template <typename IO, int W, int V, bool WIDE>
__global__ void __launch_bounds__(128) conv_fwd_kernel(const ConvArgs a) {
    const int c0 = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c0 >= a.C) return;
    const int n = min(V, a.C - c0);
    const int b = blockIdx.x / a.nseg, seg = blockIdx.x - b * a.nseg;
    const int t0 = seg * a.seg;
    const int t1 = min(t0 + a.seg, a.T);
    const int len = tokens_of(a.seqlens, b, a.T);
    const Rows<const IO> X{static_cast<const IO*>(a.x.p), a.x.bs, a.x.ts};
    const Rows<IO> Y{static_cast<IO*>(a.y.p), a.y.bs, a.y.ts};
    IO* st = static_cast<IO*>(a.state) + (long long)b * (W - 1) * a.C + c0;

    float w[W][V], bias[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        bias[i] = (a.bias && i < n) ? a.bias[c0 + i] : 0.f;
#pragma unroll
        for (int k = 0; k < W; k++) w[k][i] = i < n ? a.weight[(long long)(c0 + i) * W + k] : 0.f;
    }
    // win[j] holds u_{t-W+1+j}; the newest, win[W-1], is the current token
    float win[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; j++) {
        const int t = t0 - (W - 1) + j;
        if (t >= 0)
            Vec<IO, V>::template load<WIDE>(win[j], X.at(b, t) + c0, t < len ? n : 0);
        else
            Vec<IO, V>::template load<WIDE>(win[j], st + (long long)(t + W - 1) * a.C, n);
    }
    const int te = min(t1, len);
    constexpr int U = 4;      // tokens requested together
    for (int t = t0; t < te; t += U) {
        float nx[U][V];
#pragma unroll
        for (int u = 0; u < U; u++)
            Vec<IO, V>::template load<WIDE>(nx[u], X.at(b, min(t + u, te - 1)) + c0, n);
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (t + u < te) {
                float y[V];
#pragma unroll
                for (int i = 0; i < V; i++) {
                    win[W - 1][i] = nx[u][i];
                    float s = bias[i];
#pragma unroll
                    for (int k = 0; k < W; k++) s = fmaf(w[k][i], win[k][i], s);
                    y[i] = a.silu ? s * sigmoid_f<IO>(s) : s;
#pragma unroll
                    for (int k = 0; k < W - 1; k++) win[k][i] = win[k + 1][i];
                }
                Vec<IO, V>::template store<WIDE>(y, Y.at(b, t + u) + c0, n);
            }
        }
    }
    const float zero[V] = {};
    for (int t = max(t0, te); t < t1; t++) Vec<IO, V>::template store<WIDE>(zero, Y.at(b, t) + c0, n);

    // The first segment alone reads the state, so it also writes the new one: the last W - 1
    // tokens of [state | x], oldest first (place j is u_{len-W+1+j}; each source is at or behind
    // the place that it goes to, and a place is read before a later step writes it).
    if (seg == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; j++) {
            const int t = len - (W - 1) + j;
            float v[V];
            if (t >= 0)
                Vec<IO, V>::template load<WIDE>(v, X.at(b, t) + c0, n);
            else
                Vec<IO, V>::template load<WIDE>(v, st + (long long)(t + W - 1) * a.C, n);
            Vec<IO, V>::template store<WIDE>(v, st + (long long)j * a.C, n);
        }
    }
}

// ------------------------------------------------------------------ one token

template <typename IO, int W, int V, bool WIDE>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvArgs a) {
    const long long per = (a.C + V - 1) / V;
    const long long id = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (id >= per * a.batch) return;
    const int b = (int)(id / per), c0 = (int)(id - b * per) * V;
    const int n = min(V, a.C - c0);
    IO* st = static_cast<IO*>(a.state) + (long long)b * (W - 1) * a.C + c0;
    float win[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; j++)
        Vec<IO, V>::template load<WIDE>(win[j], st + (long long)j * a.C, n);
    Vec<IO, V>::template load<WIDE>(win[W - 1], static_cast<const IO*>(a.x.p) + b * a.x.bs + c0, n);
    float y[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        float s = (a.bias && i < n) ? a.bias[c0 + i] : 0.f;
#pragma unroll
        for (int k = 0; k < W; k++)
            s = fmaf(i < n ? a.weight[(long long)(c0 + i) * W + k] : 0.f, win[k][i], s);
        y[i] = a.silu ? s * sigmoid_f<IO>(s) : s;
    }
#pragma unroll
    for (int j = 0; j < W - 1; j++)
        Vec<IO, V>::template store<WIDE>(win[j + 1], st + (long long)j * a.C, n);
    Vec<IO, V>::template store<WIDE>(y, static_cast<IO*>(a.y.p) + b * a.y.bs + c0, n);
}

// ------------------------------------------------------------------ backward
//
// g_t = dy_t act'(pre_t);  dx_s = sum_k w[k] g_{s+W-1-k};  dw[k] = sum_t g_t u_{t-W+1+k}.
// A thread walks the tokens t0 .. t1 + W - 2 of its run, recomputing pre from x.  Its own
// tokens' g go into dw; dx_s is complete once g_{s+W-1} is known.  The first segment also
// covers s = -(W-1) .. -1, the gradients of the carried tokens.

template <typename IO, int W, int V, bool WIDE>
__global__ void __launch_bounds__(128) conv_bwd_kernel(const ConvArgs a) {
    const int c0 = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c0 >= a.C) return;
    const int n = min(V, a.C - c0);
    const int b = blockIdx.x / a.nseg, seg = blockIdx.x - b * a.nseg;
    const int t0 = seg * a.seg;
    const int t1 = min(t0 + a.seg, a.T);
    const int len = tokens_of(a.seqlens, b, a.T);
    const Rows<const IO> X{static_cast<const IO*>(a.x.p), a.x.bs, a.x.ts};
    const Rows<const IO> DY{static_cast<const IO*>(a.dy.p), a.dy.bs, a.dy.ts};
    const Rows<IO> DX{static_cast<IO*>(a.dx.p), a.dx.bs, a.dx.ts};
    const IO* st = static_cast<const IO*>(a.state) + (long long)b * (W - 1) * a.C + c0;

    float w[W][V], bias[V], dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        bias[i] = (a.bias && i < n) ? a.bias[c0 + i] : 0.f;
        db[i] = 0.f;
#pragma unroll
        for (int k = 0; k < W; k++) {
            w[k][i] = i < n ? a.weight[(long long)(c0 + i) * W + k] : 0.f;
            dw[k][i] = 0.f;
        }
    }
    float win[W][V];   // u_{t-W+1+j}
    float acc[W][V];   // acc[j]: dx_{t-W+1+j} so far
#pragma unroll
    for (int j = 0; j < W; j++)
#pragma unroll
        for (int i = 0; i < V; i++) acc[j][i] = 0.f;
#pragma unroll
    for (int j = 0; j < W - 1; j++) {
        const int t = t0 - (W - 1) + j;
        if (t >= 0)
            Vec<IO, V>::template load<WIDE>(win[j], X.at(b, t) + c0, t < len ? n : 0);
        else
            Vec<IO, V>::template load<WIDE>(win[j], st + (long long)(t + W - 1) * a.C, n);
    }
    // tokens t1 .. t1 + W - 2 only finish this run's dx (they are the next run's own)
    for (int t = t0; t < t1 + W - 1; t++) {
        float dy[V];
        const bool in = t < len;
        Vec<IO, V>::template load<WIDE>(win[W - 1], X.at(b, min(t, a.T - 1)) + c0, in ? n : 0);
        Vec<IO, V>::template load<WIDE>(dy, DY.at(b, min(t, a.T - 1)) + c0, in ? n : 0);
        const bool mine = t < t1;
#pragma unroll
        for (int i = 0; i < V; i++) {
            float g = dy[i];
            if (a.silu) {
                float s = bias[i];
#pragma unroll
                for (int k = 0; k < W; k++) s = fmaf(w[k][i], win[k][i], s);
                const float sg = sigmoid_f<IO>(s);
                g *= sg * (1.f + s * (1.f - sg));
            }
            if (!in) g = 0.f;      // past the length: dy is not looked at, 0 * inf stays out
            const float own = mine ? g : 0.f;
            db[i] += own;
#pragma unroll
            for (int k = 0; k < W; k++) {
                dw[k][i] = fmaf(own, win[k][i], dw[k][i]);
                acc[k][i] = fmaf(w[k][i], g, acc[k][i]);
            }
        }
        // acc[0] is complete: the gradient of token t - W + 1
        const int s = t - (W - 1);
        if (s >= t0) {
            if (s < t1) Vec<IO, V>::template store<WIDE>(acc[0], DX.at(b, s) + c0, n);
        } else if (seg == 0 && a.dstate) {
            // s < 0: a carried token (s >= t0 = 0 was taken above)
            float* o = a.dstate + ((long long)b * (W - 1) + (s + W - 1)) * a.C + c0;
#pragma unroll
            for (int i = 0; i < V; i++)
                if (i < n) o[i] = acc[0][i];
        }
#pragma unroll
        for (int i = 0; i < V; i++) {
#pragma unroll
            for (int k = 0; k < W - 1; k++) {
                win[k][i] = win[k + 1][i];
                acc[k][i] = acc[k + 1][i];
            }
            acc[W - 1][i] = 0.f;
        }
    }
    // shares of this run: [b * nseg + seg][W + 1][C]
    float* part = a.part + (long long)blockIdx.x * (W + 1) * a.C + c0;
#pragma unroll
    for (int i = 0; i < V; i++)
        if (i < n) {
#pragma unroll
            for (int k = 0; k < W; k++) part[(long long)k * a.C + i] = dw[k][i];
            part[(long long)W * a.C + i] = db[i];
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
    constexpr int V = 16 / sizeof(IO);
    const dim3 grid(a.batch * a.nseg, (a.C + 128 * V - 1) / (128 * V));
    conv_fwd_kernel<IO, W, V, WIDE><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, int W, bool WIDE>
cudaError_t step_t(const ConvArgs& a, cudaStream_t s) {
    constexpr int V = WIDE ? 16 / (int)sizeof(IO) : 1;
    const long long n = (long long)a.batch * ((a.C + V - 1) / V);
    conv_step_kernel<IO, W, V, WIDE><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, int W, bool WIDE>
cudaError_t bwd_t(const ConvArgs& a, cudaStream_t s) {
    constexpr int V = 4;
    const dim3 grid(a.batch * a.nseg, (a.C + 128 * V - 1) / (128 * V));
    conv_bwd_kernel<IO, W, V, WIDE><<<grid, 128, 0, s>>>(a);
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
