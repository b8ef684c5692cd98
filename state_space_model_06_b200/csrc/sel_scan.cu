// sel_scan.cu -- selective scan with a diagonal state per channel: prompts and single tokens
// (m3_sel_fwd, m3_sel_step).
//
//   h_t[c][n] = e^{delta_t[c] A[c][n]} h_{t-1}[c][n] + delta_t[c] x_t[c] B_t[n]
//   y_t[c]    = (sum_n C_t[n] h_t[c][n] + D[c] x_t[c]) SiLU(z_t[c])
//
// Every (token, channel, state) needs an exponential, and every channel and state has a decay of
// its own, so the chunked matrix form of the mixer's scan does not apply: the work is one ex2 and
// four fp32 operations a cell on registers, and what bounds it is the exponential unit
// (16 a clock and SM) well above the memory's share for N >= 8.
#include "block_internal.h"
#include "sel_tile.cuh"

namespace m3 {

namespace {

// One block: CB channels of one group over one segment.  LOCAL: the segment's own end state from
// no entry state, and its sum of delta (no y).  Otherwise the outputs, from the entry state in
// hseg (segmented) or in h.
template <typename IO, typename SH, bool LOCAL>
__global__ void __launch_bounds__(SH::THREADS) sel_scan_kernel(const SelArgs a) {
    constexpr int L = SH::L, NT = SH::NT, S = SH::S, CW = SH::CW, CB = SH::CB, NP = SH::NP;
    __shared__ alignas(16) float bc[L * 2 * NP];
    __shared__ float2 dd[L][CB];     // delta, delta * x
    const SelPlace p = sel_place(a, CB);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int cl = wid * CW + lane % CW;     // channel within the block
    const int s = lane / CW;                 // which NT states
    const bool live = cl < p.nc;
    const int c = p.c0 + cl;

    float h[NT], A2[NT];
    const long long row = ((long long)p.b * a.D + c) * a.N;
    const long long rowseg = (((long long)p.b * a.nseg + p.seg) * a.D + c) * a.N;
#pragma unroll
    for (int i = 0; i < NT; i++) {
        const int n = s * NT + i;
        const bool on = live && n < a.N;
        A2[i] = on ? a.A[(long long)c * a.N + n] * kLog2e : 0.f;
        h[i] = 0.f;
        if (!LOCAL && on) h[i] = a.nseg > 1 ? a.hseg[rowseg + n] : a.h[row + n];
    }
    float total = 0.f;
    const int end = min(p.t1, p.len);
    const Rows<const IO> X{static_cast<const IO*>(a.x.p), a.x.bs, a.x.ts};
    const Rows<const IO> DT{static_cast<const IO*>(a.dt.p), a.dt.bs, a.dt.ts};
    const Rows<const IO> Z{static_cast<const IO*>(a.z.p), a.z.bs, a.z.ts};
    const Rows<IO> Y{static_cast<IO*>(a.y.p), a.y.bs, a.y.ts};

    for (int t0 = p.t0; t0 < end; t0 += L) {
        __syncthreads();
        sel_stage_bc<IO, NP, L, SH::THREADS>(a, p, t0, end, bc);
        for (int i = threadIdx.x; i < L * CB; i += SH::THREADS) {
            const int k = i % CB, t = t0 + i / CB;
            float2 v = make_float2(0.f, 0.f);
            if (t < end && k < p.nc) {
                v.x = sel_delta(to_f(DT.at(p.b, t)[p.c0 + k]), a.dt_bias ? a.dt_bias[p.c0 + k] : 0.f,
                                a.softplus);
                v.y = v.x * to_f(X.at(p.b, t)[p.c0 + k]);
            }
            dd[i / CB][k] = v;
        }
        __syncthreads();
        const int count = min(L, end - t0);
        for (int u0 = 0; u0 < count; u0 += S) {
            float y[S];
#pragma unroll
            for (int u = 0; u < S; u++) {
                const float2 d = dd[u0 + u][cl];       // zero past the end: h stays
                const float4* pb = reinterpret_cast<const float4*>(bc + (u0 + u) * 2 * NP + s * NT);
                const float4* pc = reinterpret_cast<const float4*>(bc + ((u0 + u) * 2 + 1) * NP + s * NT);
                float acc = 0.f;
#pragma unroll
                for (int q = 0; q < NT / 4; q++) {
                    const float4 B4 = pb[q];
                    float4 C4;
                    if (!LOCAL) C4 = pc[q];
                    const float Bv[4] = {B4.x, B4.y, B4.z, B4.w};
                    const float Cv[4] = {C4.x, C4.y, C4.z, C4.w};
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int i = q * 4 + j;
                        h[i] = fmaf(ex2(d.x * A2[i]), h[i], d.y * Bv[j]);
                        if (!LOCAL) acc = fmaf(Cv[j], h[i], acc);
                    }
                }
                y[u] = acc;
                if (LOCAL) total += d.x;
            }
            if (!LOCAL) {
                // lanes of one channel: each ends with the sum of one of the S tokens
                const int u = u0 + lane_sum<S, S, CW>(y, lane);
                const int t = t0 + u;
                if (live && t < end) {
                    float v = y[0];
                    if (a.Dskip) v = fmaf(a.Dskip[c], to_f(X.at(p.b, t)[c]), v);
                    if (a.z.p) {
                        const float z = to_f(Z.at(p.b, t)[c]);
                        v *= z * sigmoid_f<IO>(z);
                    }
                    Y.at(p.b, t)[c] = from_f<IO>(v);
                }
            }
        }
    }
    if (!LOCAL)       // rows past the sequence's length
        for (int t = max(p.t0, p.len); t < p.t1; t++)
            for (int k = threadIdx.x; k < p.nc; k += SH::THREADS)
                Y.at(p.b, t)[p.c0 + k] = from_f<IO>(0.f);
    if (live) {
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const int n = s * NT + i;
            if (n < a.N) {
                if (LOCAL)
                    a.hseg[rowseg + n] = h[i];
                else if (p.seg == a.nseg - 1)
                    a.h[row + n] = h[i];
            }
        }
        if (LOCAL && s == 0) a.dsum[((long long)p.b * a.nseg + p.seg) * a.D + c] = total;
    }
}

// Chains the segments: entry state of segment k + 1 = e^{A sum delta_k} (entry of k) + own end of k.
__global__ void __launch_bounds__(256) sel_chain_kernel(const SelArgs a) {
    const long long per = (long long)a.D * a.N;
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= per * a.batch) return;
    const int b = (int)(i / per);
    const long long dn = i - b * per;
    const int d = (int)(dn / a.N);
    const float A2 = a.A[dn] * kLog2e;
    float h = a.h[i];
    for (int k = 0; k < a.nseg; k++) {
        float* at = a.hseg + ((long long)b * a.nseg + k) * per + dn;
        const float own = *at;
        *at = h;
        h = fmaf(ex2(A2 * a.dsum[((long long)b * a.nseg + k) * a.D + d]), h, own);
    }
}

// One token: SL lanes share a channel, each taking 4 states at a time.
template <typename IO, int SL, bool WIDE>
__global__ void __launch_bounds__(128) sel_step_kernel(const SelArgs a) {
    const long long cell = (blockIdx.x * 128ll + threadIdx.x) / SL;
    const int s = threadIdx.x % SL;
    const bool live = cell < (long long)a.batch * a.D;
    const int b = live ? (int)(cell / a.D) : 0;
    const int c = live ? (int)(cell - (long long)b * a.D) : 0;
    const int g = c / (a.D / a.G);
    const IO* px = static_cast<const IO*>(a.x.p) + b * a.x.bs;
    const IO* pb = static_cast<const IO*>(a.B.p) + b * a.B.bs + (long long)g * a.N;
    const IO* pc = static_cast<const IO*>(a.C.p) + b * a.C.bs + (long long)g * a.N;
    const float x = to_f(px[c]);
    const float delta = sel_delta(to_f((static_cast<const IO*>(a.dt.p) + b * a.dt.bs)[c]),
                                  a.dt_bias ? a.dt_bias[c] : 0.f, a.softplus);
    float* hr = a.h + ((long long)b * a.D + c) * a.N;
    const float* Ar = a.A + (long long)c * a.N;
    float acc = 0.f;
    for (int n = s * 4; n < a.N; n += SL * 4) {
        float h[4], A[4], Bv[4], Cv[4];
        const int m = live ? min(4, a.N - n) : 0;
        Vec<float, 4>::load<WIDE>(h, hr + n, m);
        Vec<float, 4>::load<WIDE>(A, Ar + n, m);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            Bv[j] = j < m ? to_f(pb[n + j]) : 0.f;
            Cv[j] = j < m ? to_f(pc[n + j]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            h[j] = fmaf(ex2(delta * (A[j] * kLog2e)), h[j], delta * x * Bv[j]);
            acc = fmaf(Cv[j], h[j], acc);
        }
        Vec<float, 4>::store<WIDE>(h, hr + n, m);
    }
#pragma unroll
    for (int o = SL / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (live && s == 0) {
        if (a.Dskip) acc = fmaf(a.Dskip[c], x, acc);
        if (a.z.p) {
            const float z = to_f((static_cast<const IO*>(a.z.p) + b * a.z.bs)[c]);
            acc *= z * sigmoid_f<IO>(z);
        }
        (static_cast<IO*>(a.y.p) + b * a.y.bs)[c] = from_f<IO>(acc);
    }
}

template <typename IO, typename SH>
cudaError_t fwd_t(const SelArgs& a, cudaStream_t s) {
    const unsigned grid = (unsigned)((long long)sel_tiles(a.D, a.G, SH::CB) * a.nseg * a.batch);
    if (a.nseg > 1) {
        sel_scan_kernel<IO, SH, true><<<grid, SH::THREADS, 0, s>>>(a);
        const long long n = (long long)a.batch * a.D * a.N;
        sel_chain_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a);
    }
    sel_scan_kernel<IO, SH, false><<<grid, SH::THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t fwd_by_n(const SelArgs& a, cudaStream_t s) {
    if (a.N <= 4) return fwd_t<IO, SelShape<4, 1, 4>>(a, s);
    if (a.N <= 8) return fwd_t<IO, SelShape<8, 1, 4>>(a, s);
    if (a.N <= 16) return fwd_t<IO, SelShape<8, 2, 4>>(a, s);
    if (a.N <= 32) return fwd_t<IO, SelShape<8, 4, 4>>(a, s);
    if (a.N <= 64) return fwd_t<IO, SelShape<8, 8, 4>>(a, s);
    if (a.N <= 128) return fwd_t<IO, SelShape<8, 16, 4>>(a, s);
    return fwd_t<IO, SelShape<16, 16, 4, 16>>(a, s);
}

template <typename IO, bool WIDE>
cudaError_t step_t(const SelArgs& a, cudaStream_t s) {
    const long long cells = (long long)a.batch * a.D;
    auto blocks = [&](int sl) { return (unsigned)((cells * sl + 127) / 128); };
    if (a.N <= 4)
        sel_step_kernel<IO, 1, WIDE><<<blocks(1), 128, 0, s>>>(a);
    else if (a.N <= 8)
        sel_step_kernel<IO, 2, WIDE><<<blocks(2), 128, 0, s>>>(a);
    else if (a.N <= 16)
        sel_step_kernel<IO, 4, WIDE><<<blocks(4), 128, 0, s>>>(a);
    else
        sel_step_kernel<IO, 8, WIDE><<<blocks(8), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Channels of a forward block, by the number of states (fwd_by_n).
static int sel_fwd_channels(int N) {
    int s = 1;
    while (s < 16 && s * 8 < N) s *= 2;
    return 128 / s;
}

// Segments: none while the blocks of one pass over the channels give every SM sub-partition a
// warp to itself; else as many as bring four warps to each, of at least four tiles of tokens.
int sel_fwd_segments(int batch, int T, int D, int G, int N, int* seg) {
    const int tiles = (T + kSelTile - 1) / kSelTile;
    const long long blocks = (long long)batch * sel_tiles(D, G, sel_fwd_channels(N));
    int n = 1;
    if (blocks < 148 && tiles >= 8) {
        n = (int)((148 * 4 + blocks - 1) / blocks);
        if (n > tiles / 4) n = tiles / 4;
    }
    const int per = (tiles + n - 1) / n;
    *seg = per * kSelTile;
    return (tiles + per - 1) / per;
}

size_t sel_fwd_workspace(int batch, int T, int D, int G, int N) {
    int seg;
    const int n = sel_fwd_segments(batch, T, D, G, N, &seg);
    return n > 1 ? sizeof(float) * (size_t)batch * n * D * (N + 1) : 0;
}

cudaError_t launch_sel_fwd(const SelArgs& a, int io_dtype, cudaStream_t s) {
    return io_dtype == M3_BF16 ? fwd_by_n<__nv_bfloat16>(a, s) : fwd_by_n<float>(a, s);
}

cudaError_t launch_sel_step(const SelArgs& a, int io_dtype, cudaStream_t s) {
    if (io_dtype == M3_BF16)
        return a.wide ? step_t<__nv_bfloat16, true>(a, s) : step_t<__nv_bfloat16, false>(a, s);
    return a.wide ? step_t<float, true>(a, s) : step_t<float, false>(a, s);
}

}  // namespace m3
