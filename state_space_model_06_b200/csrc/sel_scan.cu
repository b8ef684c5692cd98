// sel_scan.cu -- selective scan with a diagonal state per channel: prompts and single tokens
// (m3_sel_fwd, m3_sel_step).
//
//   h_t[c][n] = e^{delta_t[c] A[c][n]} h_{t-1}[c][n] + delta_t[c] x_t[c] B_t[n]
//   y_t[c]    = (sum_n C_t[n] h_t[c][n] + D[c] x_t[c]) SiLU(z_t[c])
//
// Every (token, channel, state) needs an exponential, and every channel and state has a decay of
// its own, so the chunked matrix form of the mixer's scan does not apply: the work is one ex2 and
// four fp32 operations a cell on registers.  The exponential unit (16 a clock and SM) bounds it:
// 8 x 2048 tokens of 4096 channels of 16 states need 1.34e9 of them with softplus and gate, 298 us,
// where the memory would take 83.  The prompt kernel takes 503 us there (the unit 58 % busy, issue
// slots 68 %, shared memory 69 %): 189 instructions for 32 channel-tokens of 16 states, of which the
// recurrence itself is half; the rest is the step and the gate (49), the sum over the lanes of a
// channel (28) and the staging.  What was measured and not kept: two, four or eight tokens' decays
// ahead of the chain through the states (no change), a quarter to a half of the exponentials by a
// polynomial on the FMA pipe (3 to 16 % slower: issue slots are short too), one channel a lane
// (650 us: the broadcast reads of B and C fill the shared memory), 8 and 16 states a lane (650 to
// 800 us: too few warps).
#include "block_internal.h"
#include "sel_tile.cuh"

namespace m3 {

namespace {

// One block: CB channels of one group over one segment, L tokens at a time.  While a tile is
// worked on, the next one's x, dt, z, B and C are on their way to the other half of the raw
// buffers.  Of each tile delta, delta x and the fp32 B and C are laid out first, once for all
// the lanes that share them.
// LOCAL: the segment's own end state from no entry state, and its sum of delta (no y).
// Otherwise the outputs, from the entry state in hseg (segmented) or in h.
//
// A lane holds NT states of two neighbouring channels.  What limits the choice: the exponential
// unit takes 8 cycles for 32 of them (a channel-token of 16 states on 32 lanes: 170 cycles of a
// sub-partition with softplus and gate), a broadcast 16-byte read of B or C takes 4 cycles of the
// SM's shared memory however few lanes differ, and a warp alone cannot keep the exponential unit
// busy.  Two channels a lane halve the reads of B and C; four states a lane leave enough warps.
template <typename IO, typename SH>
struct FwdSmem {
    static constexpr int L = SH::L, CB = SH::CB;
    // B and C rows keep a multiple of 16 bytes
    static constexpr int NR = (SH::NP * (int)sizeof(IO) + 15) / 16 * 16 / (int)sizeof(IO);
    struct Raw {
        alignas(16) IO x[L][CB], dt[L][CB], z[L][CB], B[L][NR], C[L][NR];
    };
    Raw raw[2];
    alignas(16) float bc[L][2][SH::NP];
    alignas(16) float4 dd[L][CB / 2];     // of two channels: delta, delta, delta x, delta x
};

template <typename IO, typename SH, bool WIDE, bool LOCAL>
__global__ void __launch_bounds__(SH::THREADS) sel_scan_kernel(const SelArgs a) {
    constexpr int L = SH::L, NT = SH::NT, S = SH::S, CW = SH::CW, CB = SH::CB, NP = SH::NP;
    constexpr int THREADS = SH::THREADS;
    static_assert(L % S == 0, "");
    using Smem = FwdSmem<IO, SH>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const SelPlace p = sel_place(a, CB);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int pl = wid * CW + lane % CW;     // pair of channels within the block
    const int s = lane / CW;                 // which NT states
    const int c = p.c0 + 2 * pl;
    const int mine = min(max(p.nc - 2 * pl, 0), 2);     // channels of the pair that exist
    const int end = min(p.t1, p.len);

    auto request = [&](int t0, typename Smem::Raw& r) {
        const long long bn = (long long)p.g * a.N;
        stage_rows<IO, WIDE, L, CB, THREADS>(&r.x[0][0], a.x, p.b, p.c0, t0, end, p.nc);
        stage_rows<IO, WIDE, L, CB, THREADS>(&r.dt[0][0], a.dt, p.b, p.c0, t0, end, p.nc);
        if (!LOCAL && a.z.p)
            stage_rows<IO, WIDE, L, CB, THREADS>(&r.z[0][0], a.z, p.b, p.c0, t0, end, p.nc);
        if (WIDE && a.wide_bc) {
            stage_rows<IO, true, L, Smem::NR, THREADS>(&r.B[0][0], a.B, p.b, bn, t0, end, a.N);
            if (!LOCAL)
                stage_rows<IO, true, L, Smem::NR, THREADS>(&r.C[0][0], a.C, p.b, bn, t0, end, a.N);
        } else {
            stage_rows<IO, false, L, Smem::NR, THREADS>(&r.B[0][0], a.B, p.b, bn, t0, end, a.N);
            if (!LOCAL)
                stage_rows<IO, false, L, Smem::NR, THREADS>(&r.C[0][0], a.C, p.b, bn, t0, end, a.N);
        }
    };
    if (p.t0 < end) request(p.t0, sm.raw[0]);
    cp_async_commit();

    f2 h[2][NT / 2], A2[2][NT / 2];      // pairs of neighbouring states
    const long long row = ((long long)p.b * a.D + c) * a.N;
    const long long rowseg = (((long long)p.b * a.nseg + p.seg) * a.D + c) * a.N;
#pragma unroll
    for (int q = 0; q < 2; q++)
#pragma unroll
        for (int i = 0; i < NT / 2; i++) {
            float hv[2] = {0.f, 0.f}, av[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int n = s * NT + 2 * i + j;
                if (q < mine && n < a.N) {
                    av[j] = a.A[(long long)(c + q) * a.N + n] * kLog2e;
                    if (!LOCAL)
                        hv[j] = a.nseg > 1 ? a.hseg[rowseg + q * a.N + n] : a.h[row + q * a.N + n];
                }
            }
            A2[q][i] = pack2(av[0], av[1]);
            h[q][i] = pack2(hv[0], hv[1]);
        }
    float skip[2] = {0.f, 0.f};
    if (a.Dskip)
#pragma unroll
        for (int q = 0; q < 2; q++)
            if (q < mine) skip[q] = a.Dskip[c + q];
    // the pair of channels whose deltas this thread lays out
    const int kd = threadIdx.x % (CB / 2);
    float bias[2] = {0.f, 0.f};
    if (a.dt_bias)
#pragma unroll
        for (int q = 0; q < 2; q++)
            if (2 * kd + q < p.nc) bias[q] = a.dt_bias[p.c0 + 2 * kd + q];
    float total[2] = {0.f, 0.f};
    const Rows<IO> Y{static_cast<IO*>(a.y.p), a.y.bs, a.y.ts};

    int stage = 0;
    for (int t0 = p.t0; t0 < end; t0 += L, stage ^= 1) {
        cp_async_wait<0>();
        __syncthreads();     // this tile has arrived; the one before is done with
        const typename Smem::Raw& r = sm.raw[stage];
        if (t0 + L < end) request(t0 + L, sm.raw[stage ^ 1]);
        cp_async_commit();
#pragma unroll 4
        for (int i = threadIdx.x; i < L * NP; i += THREADS) {
            const int u = i / NP, n = i % NP;
            sm.bc[u][0][n] = n < a.N ? to_f(r.B[u][n]) : 0.f;
            if (!LOCAL) sm.bc[u][1][n] = n < a.N ? to_f(r.C[u][n]) : 0.f;
        }
#pragma unroll 4
        for (int u = threadIdx.x / (CB / 2); u < L; u += THREADS / (CB / 2)) {
            float2 delta = make_float2(0.f, 0.f), dx = delta;
            if (t0 + u < end) {
                const float2 dt = pair_of(&r.dt[u][2 * kd]), x = pair_of(&r.x[u][2 * kd]);
                delta.x = sel_delta(dt.x, bias[0], a.softplus);
                delta.y = sel_delta(dt.y, bias[1], a.softplus);
                dx.x = delta.x * x.x;
                dx.y = delta.y * x.y;
            }
            sm.dd[u][kd] = make_float4(delta.x, delta.y, dx.x, dx.y);
        }
        __syncthreads();
        const int count = min(L, end - t0);
        for (int u0 = 0; u0 < count; u0 += S) {
            float y[2 * S];
#pragma unroll
            for (int u = 0; u < S; u++) {
                const float4 d = sm.dd[u0 + u][pl];       // zero past the end: h stays
                const f2 delta[2] = {pack2(d.x, d.x), pack2(d.y, d.y)};
                const f2 dx[2] = {pack2(d.z, d.z), pack2(d.w, d.w)};
                f2 B[NT / 2], C[NT / 2], acc[2];
                load_pairs(B, &sm.bc[u0 + u][0][s * NT]);
                if (!LOCAL) load_pairs(C, &sm.bc[u0 + u][1][s * NT]);
#pragma unroll
                for (int i = 0; i < NT / 2; i++)
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        h[q][i] = fma2(ex2_2(mul2(delta[q], A2[q][i])), h[q][i], mul2(dx[q], B[i]));
                        if (!LOCAL)
                            acc[q] = i == 0 ? mul2(C[i], h[q][i]) : fma2(C[i], h[q][i], acc[q]);
                    }
                if (LOCAL) {
                    total[0] += d.x;
                    total[1] += d.y;
                } else {
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        float lo, hi;
                        unpack2(acc[q], lo, hi);
                        y[2 * u + q] = lo + hi;
                    }
                }
            }
            if (!LOCAL) {
                // lanes of one pair of channels: each ends with the sums of one of the S tokens
                const int u = u0 + lane_sum<2 * S, S, CW>(y, lane) / 2;
                const int t = t0 + u;
                if (mine && t < end) {
                    const float2 x = pair_of(&r.x[u][2 * pl]);
                    float v[2] = {y[0], y[1]};
                    if (a.Dskip) {      // no 0 * inf without D
                        v[0] = fmaf(skip[0], x.x, v[0]);
                        v[1] = fmaf(skip[1], x.y, v[1]);
                    }
                    if (a.z.p) {
                        const float2 z = pair_of(&r.z[u][2 * pl]);
                        v[0] *= z.x * sigmoid_f<IO>(z.x);
                        v[1] *= z.y * sigmoid_f<IO>(z.y);
                    }
                    Vec<IO, 2>::template store<WIDE>(v, Y.at(p.b, t) + c, mine);
                }
            }
        }
    }
    cp_async_wait<0>();
    if (!LOCAL)       // rows past the sequence's length
        for (int t = max(p.t0, p.len); t < p.t1; t++)
            for (int k = threadIdx.x; k < p.nc; k += THREADS)
                Y.at(p.b, t)[p.c0 + k] = from_f<IO>(0.f);
#pragma unroll
    for (int q = 0; q < 2; q++) {
        if (q >= mine) break;
#pragma unroll
        for (int i = 0; i < NT / 2; i++) {
            float hv[2];
            unpack2(h[q][i], hv[0], hv[1]);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int n = s * NT + 2 * i + j;
                if (n < a.N) {
                    if (LOCAL)
                        a.hseg[rowseg + q * a.N + n] = hv[j];
                    else if (p.seg == a.nseg - 1)
                        a.h[row + q * a.N + n] = hv[j];
                }
            }
        }
        if (LOCAL && s == 0) a.dsum[((long long)p.b * a.nseg + p.seg) * a.D + c + q] = total[q];
    }
}

// Chains the segments: entry state of segment k + 1 = e^{A sum delta_k} (entry of k) + own end of k.
__global__ void __launch_bounds__(128) sel_chain_kernel(const SelArgs a) {
    const long long per = (long long)a.D * a.N;
    const long long i = blockIdx.x * 128ll + threadIdx.x;
    if (i >= per * a.batch) return;
    const int b = (int)(i / per);
    const long long dn = i - b * per;
    const float A2 = a.A[dn] * kLog2e;
    float* hs = a.hseg + (long long)b * a.nseg * per + dn;
    const float* ds = a.dsum + (long long)b * a.nseg * a.D + (int)(dn / a.N);
    constexpr int U = 8;          // segments requested together
    float h = a.h[i];
    for (int k0 = 0; k0 < a.nseg; k0 += U) {
        float own[U], dec[U];
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 + u < a.nseg) {
                own[u] = hs[(k0 + u) * per];
                dec[u] = ds[(long long)(k0 + u) * a.D];
            }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 + u < a.nseg) {
                hs[(k0 + u) * per] = h;
                h = fmaf(ex2(A2 * dec[u]), h, own[u]);
            }
    }
}

// One token: SL lanes share a channel, each taking 4 states at a time.
template <typename IO>
struct alignas(4 * sizeof(IO)) Quad4 {
    IO v[4];
};

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

// One token for N = 4 SL up to 32 and rows on 16 bytes: SL lanes share a channel, four states
// each.  A warp takes 32 channels of one sequence: each lane loads and prepares one channel's x, dt
// and z; then SL turns go over 32 / SL channels each, whose states are one contiguous stretch of
// memory.  The state's bytes bound it: 26 us at 256 sequences of 4096 channels of 16 states, one call
// after another (5.5 TB/s), 23 alone in a graph.  There, warps that keep A over 2, 4, 8 sequences take 30, 28, 28 us: they need twice the
// registers, and half as many fit an SM.  Everything is asked for before anything is used: with D
// loaded where it is needed, behind the sums, it takes 27 us.
template <typename IO, int SL>
__global__ void __launch_bounds__(128) sel_step_rows_kernel(const SelArgs a) {
    const int lane = threadIdx.x & 31, k = lane / SL, s = lane % SL;
    constexpr int CW = 32 / SL;                       // channels of a turn
    const int per_g = a.D / a.G, tiles_g = (per_g + 31) / 32;
    const int tile = blockIdx.x * 4 + (threadIdx.x >> 5), b = blockIdx.y;
    if (tile >= tiles_g * a.G) return;
    const int g = tile / tiles_g, c0 = g * per_g + (tile - g * tiles_g) * 32;
    const int nc = min(32, (g + 1) * per_g - c0);     // channels of this warp
    const int own = CW * s + k;                       // the channel this lane prepares and writes
    const bool mine = own < nc;
    const int c = c0 + (mine ? own : 0);
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.Dskip ? a.Dskip[c] : 0.f;
    float* state = a.h + ((long long)b * a.D + c0) * (4 * SL) + 4 * lane;
    const float* rate = a.A + (long long)c0 * (4 * SL) + 4 * lane;
    float4 h[SL], A[SL];
#pragma unroll
    for (int i = 0; i < SL; i++) {
        h[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i * CW + k < nc) h[i] = *reinterpret_cast<const float4*>(state + i * 128);
    }
    const float x = to_f((static_cast<const IO*>(a.x.p) + b * a.x.bs)[c]);
    const float dt = to_f((static_cast<const IO*>(a.dt.p) + b * a.dt.bs)[c]);
    const float z = a.z.p ? to_f((static_cast<const IO*>(a.z.p) + b * a.z.bs)[c]) : 0.f;
    const long long at = (long long)g * a.N + 4 * s;
    const Quad4<IO> B4 = *reinterpret_cast<const Quad4<IO>*>(static_cast<const IO*>(a.B.p) + b * a.B.bs + at);
    const Quad4<IO> C4 = *reinterpret_cast<const Quad4<IO>*>(static_cast<const IO*>(a.C.p) + b * a.C.bs + at);
#pragma unroll
    for (int i = 0; i < SL; i++) {
        A[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i * CW + k < nc) {
            A[i] = *reinterpret_cast<const float4*>(rate + i * 128);
            A[i].x *= kLog2e; A[i].y *= kLog2e; A[i].z *= kLog2e; A[i].w *= kLog2e;
        }
    }
    float Bv[4], Cv[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        Bv[j] = to_f(B4.v[j]);
        Cv[j] = to_f(C4.v[j]);
    }
    const float delta = sel_delta(dt, bias, a.softplus), dx = delta * x;
    float y[SL];
#pragma unroll
    for (int i = 0; i < SL; i++) {
        // turn i works on channel i CW + k, which lane k SL + i of this warp prepared
        const float d = __shfl_sync(0xffffffffu, delta, k * SL + i);
        const float u = __shfl_sync(0xffffffffu, dx, k * SL + i);
        h[i].x = fmaf(ex2(d * A[i].x), h[i].x, u * Bv[0]);
        h[i].y = fmaf(ex2(d * A[i].y), h[i].y, u * Bv[1]);
        h[i].z = fmaf(ex2(d * A[i].z), h[i].z, u * Bv[2]);
        h[i].w = fmaf(ex2(d * A[i].w), h[i].w, u * Bv[3]);
        y[i] = fmaf(Cv[0], h[i].x, fmaf(Cv[1], h[i].y, fmaf(Cv[2], h[i].z, Cv[3] * h[i].w)));
        if (i * CW + k < nc) *reinterpret_cast<float4*>(state + i * 128) = h[i];
    }
    lane_sum<SL, SL, 1>(y, lane);      // lane k SL + i ends with channel i CW + k: its own
    if (mine) {
        float v = a.Dskip ? fmaf(skip, x, y[0]) : y[0];      // no 0 * inf without D
        if (a.z.p) v *= z * sigmoid_f<IO>(z);
        (static_cast<IO*>(a.y.p) + b * a.y.bs)[c] = from_f<IO>(v);
    }
}

template <typename IO, typename SH, bool WIDE>
cudaError_t fwd_w(const SelArgs& a, cudaStream_t s) {
    constexpr int bytes = (int)sizeof(FwdSmem<IO, SH>);
    static_assert(bytes <= 227 * 1024, "");
    const unsigned grid = (unsigned)((long long)sel_tiles(a.D, a.G, SH::CB) * a.nseg * a.batch);
    cudaError_t e = allow_smem(sel_scan_kernel<IO, SH, WIDE, false>, bytes);
    if (e != cudaSuccess) return e;
    if (a.nseg > 1) {
        e = allow_smem(sel_scan_kernel<IO, SH, WIDE, true>, bytes);
        if (e != cudaSuccess) return e;
        sel_scan_kernel<IO, SH, WIDE, true><<<grid, SH::THREADS, bytes, s>>>(a);
        const long long n = (long long)a.batch * a.D * a.N;
        sel_chain_kernel<<<(unsigned)((n + 127) / 128), 128, 0, s>>>(a);
    }
    sel_scan_kernel<IO, SH, WIDE, false><<<grid, SH::THREADS, bytes, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, typename SH>
cudaError_t fwd_t(const SelArgs& a, cudaStream_t s) {
    return a.wide ? fwd_w<IO, SH, true>(a, s) : fwd_w<IO, SH, false>(a, s);
}

// The lane shape of a forward call, by the number of states.  For up to 16 states: with the whole
// sequence in one piece the channels alone make the warps, so a lane holds two states (8 x 2048
// tokens of 4096 channels: four a lane take 9 % longer); segments bring as many warps as one likes, and
// four states a lane take fewer instructions (16384 tokens of 2048 channels: two a lane take 10 % longer).
template <typename F>
auto fwd_shape(int N, bool segments, F f) {
    if (N <= 4) return f(SelShape<2, 2, 2, 32>{});
    if (N <= 8) return f(SelShape<2, 4, 4, 32>{});
    if (N <= 16) return segments ? f(SelShape<4, 4, 4, 16>{}) : f(SelShape<2, 8, 4, 32>{});
    if (N <= 32) return f(SelShape<4, 8, 4, 16>{});
    if (N <= 64) return f(SelShape<8, 8, 4, 32>{});
    if (N <= 128) return f(SelShape<8, 16, 4, 32>{});
    return f(SelShape<16, 16, 4, 16>{});
}

template <typename IO, int SL>
cudaError_t step_rows_t(const SelArgs& a, cudaStream_t s) {
    sel_step_rows_kernel<IO, SL><<<dim3((sel_tiles(a.D, a.G, 32) + 3) / 4, a.batch), 128, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, bool WIDE>
cudaError_t step_t(const SelArgs& a, cudaStream_t s) {
    if (WIDE && a.step_rows) {
        if (a.N == 4) return step_rows_t<IO, 1>(a, s);
        if (a.N == 8) return step_rows_t<IO, 2>(a, s);
        if (a.N == 16) return step_rows_t<IO, 4>(a, s);
        if (a.N == 32) return step_rows_t<IO, 8>(a, s);
    }
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

// Segments.  A segmented call computes every decay twice (measured 1.75 times the work) and takes
// three launches instead of one, so it pays for more than about 128 tokens where the blocks of one
// pass would leave more than half of the GPU idle: then as many segments as fill it about twice (14
// blocks an SM: 391 us for 16384 tokens of 2048 channels, one call after another; 8 take 5 % longer),
// down to one tile of tokens each (3 x 509 tokens of 1001 channels, alone in a graph: 37 us, 39 with
// two tiles at least; 47 to 49 among other calls).
static int sel_fwd_most_segments(int batch, int T, int D, int G, int N) {
    auto blocks = [&](bool segments) {
        const int CB = fwd_shape(N, segments, [](auto sh) { return decltype(sh)::CB; });
        return (long long)batch * sel_tiles(D, G, CB);
    };
    const int tiles = (T + kSelTile - 1) / kSelTile;
    if (blocks(false) > 148 * 3 || tiles <= 4) return 1;
    const long long want = 148 * 14 / blocks(true);
    return want > tiles ? tiles : (int)want;
}
int sel_fwd_segments(int batch, int T, int D, int G, int N, int* seg) {
    const int n = sel_fwd_most_segments(batch, T, D, G, N), tiles = (T + kSelTile - 1) / kSelTile;
    const int per = (tiles + n - 1) / n;
    *seg = per * kSelTile;
    return (tiles + per - 1) / per;
}

static size_t sel_fwd_bytes(int n, int batch, int D, int N) {
    return n > 1 ? sizeof(float) * (size_t)batch * n * D * (N + 1) : 0;
}
size_t sel_fwd_workspace(int batch, int T, int D, int G, int N) {
    int seg;
    return sel_fwd_bytes(sel_fwd_segments(batch, T, D, G, N, &seg), batch, D, N);
}
// Whole tiles leave some lengths with fewer segments than shorter ones: the number before that
// grows with T.
size_t sel_fwd_most(int batch, int T, int D, int G, int N) {
    return sel_fwd_bytes(sel_fwd_most_segments(batch, T, D, G, N), batch, D, N);
}

cudaError_t launch_sel_fwd(const SelArgs& a, int io_dtype, cudaStream_t s) {
    return fwd_shape(a.N, a.nseg > 1, [&](auto sh) {
        using SH = decltype(sh);
        return io_dtype == M3_BF16 ? fwd_t<__nv_bfloat16, SH>(a, s) : fwd_t<float, SH>(a, s);
    });
}

cudaError_t launch_sel_step(const SelArgs& a, int io_dtype, cudaStream_t s) {
    if (io_dtype == M3_BF16)
        return a.wide ? step_t<__nv_bfloat16, true>(a, s) : step_t<__nv_bfloat16, false>(a, s);
    return a.wide ? step_t<float, true>(a, s) : step_t<float, false>(a, s);
}

}  // namespace m3
