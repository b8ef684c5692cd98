// sel_bwd.cu -- backward of the selective scan (m3_sel_bwd).
//
// With e_t = dy_t SiLU(z_t) the adjoint of the state runs back in time,
//   lam_t = C_t e_t + a_{t+1} lam_{t+1},      a_t = e^{delta_t A},
// and each token gives
//   dC_t[n] = sum_c h_t e_t;   dB_t[n] = sum_c lam_t delta_t x_t;   dx_t = delta_t sum_n lam_t B_t + D e_t;
//   ddelta_t = x_t sum_n lam_t B_t + sum_n A lam_t a_t h_{t-1};     dA = sum_t delta_t lam_t a_t h_{t-1}.
// Both recurrences are affine in the state that enters a segment, so every segment of the
// sequence works by itself once its entry state and its leaving adjoint are known:
//   1. sel_bwd_local_kernel: each segment's own end state (from 0) and own entry adjoint (to 0);
//   2. sel_bwd_chain_kernel: entry states forward and leaving adjoints backward over segments;
//   3. sel_bwd_kernel: the segment again, K tokens at a time from the last: the K states and
//      decays of a piece are recomputed into registers from a state kept in shared memory, then
//      walked backward;
//   4. the shares of the sums over channel blocks and over segments are added in a fixed order.
#include "block_internal.h"
#include "sel_tile.cuh"

namespace m3 {

namespace {

template <int NT_, int S_, int WARPS_, int L_, int K_>
struct BwdShape : SelShape<NT_, S_, WARPS_, L_> {
    using Base = SelShape<NT_, S_, WARPS_, L_>;
    static constexpr int L = L_, K = K_;      // tokens of a segment, of a piece
    // shared memory, in floats
    static constexpr int O_BC = 0;                                      // [L][2][NP]
    static constexpr int O_DELTA = O_BC + L * 2 * Base::NP;             // [L][CB]
    static constexpr int O_DX = O_DELTA + L * Base::CB;                 // [L][CB] delta x
    static constexpr int O_E = O_DX + L * Base::CB;                     // [L][CB]
    static constexpr int O_CK = O_E + L * Base::CB;                     // [L / K][CB][NP]
    static constexpr int O_RED = O_CK + L / K * Base::CB * Base::NP;    // [WARPS][K][2 NP]
    static constexpr int LOCAL_BYTES = 4 * O_CK;
    static constexpr int BYTES = 4 * (O_RED + Base::WARPS * K * 2 * Base::NP);
};

// delta, delta x and e = dy SiLU(z) of the segment's tokens (zero past the end), and B and C
template <typename IO, typename SH>
__device__ __forceinline__ void bwd_stage(const SelArgs& a, const SelPlace& p, int end, float* sm) {
    constexpr int L = SH::L, CB = SH::CB;
    const Rows<const IO> X{static_cast<const IO*>(a.x.p), a.x.bs, a.x.ts};
    const Rows<const IO> DT{static_cast<const IO*>(a.dt.p), a.dt.bs, a.dt.ts};
    const Rows<const IO> Z{static_cast<const IO*>(a.z.p), a.z.bs, a.z.ts};
    const Rows<const IO> DY{static_cast<const IO*>(a.dy.p), a.dy.bs, a.dy.ts};
    sel_stage_bc<IO, SH::NP, L, SH::THREADS>(a, p, p.t0, end, sm + SH::O_BC);
#pragma unroll 2
    for (int i = threadIdx.x; i < L * CB; i += SH::THREADS) {
        const int k = i % CB, t = p.t0 + i / CB;
        float delta = 0.f, dx = 0.f, e = 0.f;
        if (t < end && k < p.nc) {
            const int c = p.c0 + k;
            delta = sel_delta(to_f(DT.at(p.b, t)[c]), a.dt_bias ? a.dt_bias[c] : 0.f, a.softplus);
            dx = delta * to_f(X.at(p.b, t)[c]);
            e = to_f(DY.at(p.b, t)[c]);
            if (a.z.p) {
                const float z = to_f(Z.at(p.b, t)[c]);
                e *= z * sigmoid_f<IO>(z);
            }
        }
        sm[SH::O_DELTA + i] = delta;
        sm[SH::O_DX + i] = dx;
        sm[SH::O_E + i] = e;
    }
}

template <int NT>
__device__ __forceinline__ void load_states(float (&v)[NT], const float* p) {
#pragma unroll
    for (int q = 0; q < NT / 4; q++) {
        const float4 f = reinterpret_cast<const float4*>(p)[q];
        v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
    }
}

template <typename IO, typename SH>
__global__ void __launch_bounds__(SH::THREADS) sel_bwd_local_kernel(const SelArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int NT = SH::NT, CW = SH::CW, CB = SH::CB, NP = SH::NP;
    const SelPlace p = sel_place(a, CB);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int cl = wid * CW + lane % CW, s = lane / CW, c = p.c0 + cl;
    const bool live = cl < p.nc;
    const int end = min(p.t1, p.len);
    bwd_stage<IO, SH>(a, p, end, sm);
    float h[NT], g[NT], P[NT], A2[NT];
#pragma unroll
    for (int i = 0; i < NT; i++) {
        const int n = s * NT + i;
        A2[i] = live && n < a.N ? a.A[(long long)c * a.N + n] * kLog2e : 0.f;
        h[i] = g[i] = 0.f;
        P[i] = 1.f;
    }
    __syncthreads();
    float total = 0.f;
#pragma unroll 4
    for (int u = 0; u < end - p.t0; u++) {
        const float delta = sm[SH::O_DELTA + u * CB + cl], dx = sm[SH::O_DX + u * CB + cl],
                    e = sm[SH::O_E + u * CB + cl];
        float B[NT], C[NT];
        load_states(B, sm + SH::O_BC + u * 2 * NP + s * NT);
        load_states(C, sm + SH::O_BC + (u * 2 + 1) * NP + s * NT);
        total += delta;
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const float d = ex2(delta * A2[i]);
            h[i] = fmaf(d, h[i], dx * B[i]);
            P[i] *= d;                      // decay from the entry through this token
            g[i] = fmaf(P[i], C[i] * e, g[i]);
        }
    }
    if (live) {
        const long long row = (((long long)p.b * a.nseg + p.seg) * a.D + c) * a.N;
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const int n = s * NT + i;
            if (n < a.N) {
                a.hseg[row + n] = h[i];
                a.gseg[row + n] = g[i];
            }
        }
        if (s == 0) a.dsum[((long long)p.b * a.nseg + p.seg) * a.D + c] = total;
    }
}

// Entry states over the segments in order, leaving adjoints over them in reverse; dh is what
// leaves before the first.
__global__ void __launch_bounds__(128) sel_bwd_chain_kernel(const SelArgs a) {
    const long long per = (long long)a.D * a.N;
    const long long i = blockIdx.x * 128ll + threadIdx.x;
    if (i >= per * a.batch) return;
    const int b = (int)(i / per);
    const long long dn = i - b * per;
    const int d = (int)(dn / a.N);
    const float A2 = a.A[dn] * kLog2e;
    float* hs = a.hseg + (long long)b * a.nseg * per + dn;
    float* gs = a.gseg + (long long)b * a.nseg * per + dn;
    const float* ds = a.dsum + (long long)b * a.nseg * a.D + d;
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
    float g = a.dhT ? a.dhT[i] : 0.f;
    for (int k0 = a.nseg - 1; k0 >= 0; k0 -= U) {
        float own[U], dec[U];
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 - u >= 0) {
                own[u] = gs[(k0 - u) * per];
                dec[u] = ds[(long long)(k0 - u) * a.D];
            }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 - u >= 0) {
                gs[(k0 - u) * per] = g;
                g = fmaf(ex2(A2 * dec[u]), g, own[u]);
            }
    }
    if (a.dh) a.dh[i] = g;
}

template <typename IO, typename SH>
__global__ void __launch_bounds__(SH::THREADS) sel_bwd_kernel(const SelArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int NT = SH::NT, S = SH::S, CW = SH::CW, CB = SH::CB, NP = SH::NP, K = SH::K;
    constexpr int WARPS = SH::WARPS;
    const SelPlace p = sel_place(a, CB);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int cl = wid * CW + lane % CW, s = lane / CW, c = p.c0 + cl;
    const bool live = cl < p.nc;
    const int end = min(p.t1, p.len);
    const int tile = blockIdx.x % sel_tiles(a.D, a.G, CB), tiles = sel_tiles(a.D, a.G, CB);
    bwd_stage<IO, SH>(a, p, end, sm);

    const Rows<const IO> X{static_cast<const IO*>(a.x.p), a.x.bs, a.x.ts};
    const Rows<const IO> DT{static_cast<const IO*>(a.dt.p), a.dt.bs, a.dt.ts};
    const Rows<const IO> Z{static_cast<const IO*>(a.z.p), a.z.bs, a.z.ts};
    const Rows<const IO> DY{static_cast<const IO*>(a.dy.p), a.dy.bs, a.dy.ts};
    const Rows<IO> DX{static_cast<IO*>(a.dx.p), a.dx.bs, a.dx.ts};
    const Rows<IO> DDT{static_cast<IO*>(a.ddt.p), a.ddt.bs, a.ddt.ts};
    const Rows<IO> DZ{static_cast<IO*>(a.dz.p), a.dz.bs, a.dz.ts};

    float h[NT], lam[NT], A2[NT], dA[NT];
    const long long row = (((long long)p.b * a.nseg + p.seg) * a.D + c) * a.N;
#pragma unroll
    for (int i = 0; i < NT; i++) {
        const int n = s * NT + i;
        const bool on = live && n < a.N;
        A2[i] = on ? a.A[(long long)c * a.N + n] * kLog2e : 0.f;
        h[i] = on ? a.hseg[row + n] : 0.f;
        lam[i] = on ? a.gseg[row + n] : 0.f;
        dA[i] = 0.f;
    }
    const float skip = live && a.Dskip ? a.Dskip[c] : 0.f;
    const float bias = live && a.dt_bias ? a.dt_bias[c] : 0.f;
    float dD = 0.f, dbias = 0.f;
    __syncthreads();

    const int count = end > p.t0 ? end - p.t0 : 0;
    const int pieces = (count + K - 1) / K;
    // the state before each piece (a thread reads back its own values only)
    for (int j = 0; j < pieces; j++) {
        float4* ck = reinterpret_cast<float4*>(sm + SH::O_CK + (j * CB + cl) * NP + s * NT);
#pragma unroll
        for (int q = 0; q < NT / 4; q++)
            ck[q] = make_float4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
        if (j + 1 < pieces) {
#pragma unroll
            for (int k = 0; k < K; k++) {
                const int u = j * K + k;
                const float delta = sm[SH::O_DELTA + u * CB + cl], dx = sm[SH::O_DX + u * CB + cl];
                float B[NT];
                load_states(B, sm + SH::O_BC + u * 2 * NP + s * NT);
#pragma unroll
                for (int i = 0; i < NT; i++) h[i] = fmaf(ex2(delta * A2[i]), h[i], dx * B[i]);
            }
        }
    }
    for (int j = pieces - 1; j >= 0; j--) {
        float hp[K][NT], dec[K][NT];     // state before token k, decay of token k
        load_states(h, sm + SH::O_CK + (j * CB + cl) * NP + s * NT);
#pragma unroll
        for (int k = 0; k < K; k++) {
            const int u = j * K + k;     // zero past the end: the state stays
            const float delta = sm[SH::O_DELTA + u * CB + cl], dx = sm[SH::O_DX + u * CB + cl];
            float B[NT];
            load_states(B, sm + SH::O_BC + u * 2 * NP + s * NT);
#pragma unroll
            for (int i = 0; i < NT; i++) {
                hp[k][i] = h[i];
                dec[k][i] = ex2(delta * A2[i]);
                h[i] = fmaf(dec[k][i], h[i], dx * B[i]);
            }
        }
        float yv[K], lb[K], la[K];       // sums over the states: C h, lam B, A2 lam a h_before
#pragma unroll
        for (int k = K - 1; k >= 0; k--) {
            const int u = j * K + k;
            const float delta = sm[SH::O_DELTA + u * CB + cl], dx = sm[SH::O_DX + u * CB + cl],
                        e = sm[SH::O_E + u * CB + cl];
            float B[NT], C[NT], over[2 * NT];
            load_states(B, sm + SH::O_BC + u * 2 * NP + s * NT);
            load_states(C, sm + SH::O_BC + (u * 2 + 1) * NP + s * NT);
            yv[k] = lb[k] = la[k] = 0.f;
#pragma unroll
            for (int i = 0; i < NT; i++) {
                const float now = k == K - 1 ? h[i] : hp[k == K - 1 ? k : k + 1][i];
                lam[i] = fmaf(C[i], e, lam[i]);
                over[i] = lam[i] * dx;
                over[NT + i] = now * e;
                yv[k] = fmaf(C[i], now, yv[k]);
                lb[k] = fmaf(lam[i], B[i], lb[k]);
                lam[i] *= dec[k][i];
                const float q = lam[i] * hp[k][i];
                la[k] = fmaf(q, A2[i], la[k]);
                dA[i] = fmaf(q, delta, dA[i]);
            }
            // over the warp's channels
            const int off = lane_sum<2 * NT, CW, 1>(over, lane);
            constexpr int HOLD = 2 * NT > CW ? 2 * NT / CW : 1, SPARE = CW > 2 * NT ? CW / (2 * NT) : 1;
            if (lane % SPARE == 0) {
                float* red = sm + SH::O_RED + (wid * K + k) * 2 * NP;
#pragma unroll
                for (int i = 0; i < HOLD; i++) {
                    const int v = off + i;
                    red[(v / NT) * NP + s * NT + v % NT] = over[i];
                }
            }
        }
        // over the channel's lanes: each ends with the sums of K / S tokens
        const int off = lane_sum<K, S, CW>(yv, lane);
        lane_sum<K, S, CW>(lb, lane);
        lane_sum<K, S, CW>(la, lane);
        constexpr int HOLD = K > S ? K / S : 1, SPARE = S > K ? S / K : 1;
        if (live && s % SPARE == 0) {
#pragma unroll
            for (int i = 0; i < HOLD; i++) {
                const int u = j * K + off + i, t = p.t0 + u;
                if (t >= end) continue;
                const float delta = sm[SH::O_DELTA + u * CB + cl], e = sm[SH::O_E + u * CB + cl];
                const float x = to_f(X.at(p.b, t)[c]);
                if (a.z.p) {
                    const float z = to_f(Z.at(p.b, t)[c]), dy = to_f(DY.at(p.b, t)[c]);
                    const float sg = sigmoid_f<IO>(z);
                    const float y = fmaf(skip, x, yv[i]);
                    DZ.at(p.b, t)[c] = from_f<IO>(dy * y * sg * (1.f + z * (1.f - sg)));
                }
                float ddt = fmaf(x, lb[i], la[i] * kLn2);
                if (a.softplus) ddt *= sigmoid_f<IO>(to_f(DT.at(p.b, t)[c]) + bias);
                DX.at(p.b, t)[c] = from_f<IO>(fmaf(delta, lb[i], skip * e));
                DDT.at(p.b, t)[c] = from_f<IO>(ddt);
                dD = fmaf(e, x, dD);
                dbias += ddt;
            }
        }
        // over the block's warps, to the workspace
        __syncthreads();
        for (int i = threadIdx.x; i < K * 2 * NP; i += SH::THREADS) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; w++) v += sm[SH::O_RED + w * K * 2 * NP + i];
            const int t = p.t0 + j * K + i / (2 * NP);
            if (t < end)
                a.pBC[(((long long)p.b * a.T + t) * tiles + tile) * 2 * NP + i % (2 * NP)] = v;
        }
        __syncthreads();
    }
    // rows past the sequence's length
    for (int t = max(p.t0, p.len); t < p.t1; t++)
        for (int k = threadIdx.x; k < p.nc; k += SH::THREADS) {
            DX.at(p.b, t)[p.c0 + k] = from_f<IO>(0.f);
            DDT.at(p.b, t)[p.c0 + k] = from_f<IO>(0.f);
            if (a.z.p) DZ.at(p.b, t)[p.c0 + k] = from_f<IO>(0.f);
        }
#pragma unroll
    for (int o = CW; o < 32; o *= 2) {
        dD += __shfl_xor_sync(0xffffffffu, dD, o);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, o);
    }
    if (live) {
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const int n = s * NT + i;
            if (n < a.N) a.pA[row + n] = dA[i];
        }
        if (s == 0) {
            float* q = a.pD + ((long long)p.b * a.nseg + p.seg) * 2 * a.D + c;
            q[0] = dD;
            q[a.D] = dbias;
        }
    }
}

// dB and dC of one (row, group): the shares of the group's channel blocks, in order.
template <typename IO>
__global__ void __launch_bounds__(256) sel_bwd_bc_kernel(const SelArgs a, int NP, int tiles) {
    const int per_g = tiles / a.G;
    const long long total = (long long)a.batch * a.T * a.G * 2 * a.N;
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= total) return;
    const int n = (int)(i % a.N);
    long long r = i / a.N;
    const int which = (int)(r & 1);
    r >>= 1;
    const int g = (int)(r % a.G);
    r /= a.G;
    const int t = (int)(r % a.T), b = (int)(r / a.T);
    float v = 0.f;
    if (t < tokens_of(a.seqlens, b, a.T)) {
        const float* q = a.pBC + ((r * tiles + (long long)g * per_g) * 2 + which) * NP + n;
#pragma unroll 4
        for (int k = 0; k < per_g; k++) v += q[(long long)k * 2 * NP];
    }
    const long long at = (long long)g * a.N + n;
    if (which)
        static_cast<IO*>(a.dC.p)[b * a.dC.bs + t * a.dC.ts + at] = from_f<IO>(v);
    else
        static_cast<IO*>(a.dB.p)[b * a.dB.bs + t * a.dB.ts + at] = from_f<IO>(v);
}

// Column sums of rows x cols shares: a block per 32 columns, a warp every eighth row.
__global__ void __launch_bounds__(256) sel_bwd_sum_kernel(const float* part, int rows,
                                                          long long stride, long long cols,
                                                          float* out) {
    __shared__ float sm[8][33];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const long long c = blockIdx.x * 32ll + lane;
    float s = 0.f;
    if (c < cols)
        for (int r = wid; r < rows; r += 8) s += part[r * stride + c];
    sm[wid][lane] = s;
    __syncthreads();
    if (wid == 0 && c < cols) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) v += sm[i][lane];
        out[c] = v;
    }
}

template <typename IO, typename SH>
cudaError_t bwd_t(const SelArgs& a, cudaStream_t s) {
    const int tiles = sel_tiles(a.D, a.G, SH::CB);
    const unsigned grid = (unsigned)((long long)tiles * a.nseg * a.batch);
    cudaError_t e = cudaFuncSetAttribute(sel_bwd_local_kernel<IO, SH>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, SH::LOCAL_BYTES);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(sel_bwd_kernel<IO, SH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SH::BYTES);
    if (e != cudaSuccess) return e;
    sel_bwd_local_kernel<IO, SH><<<grid, SH::THREADS, SH::LOCAL_BYTES, s>>>(a);
    const long long states = (long long)a.D * a.N;
    sel_bwd_chain_kernel<<<(unsigned)((states * a.batch + 127) / 128), 128, 0, s>>>(a);
    sel_bwd_kernel<IO, SH><<<grid, SH::THREADS, SH::BYTES, s>>>(a);
    const long long bc = (long long)a.batch * a.T * a.G * 2 * a.N;
    sel_bwd_bc_kernel<IO><<<(unsigned)((bc + 255) / 256), 256, 0, s>>>(a, SH::NP, tiles);
    const int rows = a.batch * a.nseg;
    sel_bwd_sum_kernel<<<(unsigned)((states + 31) / 32), 256, 0, s>>>(a.pA, rows, states, states, a.dA);
    if (a.dD)
        sel_bwd_sum_kernel<<<(a.D + 31) / 32, 256, 0, s>>>(a.pD, rows, 2ll * a.D, a.D, a.dD);
    if (a.ddt_bias)
        sel_bwd_sum_kernel<<<(a.D + 31) / 32, 256, 0, s>>>(a.pD + a.D, rows, 2ll * a.D, a.D, a.ddt_bias);
    return cudaGetLastError();
}

template <typename IO, typename F>
cudaError_t by_n(int N, F f) {
    if (N <= 4) return f(BwdShape<4, 1, 2, 64, 8>{});
    if (N <= 8) return f(BwdShape<4, 2, 4, 64, 8>{});
    if (N <= 16) return f(BwdShape<4, 4, 8, 64, 8>{});
    if (N <= 32) return f(BwdShape<4, 8, 8, 64, 8>{});
    if (N <= 64) return f(BwdShape<8, 8, 8, 32, 4>{});
    if (N <= 128) return f(BwdShape<8, 16, 8, 32, 4>{});
    return f(BwdShape<8, 32, 8, 32, 4>{});
}

}  // namespace

size_t sel_bwd_plan(SelArgs* a, int io_dtype, char* ws) {
    int NP = 0, CB = 0;
    by_n<float>(a->N, [&](auto sh) {
        using SH = decltype(sh);
        a->seg = SH::L;
        NP = SH::NP;
        CB = SH::CB;
        return cudaSuccess;
    });
    a->nseg = (a->T + a->seg - 1) / a->seg;
    const size_t runs = (size_t)a->batch * a->nseg, states = (size_t)a->D * a->N;
    const size_t tiles = sel_tiles(a->D, a->G, CB);
    size_t at = 0;
    auto take = [&](size_t floats) {
        float* p = reinterpret_cast<float*>(ws + at);
        at += (floats * sizeof(float) + 255) / 256 * 256;
        return p;
    };
    a->hseg = take(runs * states);
    a->gseg = take(runs * states);
    a->pA = take(runs * states);
    a->dsum = take(runs * a->D);
    a->pD = take(runs * 2 * a->D);
    a->pBC = take((size_t)a->batch * a->T * tiles * 2 * NP);
    return at;
}

cudaError_t launch_sel_bwd(const SelArgs& a, int io_dtype, cudaStream_t s) {
    if (io_dtype == M3_BF16)
        return by_n<__nv_bfloat16>(a.N, [&](auto sh) { return bwd_t<__nv_bfloat16, decltype(sh)>(a, s); });
    return by_n<float>(a.N, [&](auto sh) { return bwd_t<float, decltype(sh)>(a, s); });
}

}  // namespace m3
