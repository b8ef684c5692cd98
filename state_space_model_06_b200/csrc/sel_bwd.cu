// sel_bwd.cu -- backward of the selective scan (m3_sel_bwd).
//
// With e_t = dy_t SiLU(z_t) the adjoint of the state runs back in time,
//   lam_t = C_t e_t + a_{t+1} lam_{t+1},      a_t = e^{delta_t A},
// and each token gives
//   dC_t[n] = sum_c h_t e_t;   dB_t[n] = sum_c lam_t delta_t x_t;   dx_t = delta_t sum_n lam_t B_t + D e_t;
//   ddelta_t = x_t sum_n lam_t B_t + sum_n A lam_t a_t h_{t-1};     dA = sum_t delta_t lam_t a_t h_{t-1}.
// Both recurrences are affine in what enters a segment, so every segment of the sequence works by
// itself once its entry state and its leaving adjoint are known:
//   1. sel_bwd_local_kernel: each segment's own states at the ends of its tiles (from a zero entry)
//      and its own entry adjoint (from a zero leaving one);
//   2. sel_bwd_chain_kernel: entry states forward and leaving adjoints backward over segments;
//   3. sel_bwd_kernel: the segment's tiles again, from the last.  Within a tile the states before
//      every K tokens go to shared memory; then, K tokens at a time from the last, states and
//      decays are recomputed into registers and walked backward;
//   4. the shares of the sums over channel blocks and over segments are added in a fixed order.
// A tile's entry state is its segment's entry state decayed to the tile, plus the own state of
// step 1, so only whole segments are chained.
//
// As in the forward kernel a lane holds NT states of two neighbouring channels, as packed pairs
// of states: the sums over channels (dB, dC) then cross half as many lanes, and they are what
// would cost most (a value summed over 8 lanes takes 7/8 of a shuffle and four times that in
// other instructions).
//
// Three passes over the exponentials (one in step 1, two in step 3) take 0.36 ms of the exponential
// unit at 4 x 2048 tokens of 4096 channels of 16 states; it takes 1.19 ms in all (step 1 0.27, the
// chain 0.03, step 3 0.87, the sums 0.03).  Step 3 is short of issue slots and of warps to fill
// them: 532 instructions for 32 channel-tokens, of which a third is the walk itself, at 54 % of the
// slots with 12 warps an SM (168 registers; at 128 the spills cost 40 %, and
// decays recomputed instead of kept bring 16 warps and nothing: the instructions grow as much).  The first form (one channel
// a lane, scalar arithmetic) took 1.99 ms; what brought most were the tokens' values asked for before
// the piece that ends with them (0.38 ms) and the next tile's rows on their way during a tile (0.15).
#include "block_internal.h"
#include "sel_tile.cuh"

namespace m3 {

namespace {

template <int NT_, int S_, int WARPS_, int L_, int K_>
struct BwdShape : SelShape<NT_, S_, WARPS_, L_> {
    using Base = SelShape<NT_, S_, WARPS_, L_>;
    using Base::NT; using Base::WARPS; using Base::L; using Base::PB; using Base::CB;
    using Base::NP; using Base::THREADS;
    static constexpr int K = K_;                 // tokens of a piece
    // 168 registers a thread leave room for 12 warps an SM.  Shared memory admits as many in bf16 from
    // 5 to 64 states and in fp32 from 5 to 8; else 8 (fp32: 6) up to 4 states, 8 in fp32 from 9 on,
    // and above 64 states 8, above 128 four, where the limit brings no warp.
    static constexpr int MIN_BLOCKS = NT * K <= 16 ? 384 / THREADS : 1;
    static constexpr int LOCAL_BLOCKS = NT == 4 ? 640 / THREADS : 1;      // 96 registers, 20 warps
    // shared memory, in floats
    static constexpr int O_BC = 0;                              // [L][2][NP]
    static constexpr int O_DD = O_BC + L * 2 * NP;              // [L][PB] float4: delta, delta x of two channels
    static constexpr int O_E = O_DD + L * PB * 4;               // [L][PB] float2: e
    static constexpr int O_RAW = O_E + L * PB * 2;              // the next tile's rows, as they are
    static constexpr int RED = WARPS * K * 2 * NP;              // sums over channels, of a piece and the one before
    static constexpr int KEPT = L / K > 2 ? L / K - 2 : 1;      // states before pieces 1 .. L / K - 2
    template <typename IO>
    struct Raw {
        static constexpr int NR = (NP * (int)sizeof(IO) + 15) / 16 * 16 / (int)sizeof(IO);
        alignas(16) IO x[L][CB], dt[L][CB], z[L][CB], dy[L][CB], B[L][NR], C[L][NR];
    };
    template <typename IO>
    static constexpr int O_CK = O_RAW + (int)sizeof(Raw<IO>) / 4;              // [KEPT][2][PB][NP]
    template <typename IO>
    static constexpr int O_RED = O_CK<IO> + KEPT * CB * NP;                    // [2][WARPS][K][2 NP]
    template <typename IO>
    static constexpr int LOCAL_BYTES = 4 * O_CK<IO>;
    template <typename IO>
    static constexpr int BYTES = 4 * (O_RED<IO> + 2 * RED);
};

// Two neighbouring values of a row, as they are (`two` false: the second is not there).
template <typename IO>
struct Two;
template <>
struct Two<float> {
    float2 v;
    __device__ __forceinline__ float2 f() const { return v; }
};
template <>
struct Two<__nv_bfloat16> {
    uint32_t v;       // one register, loaded as one word
    __device__ __forceinline__ float2 f() const {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
};
template <typename IO, bool WIDE>
__device__ __forceinline__ Two<IO> load_two(const IO* p, bool two) {
    Two<IO> r;
    if constexpr (WIDE) {
        r.v = *reinterpret_cast<const decltype(r.v)*>(p);
    } else if constexpr (sizeof(IO) == 4) {
        r.v = make_float2(p[0], two ? p[1] : 0.f);
    } else {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
        r.v = q[0] | (two ? (uint32_t)q[1] << 16 : 0u);
    }
    return r;
}

// Asks for the rows of a tile (with wide rows they arrive while other work goes on).
template <typename IO, typename SH, bool WIDE>
__device__ __forceinline__ void bwd_request(const SelArgs& a, const SelPlace& p, int t0, int end, float* sm) {
    using Raw = typename SH::template Raw<IO>;
    Raw& r = *reinterpret_cast<Raw*>(sm + SH::O_RAW);
    constexpr int L = SH::L, CB = SH::CB, TH = SH::THREADS;
    const long long bn = (long long)p.g * a.N;
    stage_rows<IO, WIDE, L, CB, TH>(&r.x[0][0], a.x, p.b, p.c0, t0, end, p.nc);
    stage_rows<IO, WIDE, L, CB, TH>(&r.dt[0][0], a.dt, p.b, p.c0, t0, end, p.nc);
    stage_rows<IO, WIDE, L, CB, TH>(&r.dy[0][0], a.dy, p.b, p.c0, t0, end, p.nc);
    if (a.z.p) stage_rows<IO, WIDE, L, CB, TH>(&r.z[0][0], a.z, p.b, p.c0, t0, end, p.nc);
    if (WIDE && a.wide_bc) {
        stage_rows<IO, true, L, Raw::NR, TH>(&r.B[0][0], a.B, p.b, bn, t0, end, a.N);
        stage_rows<IO, true, L, Raw::NR, TH>(&r.C[0][0], a.C, p.b, bn, t0, end, a.N);
    } else {
        stage_rows<IO, false, L, Raw::NR, TH>(&r.B[0][0], a.B, p.b, bn, t0, end, a.N);
        stage_rows<IO, false, L, Raw::NR, TH>(&r.C[0][0], a.C, p.b, bn, t0, end, a.N);
    }
    cp_async_commit();
}

// delta, delta x and e = dy SiLU(z) of the tile that was asked for (zero past the end), and its B
// and C, from the rows as they came.
template <typename IO, typename SH>
__device__ __forceinline__ void bwd_stage(const SelArgs& a, const SelPlace& p, int t0, int end, float* sm) {
    using Raw = typename SH::template Raw<IO>;
    const Raw& r = *reinterpret_cast<const Raw*>(sm + SH::O_RAW);
    constexpr int PB = SH::PB, STEP = SH::THREADS / PB, NP = SH::NP;
#pragma unroll 4
    for (int i = threadIdx.x; i < SH::L * NP; i += SH::THREADS) {
        const int u = i / NP, n = i % NP;
        const bool on = n < a.N;
        sm[SH::O_BC + u * 2 * NP + n] = on ? to_f(r.B[u][n]) : 0.f;
        sm[SH::O_BC + (u * 2 + 1) * NP + n] = on ? to_f(r.C[u][n]) : 0.f;
    }
    const int k = threadIdx.x % PB;
    float2 bias = make_float2(0.f, 0.f);
    if (a.dt_bias) {
        if (2 * k < p.nc) bias.x = a.dt_bias[p.c0 + 2 * k];
        if (2 * k + 1 < p.nc) bias.y = a.dt_bias[p.c0 + 2 * k + 1];
    }
#pragma unroll 2
    for (int u = threadIdx.x / PB; u < SH::L; u += STEP) {
        float2 delta = make_float2(0.f, 0.f), dx = delta, e = delta;
        if (t0 + u < end) {
            const float2 x = pair_of(&r.x[u][2 * k]), dt = pair_of(&r.dt[u][2 * k]);
            e = pair_of(&r.dy[u][2 * k]);
            if (a.z.p) {
                const float2 z = pair_of(&r.z[u][2 * k]);
                e.x *= z.x * sigmoid_f<IO>(z.x);
                e.y *= z.y * sigmoid_f<IO>(z.y);
            }
            delta.x = sel_delta(dt.x, bias.x, a.softplus);
            delta.y = sel_delta(dt.y, bias.y, a.softplus);
            dx.x = delta.x * x.x;
            dx.y = delta.y * x.y;
        }
        reinterpret_cast<float4*>(sm + SH::O_DD)[u * PB + k] = make_float4(delta.x, delta.y, dx.x, dx.y);
        reinterpret_cast<float2*>(sm + SH::O_E)[u * PB + k] = e;
    }
}

// A lane's NT states (as pairs) of a [..][N] row; zero where there are none.
template <int NT>
__device__ __forceinline__ void row_pairs(f2 (&v)[NT / 2], const float* p, bool live, int n0, int N,
                                          float scale) {
#pragma unroll
    for (int i = 0; i < NT / 2; i++) {
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; j++)
            f[j] = live && n0 + 2 * i + j < N ? p[n0 + 2 * i + j] * scale : 0.f;
        v[i] = pack2(f[0], f[1]);
    }
}
template <int NT>
__device__ __forceinline__ void store_pairs(const f2 (&v)[NT / 2], float* p, bool live, int n0, int N) {
#pragma unroll
    for (int i = 0; i < NT / 2; i++) {
        float f[2];
        unpack2(v[i], f[0], f[1]);
#pragma unroll
        for (int j = 0; j < 2; j++)
            if (live && n0 + 2 * i + j < N) p[n0 + 2 * i + j] = f[j];
    }
}
__device__ __forceinline__ float sum2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return lo + hi;
}

template <typename IO, typename SH, bool WIDE>
__global__ void __launch_bounds__(SH::THREADS, SH::LOCAL_BLOCKS) sel_bwd_local_kernel(const SelArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int NT = SH::NT, CW = SH::CW, PB = SH::PB, NP = SH::NP, L = SH::L;
    const SelPlace p = sel_place(a, SH::CB);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int pl = wid * CW + lane % CW, s = lane / CW, c = p.c0 + 2 * pl;
    const int end = min(p.t1, p.len), tiles = a.seg / L;
    f2 h[2][NT / 2], g[2][NT / 2], P[2][NT / 2], A2[2][NT / 2];
#pragma unroll
    for (int q = 0; q < 2; q++) {
        row_pairs<NT>(A2[q], a.A + (long long)(c + q) * a.N, 2 * pl + q < p.nc, s * NT, a.N, kLog2e);
#pragma unroll
        for (int i = 0; i < NT / 2; i++) {
            h[q][i] = g[q][i] = 0;
            P[q][i] = pack2(1.f, 1.f);
        }
    }
    float total[2] = {0.f, 0.f};
    if (p.t0 < end) bwd_request<IO, SH, WIDE>(a, p, p.t0, end, sm);
    for (int j = 0; j < tiles; j++) {
        const int t0 = p.t0 + j * L;
        const int count = min(L, end - t0);
        if (count > 0) {
            cp_async_wait<0>();
            __syncthreads();      // the rows are here; the tile before is done with
            bwd_stage<IO, SH>(a, p, t0, end, sm);
            __syncthreads();
            if (t0 + L < end && j + 1 < tiles) bwd_request<IO, SH, WIDE>(a, p, t0 + L, end, sm);
        }
#pragma unroll 2
        for (int u = 0; u < count; u++) {
            const float4 d = reinterpret_cast<const float4*>(sm + SH::O_DD)[u * PB + pl];
            const float2 e = reinterpret_cast<const float2*>(sm + SH::O_E)[u * PB + pl];
            const float dv[2] = {d.x, d.y}, xv[2] = {d.z, d.w}, ev[2] = {e.x, e.y};
            f2 B[NT / 2], C[NT / 2];
            load_pairs(B, sm + SH::O_BC + u * 2 * NP + s * NT);
            load_pairs(C, sm + SH::O_BC + (u * 2 + 1) * NP + s * NT);
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const f2 delta = pack2(dv[q], dv[q]), dx = pack2(xv[q], xv[q]), eq = pack2(ev[q], ev[q]);
                total[q] += dv[q];
#pragma unroll
                for (int i = 0; i < NT / 2; i++) {
                    const f2 dec = ex2_2(mul2(delta, A2[q][i]));
                    h[q][i] = fma2(dec, h[q][i], mul2(dx, B[i]));
                    P[q][i] = mul2(P[q][i], dec);      // decay from the entry through this token
                    g[q][i] = fma2(P[q][i], mul2(C[i], eq), g[q][i]);
                }
            }
        }
        // at the end of each of the backward walk's tiles (the last segment may have fewer)
        const int ends = (j + 1) * L;
        if (ends % a.tile == 0 && p.t0 + ends - a.tile < p.t1) {
            const long long k = (long long)p.b * a.ntile + p.seg * (a.seg / a.tile) + ends / a.tile - 1;
#pragma unroll
            for (int q = 0; q < 2; q++) {
                store_pairs<NT>(h[q], a.hloc + (k * a.D + c + q) * a.N, 2 * pl + q < p.nc, s * NT, a.N);
                if (s == 0 && 2 * pl + q < p.nc) a.dsum[k * a.D + c + q] = total[q];
            }
        }
    }
    const long long k = (long long)p.b * a.nseg + p.seg;
#pragma unroll
    for (int q = 0; q < 2; q++)
        store_pairs<NT>(g[q], a.gseg + (k * a.D + c + q) * a.N, 2 * pl + q < p.nc, s * NT, a.N);
}

// Entry states over the segments in order (the grid's first half), leaving adjoints over them in
// reverse (its second half); dh is what leaves before the first.
__global__ void __launch_bounds__(128) sel_bwd_chain_kernel(const SelArgs a, int blocks) {
    const long long per = (long long)a.D * a.N;
    const bool back = blockIdx.x >= blocks;
    const long long i = (back ? blockIdx.x - blocks : blockIdx.x) * 128ll + threadIdx.x;
    if (i >= per * a.batch) return;
    const int b = (int)(i / per);
    const long long dn = i - b * per;
    const int d = (int)(dn / a.N);
    const float A2 = a.A[dn] * kLog2e;
    const int tiles = a.seg / a.tile;
    // the last tile of segment k
    auto tile_of = [&](int k) { return (long long)b * a.ntile + min((k + 1) * tiles, a.ntile) - 1; };
    const float* ds = a.dsum + d;
    float* out = (back ? a.gseg : a.hseg) + (long long)b * a.nseg * per + dn;
    constexpr int U = 8;          // segments requested together
    float v = back ? (a.dhT ? a.dhT[i] : 0.f) : a.h[i];
    for (int k0 = 0; k0 < a.nseg; k0 += U) {
        float own[U], dec[U];
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 + u < a.nseg) {
                const int k = back ? a.nseg - 1 - (k0 + u) : k0 + u;
                own[u] = back ? out[k * per] : a.hloc[tile_of(k) * per + dn];
                dec[u] = ds[tile_of(k) * a.D];
            }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 + u < a.nseg) {
                const int k = back ? a.nseg - 1 - (k0 + u) : k0 + u;
                out[k * per] = v;
                v = fmaf(ex2(A2 * dec[u]), v, own[u]);
            }
    }
    if (back && a.dh) a.dh[i] = v;
}

template <typename IO, typename SH, bool WIDE>
__global__ void __launch_bounds__(SH::THREADS, SH::MIN_BLOCKS) sel_bwd_kernel(const SelArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int NT = SH::NT, S = SH::S, CW = SH::CW, PB = SH::PB, CB = SH::CB, NP = SH::NP;
    constexpr int K = SH::K, L = SH::L, WARPS = SH::WARPS;
    const SelPlace p = sel_place(a, CB);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int pl = wid * CW + lane % CW, s = lane / CW, c = p.c0 + 2 * pl;
    const int mine = min(max(p.nc - 2 * pl, 0), 2);      // channels of the pair that exist
    const int end = min(p.t1, p.len);
    const int blk = blockIdx.x % sel_tiles(a.D, a.G, CB), blks = sel_tiles(a.D, a.G, CB);

    const Rows<const IO> X{static_cast<const IO*>(a.x.p), a.x.bs, a.x.ts};
    const Rows<const IO> DT{static_cast<const IO*>(a.dt.p), a.dt.bs, a.dt.ts};
    const Rows<const IO> Z{static_cast<const IO*>(a.z.p), a.z.bs, a.z.ts};
    const Rows<const IO> DY{static_cast<const IO*>(a.dy.p), a.dy.bs, a.dy.ts};
    const Rows<IO> DX{static_cast<IO*>(a.dx.p), a.dx.bs, a.dx.ts};
    const Rows<IO> DDT{static_cast<IO*>(a.ddt.p), a.ddt.bs, a.ddt.ts};
    const Rows<IO> DZ{static_cast<IO*>(a.dz.p), a.dz.bs, a.dz.ts};

    f2 lam[2][NT / 2], A2[2][NT / 2], dA[2][NT / 2];
    float skip[2] = {0.f, 0.f}, bias[2] = {0.f, 0.f}, dD[2] = {0.f, 0.f}, dbias[2] = {0.f, 0.f};
    const long long row = (((long long)p.b * a.nseg + p.seg) * a.D + c) * a.N;
    // a sequence of one tile is not chained: it starts from h0 and dhT (row is theirs then)
    const bool single = a.ntile == 1;
    const float* entry = single ? a.h : a.hseg;
    const float* leaving = single ? a.dhT : a.gseg;
#pragma unroll
    for (int q = 0; q < 2; q++) {
        row_pairs<NT>(A2[q], a.A + (long long)(c + q) * a.N, q < mine, s * NT, a.N, kLog2e);
        row_pairs<NT>(lam[q], leaving + row + q * a.N, q < mine && leaving, s * NT, a.N, 1.f);
#pragma unroll
        for (int i = 0; i < NT / 2; i++) dA[q][i] = 0;
        if (q < mine && a.Dskip) skip[q] = a.Dskip[c + q];
        if (q < mine && a.dt_bias) bias[q] = a.dt_bias[c + q];
    }

    const int tiles = a.seg / L;
    const int last = end > p.t0 ? (end - p.t0 - 1) / L : -1;      // the last tile that holds tokens
    if (last >= 0) bwd_request<IO, SH, WIDE>(a, p, p.t0 + last * L, end, sm);
    for (int jt = last; jt >= 0; jt--) {
        const int t0 = p.t0 + jt * L;
        const int count = min(L, end - t0);
        f2 h[2][NT / 2], h0[2][NT / 2];      // h0: the tile's entry state
#pragma unroll
        for (int q = 0; q < 2; q++) {
            row_pairs<NT>(h[q], entry + row + q * a.N, q < mine, s * NT, a.N, 1.f);
            if (jt > 0) {
                // decayed from the segment's entry, plus the segment's own
                const long long k = (long long)p.b * a.ntile + p.seg * tiles + jt - 1;
                const float sum = q < mine ? a.dsum[k * a.D + c + q] : 0.f;
                f2 own[NT / 2];
                row_pairs<NT>(own, a.hloc + (k * a.D + c + q) * a.N, q < mine, s * NT, a.N, 1.f);
#pragma unroll
                for (int i = 0; i < NT / 2; i++)
                    h[q][i] = fma2(ex2_2(mul2(pack2(sum, sum), A2[q][i])), h[q][i], own[i]);
            }
#pragma unroll
            for (int i = 0; i < NT / 2; i++) h0[q][i] = h[q][i];
        }
        cp_async_wait<0>();
        __syncthreads();      // the rows are here; the tile before is done with
        bwd_stage<IO, SH>(a, p, t0, end, sm);
        __syncthreads();
        if (jt > 0) bwd_request<IO, SH, WIDE>(a, p, t0 - L, end, sm);

        const float4* dd = reinterpret_cast<const float4*>(sm + SH::O_DD) + pl;
        const float2* ee = reinterpret_cast<const float2*>(sm + SH::O_E) + pl;
        const int pieces = (count + K - 1) / K;
        // the state before each piece but the first and the last (a thread reads back its own
        // values only)
        auto kept = [&](int j, int q) {
            return sm + SH::template O_CK<IO> + (((j - 1) * 2 + q) * PB + pl) * NP + s * NT;
        };
        for (int j = 0; j < pieces; j++) {
            if (j > 0 && j + 1 < pieces)
#pragma unroll
                for (int q = 0; q < 2; q++)
#pragma unroll
                    for (int i = 0; i < NT / 2; i++) reinterpret_cast<f2*>(kept(j, q))[i] = h[q][i];
            if (j + 1 < pieces) {
#pragma unroll
                for (int k = 0; k < K; k++) {
                    const int u = j * K + k;
                    const float4 d = dd[u * PB];
                    const float dv[2] = {d.x, d.y}, xv[2] = {d.z, d.w};
                    f2 B[NT / 2];
                    load_pairs(B, sm + SH::O_BC + u * 2 * NP + s * NT);
#pragma unroll
                    for (int q = 0; q < 2; q++)
#pragma unroll
                        for (int i = 0; i < NT / 2; i++)
                            h[q][i] = fma2(ex2_2(mul2(pack2(dv[q], dv[q]), A2[q][i])), h[q][i],
                                           mul2(pack2(xv[q], xv[q]), B[i]));
                }
            }
        }
        for (int j = pieces - 1; j >= 0; j--) {
            // the tokens whose sums this lane ends with, and their values, on their way early
            constexpr int TOKENS = K > S ? K / S : 1, SAME = S > K ? S / K : 1;
            const int own = s / SAME * TOKENS;
            Two<IO> rx[TOKENS], rt[TOKENS], rz[TOKENS], ry[TOKENS];
#pragma unroll
            for (int i = 0; i < TOKENS; i++) {
                const int t = t0 + j * K + own + i;
                if (mine && t < end) {
                    rx[i] = load_two<IO, WIDE>(X.at(p.b, t) + c, mine == 2);
                    if (a.softplus) rt[i] = load_two<IO, WIDE>(DT.at(p.b, t) + c, mine == 2);
                    if (a.z.p) {
                        rz[i] = load_two<IO, WIDE>(Z.at(p.b, t) + c, mine == 2);
                        ry[i] = load_two<IO, WIDE>(DY.at(p.b, t) + c, mine == 2);
                    }
                }
            }
            f2 hp[K][2][NT / 2], dec[K][2][NT / 2];     // state before token k, decay of token k
            if (j + 1 < pieces) {
                if (j == 0) {
#pragma unroll
                    for (int q = 0; q < 2; q++)
#pragma unroll
                        for (int i = 0; i < NT / 2; i++) h[q][i] = h0[q][i];
                } else {
#pragma unroll
                    for (int q = 0; q < 2; q++) load_pairs(h[q], kept(j, q));
                }
            }
#pragma unroll
            for (int k = 0; k < K; k++) {
                const int u = j * K + k;     // zero past the end: the state stays
                const float4 d = dd[u * PB];
                const float dv[2] = {d.x, d.y}, xv[2] = {d.z, d.w};
                f2 B[NT / 2];
                load_pairs(B, sm + SH::O_BC + u * 2 * NP + s * NT);
#pragma unroll
                for (int q = 0; q < 2; q++)
#pragma unroll
                    for (int i = 0; i < NT / 2; i++) {
                        hp[k][q][i] = h[q][i];
                        dec[k][q][i] = ex2_2(mul2(pack2(dv[q], dv[q]), A2[q][i]));
                        h[q][i] = fma2(dec[k][q][i], h[q][i], mul2(pack2(xv[q], xv[q]), B[i]));
                    }
            }
            // sums over the states of both channels: C h, lam B, A2 lam a h_before
            float yv[2][K], lb[2][K], la[2][K];
#pragma unroll
            for (int k = K - 1; k >= 0; k--) {
                const int u = j * K + k;
                const float4 d = dd[u * PB];
                const float2 e2 = ee[u * PB];
                const float dv[2] = {d.x, d.y}, xv[2] = {d.z, d.w}, ev[2] = {e2.x, e2.y};
                f2 B[NT / 2], C[NT / 2], ob[NT / 2], oc[NT / 2];
                load_pairs(B, sm + SH::O_BC + u * 2 * NP + s * NT);
                load_pairs(C, sm + SH::O_BC + (u * 2 + 1) * NP + s * NT);
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    const f2 delta = pack2(dv[q], dv[q]), dx = pack2(xv[q], xv[q]), e = pack2(ev[q], ev[q]);
                    f2 y = 0, b = 0, l = 0;
#pragma unroll
                    for (int i = 0; i < NT / 2; i++) {
                        const f2 now = k == K - 1 ? h[q][i] : hp[k == K - 1 ? k : k + 1][q][i];
                        lam[q][i] = fma2(C[i], e, lam[q][i]);
                        ob[i] = q == 0 ? mul2(lam[q][i], dx) : fma2(lam[q][i], dx, ob[i]);
                        oc[i] = q == 0 ? mul2(now, e) : fma2(now, e, oc[i]);
                        y = i == 0 ? mul2(C[i], now) : fma2(C[i], now, y);
                        b = i == 0 ? mul2(lam[q][i], B[i]) : fma2(lam[q][i], B[i], b);
                        lam[q][i] = mul2(lam[q][i], dec[k][q][i]);
                        const f2 lh = mul2(lam[q][i], hp[k][q][i]);
                        l = i == 0 ? mul2(lh, A2[q][i]) : fma2(lh, A2[q][i], l);
                        dA[q][i] = fma2(lh, delta, dA[q][i]);
                    }
                    yv[q][k] = sum2(y);
                    lb[q][k] = sum2(b);
                    la[q][k] = sum2(l);
                }
                // over the warp's channels
                float over[2 * NT];
#pragma unroll
                for (int i = 0; i < NT / 2; i++) {
                    unpack2(ob[i], over[2 * i], over[2 * i + 1]);
                    unpack2(oc[i], over[NT + 2 * i], over[NT + 2 * i + 1]);
                }
                const int off = lane_sum<2 * NT, CW, 1>(over, lane);
                constexpr int HOLD = 2 * NT > CW ? 2 * NT / CW : 1, SPARE = CW > 2 * NT ? CW / (2 * NT) : 1;
                if (lane % SPARE == 0) {
                    float* red = sm + SH::template O_RED<IO> + (j & 1) * SH::RED + (wid * K + k) * 2 * NP;
#pragma unroll
                    for (int i = 0; i < HOLD; i++) {
                        const int v = off + i;
                        red[(v / NT) * NP + s * NT + v % NT] = over[i];
                    }
                }
            }
            // over the pair's lanes: each ends with the sums of K / S tokens, or S / K lanes with
            // those of the same one
#pragma unroll
            for (int q = 0; q < 2; q++) {
                lane_sum<K, S, CW>(yv[q], lane);
                lane_sum<K, S, CW>(lb[q], lane);
                lane_sum<K, S, CW>(la[q], lane);
            }
            if (mine && s % SAME == 0) {
#pragma unroll
                for (int i = 0; i < TOKENS; i++) {
                    const int u = j * K + own + i, t = t0 + u;
                    if (t >= end) continue;
                    const float4 d = dd[u * PB];
                    const float2 e = ee[u * PB];
                    const float2 x = rx[i].f();
                    float o[2];
                    if (a.z.p) {
                        const float2 z = rz[i].f(), dy = ry[i].f();
                        const float s0 = sigmoid_f<IO>(z.x), s1 = sigmoid_f<IO>(z.y);
                        float y0 = yv[0][i], y1 = yv[1][i];
                        if (a.Dskip) {      // no 0 * inf without D
                            y0 = fmaf(skip[0], x.x, y0);
                            y1 = fmaf(skip[1], x.y, y1);
                        }
                        o[0] = dy.x * y0 * fmaf(z.x * s0, 1.f - s0, s0);
                        o[1] = dy.y * y1 * fmaf(z.y * s1, 1.f - s1, s1);
                        Vec<IO, 2>::template store<WIDE>(o, DZ.at(p.b, t) + c, mine);
                    }
                    o[0] = d.x * lb[0][i];
                    o[1] = d.y * lb[1][i];
                    if (a.Dskip) {
                        o[0] = fmaf(skip[0], e.x, o[0]);
                        o[1] = fmaf(skip[1], e.y, o[1]);
                    }
                    Vec<IO, 2>::template store<WIDE>(o, DX.at(p.b, t) + c, mine);
                    o[0] = fmaf(x.x, lb[0][i], la[0][i] * kLn2);
                    o[1] = fmaf(x.y, lb[1][i], la[1][i] * kLn2);
                    if (a.softplus) {
                        const float2 dt = rt[i].f();
                        o[0] *= sigmoid_f<IO>(dt.x + bias[0]);
                        o[1] *= sigmoid_f<IO>(dt.y + bias[1]);
                    }
                    Vec<IO, 2>::template store<WIDE>(o, DDT.at(p.b, t) + c, mine);
                    dD[0] = fmaf(e.x, x.x, dD[0]);
                    dD[1] = fmaf(e.y, x.y, dD[1]);
                    dbias[0] += o[0];
                    dbias[1] += o[1];
                }
            }
            // over the block's warps, to the workspace
            __syncthreads();
            for (int i = threadIdx.x; i < K * 2 * NP; i += SH::THREADS) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; w++) v += sm[SH::template O_RED<IO> + (j & 1) * SH::RED + w * K * 2 * NP + i];
                const int t = t0 + j * K + i / (2 * NP);
                if (t < end)
                    a.pBC[(((long long)p.b * a.T + t) * blks + blk) * 2 * NP + i % (2 * NP)] = v;
            }
        }
    }
    // rows past the sequence's length
    for (int t = max(p.t0, p.len); t < p.t1; t++)
        for (int k = threadIdx.x; k < p.nc; k += SH::THREADS) {
            DX.at(p.b, t)[p.c0 + k] = from_f<IO>(0.f);
            DDT.at(p.b, t)[p.c0 + k] = from_f<IO>(0.f);
            if (a.z.p) DZ.at(p.b, t)[p.c0 + k] = from_f<IO>(0.f);
        }
#pragma unroll
    for (int q = 0; q < 2; q++) {
#pragma unroll
        for (int o = CW; o < 32; o *= 2) {
            dD[q] += __shfl_xor_sync(0xffffffffu, dD[q], o);
            dbias[q] += __shfl_xor_sync(0xffffffffu, dbias[q], o);
        }
        store_pairs<NT>(dA[q], a.pA + row + q * a.N, q < mine, s * NT, a.N);
        if (single && a.dh) store_pairs<NT>(lam[q], a.dh + row + q * a.N, q < mine, s * NT, a.N);
        if (q < mine && s == 0) {
            float* o = a.pD + ((long long)p.b * a.nseg + p.seg) * 2 * a.D + c + q;
            o[0] = dD[q];
            o[a.D] = dbias[q];
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

// Sums of the segments' shares: dA ([runs][D N]), then dD and ddt_bias ([runs][2][D]).
__global__ void __launch_bounds__(1024) sel_bwd_sum_kernel(const SelArgs a) {
    const long long states = (long long)a.D * a.N, c = blockIdx.x * 32ll + (threadIdx.x & 31);
    const bool in_A = c < states, on = c < states + 2 * a.D;
    const float v = column_sum(in_A ? a.pA + c : a.pD + (c - states), a.batch * a.nseg,
                               in_A ? states : 2ll * a.D, on);
    if (threadIdx.x < 32 && on) {
        if (in_A)
            a.dA[c] = v;
        else if (c < states + a.D) {
            if (a.dD) a.dD[c - states] = v;
        } else if (a.ddt_bias)
            a.ddt_bias[c - states - a.D] = v;
    }
}

template <typename IO, typename SH, bool WIDE>
cudaError_t bwd_w(const SelArgs& a, cudaStream_t s) {
    static_assert(SH::template BYTES<IO> <= 227 * 1024, "");
    const int tiles = sel_tiles(a.D, a.G, SH::CB);
    const unsigned grid = (unsigned)((long long)tiles * a.nseg * a.batch);
    // the first step walks shorter tiles, so that more blocks fit an SM
    using LSH = BwdShape<SH::NT, SH::S, SH::WARPS, 16, SH::K>;
    static_assert(SH::L % LSH::L == 0, "");
    cudaError_t e = allow_smem(sel_bwd_local_kernel<IO, LSH, WIDE>, LSH::template LOCAL_BYTES<IO>);
    if (e == cudaSuccess) e = allow_smem(sel_bwd_kernel<IO, SH, WIDE>, SH::template BYTES<IO>);
    if (e != cudaSuccess) return e;
    const long long states = (long long)a.D * a.N;
    if (a.ntile > 1) {
        sel_bwd_local_kernel<IO, LSH, WIDE><<<grid, LSH::THREADS, LSH::template LOCAL_BYTES<IO>, s>>>(a);
        const int blocks = (int)((states * a.batch + 127) / 128);
        sel_bwd_chain_kernel<<<2 * blocks, 128, 0, s>>>(a, blocks);
    }
    sel_bwd_kernel<IO, SH, WIDE><<<grid, SH::THREADS, SH::template BYTES<IO>, s>>>(a);
    const long long bc = (long long)a.batch * a.T * a.G * 2 * a.N;
    sel_bwd_bc_kernel<IO><<<(unsigned)((bc + 255) / 256), 256, 0, s>>>(a, SH::NP, tiles);
    sel_bwd_sum_kernel<<<(unsigned)((states + 2 * a.D + 31) / 32), column_threads(states + 2 * a.D), 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, typename SH>
cudaError_t bwd_t(const SelArgs& a, cudaStream_t s) {
    return a.wide ? bwd_w<IO, SH, true>(a, s) : bwd_w<IO, SH, false>(a, s);
}

// The lane shape by the number of states.  At 16 states (4 x 2048 tokens of 4096 channels) four a lane
// take 1.19 ms; two a lane, with 16 warps an SM instead of 12, take 1.47 (more lanes to sum over), and
// blocks of two warps 1.29; at 64, eight a lane take half as long again (registers spill).
template <typename F>
cudaError_t by_n(int N, F f) {
    if (N <= 4) return f(BwdShape<2, 2, 2, 32, 4>{});
    if (N <= 8) return f(BwdShape<2, 4, 4, 32, 4>{});
    if (N <= 16) return f(BwdShape<4, 4, 4, 32, 4>{});
    if (N <= 32) return f(BwdShape<4, 8, 4, 32, 4>{});
    if (N <= 64) return f(BwdShape<4, 16, 4, 32, 4>{});
    if (N <= 128) return f(BwdShape<8, 16, 4, 16, 2>{});
    return f(BwdShape<8, 32, 4, 16, 2>{});
}

}  // namespace

// Blocks of channels, and how many blocks the segments must make before they get more tiles.
static long long sel_bwd_blocks(const SelArgs& a) {
    int CB = 0;
    by_n(a.N, [&](auto sh) {
        CB = decltype(sh)::CB;
        return cudaSuccess;
    });
    return sel_tiles(a.D, a.G, CB);
}
constexpr long long kBwdBlocks = 148 * 12;

size_t sel_bwd_plan(SelArgs* a, char* ws) {
    int NP = 0;
    by_n(a->N, [&](auto sh) {
        a->tile = decltype(sh)::L;
        NP = decltype(sh)::NP;
        return cudaSuccess;
    });
    const size_t blks = sel_bwd_blocks(*a);
    a->ntile = (a->T + a->tile - 1) / a->tile;
    // Tiles of a segment: four where the segments still give every SM its blocks several times
    // over (fewer segments are chained, and fewer shares of dA summed), else fewer.
    int m = 4;
    while (m > 1 && (long long)blks * a->batch * ((a->ntile + m - 1) / m) < kBwdBlocks) m /= 2;
    a->seg = m * a->tile;
    a->nseg = (a->ntile + m - 1) / m;
    const size_t runs = (size_t)a->batch * a->nseg, states = (size_t)a->D * a->N;
    const size_t all = (size_t)a->batch * a->ntile;
    size_t at = 0;
    auto take = [&](size_t floats) {
        float* p = reinterpret_cast<float*>(ws + at);
        at += (floats * sizeof(float) + 255) / 256 * 256;
        return p;
    };
    a->hloc = take(all * states);
    a->dsum = take(all * a->D);
    a->hseg = take(runs * states);
    a->gseg = take(runs * states);
    a->pA = take(runs * states);
    a->pD = take(runs * 2 * a->D);
    a->pBC = take((size_t)a->batch * a->T * blks * 2 * NP);
    return at;
}

// The size grows with T but where a segment gets more tiles: the longest length with each number
// of tiles a segment is looked at.
size_t sel_bwd_most(SelArgs a) {
    size_t most = sel_bwd_plan(&a, nullptr);
    const int tile = a.tile, ntile = a.ntile;
    const long long columns = (long long)a.batch * sel_bwd_blocks(a), segments = (kBwdBlocks - 1) / columns;
    for (int m = 1; m < 4; m *= 2) {
        const long long tiles = 2 * m * segments;      // the most that 2 m a segment are too few for
        if (tiles < 1 || tiles >= ntile) continue;
        a.T = (int)tiles * tile;
        const size_t n = sel_bwd_plan(&a, nullptr);
        if (n > most) most = n;
    }
    return most;
}

cudaError_t launch_sel_bwd(const SelArgs& a, int io_dtype, cudaStream_t s) {
    if (io_dtype == M3_BF16)
        return by_n(a.N, [&](auto sh) { return bwd_t<__nv_bfloat16, decltype(sh)>(a, s); });
    return by_n(a.N, [&](auto sh) { return bwd_t<float, decltype(sh)>(a, s); });
}

}  // namespace m3
