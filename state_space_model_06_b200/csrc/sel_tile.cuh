// sel_tile.cuh -- how the selective scan's kernels lay a tile out over lanes and shared memory.
//
// A channel's N states are spread over S lanes (a power of two), NT states each, and a lane holds
// two neighbouring channels, so a warp holds CW = 32 / S pairs of channels.  Lane l of a warp owns
// pair l % CW and states (l / CW) NT ..: lanes that differ in the high bits share a pair,
// neighbouring lanes hold neighbouring pairs.
#pragma once

#include "block_common.cuh"

namespace m3 {

template <int NT_, int S_, int WARPS_, int L_>
struct SelShape {
    static constexpr int NT = NT_, S = S_, WARPS = WARPS_;
    static constexpr int L = L_;                 // tokens of a tile
    static constexpr int CW = 32 / S;            // pairs of channels of a warp
    static constexpr int PB = CW * WARPS;        // pairs of channels of a block
    static constexpr int CB = 2 * PB;            // channels of a block
    static constexpr int NP = NT * S;            // states, padded
    static constexpr int THREADS = 32 * WARPS;
    static_assert(THREADS % PB == 0, "");
};

// Where a block works: its batch row, segment and channels.  A block's channels all lie in one
// group.
struct SelPlace {
    int b, seg, g, c0, nc, t0, t1, len;
};

__device__ __forceinline__ SelPlace sel_place(const SelArgs& a, int CB) {
    SelPlace p;
    const int per_g = a.D / a.G, tiles_g = (per_g + CB - 1) / CB, tiles = tiles_g * a.G;
    const int tile = blockIdx.x % tiles;
    const int rest = blockIdx.x / tiles;
    p.seg = rest % a.nseg;
    p.b = rest / a.nseg;
    p.g = tile / tiles_g;
    const int k = (tile - p.g * tiles_g) * CB;
    p.c0 = p.g * per_g + k;
    p.nc = min(CB, per_g - k);
    p.t0 = p.seg * a.seg;
    p.len = tokens_of(a.seqlens, p.b, a.T);
    p.t1 = min(p.t0 + a.seg, a.T);
    return p;
}

__host__ __device__ inline int sel_tiles(int D, int G, int CB) { return (D / G + CB - 1) / CB * G; }

__device__ __forceinline__ float sel_delta(float dt, float bias, bool softplus) {
    const float v = dt + bias;
    return softplus ? softplus_f(v) : v;
}

__device__ __forceinline__ f2 ex2_2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(ex2(lo), ex2(hi));
}

// 2 M neighbouring floats of shared memory as pairs, in 16-byte reads where there are four
template <int M>
__device__ __forceinline__ void load_pairs(f2 (&v)[M], const float* p) {
    if constexpr (M == 1) {
        v[0] = *reinterpret_cast<const f2*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < M / 2; i++) {
            const ulonglong2 q = reinterpret_cast<const ulonglong2*>(p)[i];
            v[2 * i] = q.x;
            v[2 * i + 1] = q.y;
        }
    }
}

// ------------------------------------------------------------------ asynchronous tiles
// Rows t0 .. t0 + L - 1 of an activation, `width` values of each from `off` on, into sm[L][W]
// as io values; rows at or past `end` and values past `width` read zero.  WIDE: 16-byte
// asynchronous copies (rows on 16 bytes, width a multiple of 16 bytes); otherwise the values
// are loaded and stored one by one.
template <typename IO, bool WIDE, int L, int W, int THREADS>
__device__ __forceinline__ void stage_rows(IO* sm, const View& v, int b, long long off, int t0,
                                           int end, int width) {
    const IO* p = static_cast<const IO*>(v.p) + b * v.bs + off;
    if constexpr (WIDE) {
        constexpr int V = 16 / sizeof(IO), PER = W / V;
        static_assert(PER > 0 && W % V == 0, "a tile's rows are whole 16-byte pieces");
#pragma unroll
        for (int i = threadIdx.x; i < L * PER; i += THREADS) {
            const int u = i / PER, k = (i % PER) * V;
            const bool on = t0 + u < end && k < width;
            cp_async16(sm + u * W + k, on ? p + (t0 + u) * v.ts + k : p, on);
        }
    } else if constexpr (sizeof(IO) == 4) {
#pragma unroll 4
        for (int i = threadIdx.x; i < L * W; i += THREADS) {
            const int u = i / W, k = i % W;
            const bool on = t0 + u < end && k < width;
            cp_async4(sm + i, on ? p + (t0 + u) * v.ts + k : p, on);
        }
    } else {
#pragma unroll 8
        for (int i = threadIdx.x; i < L * W; i += THREADS) {
            const int u = i / W, k = i % W;
            IO q = from_f<IO>(0.f);
            if (t0 + u < end && k < width) q = p[(t0 + u) * v.ts + k];
            sm[i] = q;
        }
    }
}

// Two neighbouring values as floats.
template <typename IO>
__device__ __forceinline__ float2 pair_of(const IO* p) {
    if constexpr (sizeof(IO) == 2) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
    } else {
        return *reinterpret_cast<const float2*>(p);
    }
}

}  // namespace m3
