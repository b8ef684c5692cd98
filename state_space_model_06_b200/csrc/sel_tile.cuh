// sel_tile.cuh -- how the selective scan's kernels lay a tile out over lanes and shared memory.
//
// A channel's N states are spread over S lanes (a power of two), NT states each, so a warp
// holds 32 / S channels.  Lane l of a warp owns channel l % CW and states (l / CW) NT ..: lanes
// that differ in the high bits share a channel, neighbouring lanes hold neighbouring channels.
#pragma once

#include "block_common.cuh"

namespace m3 {

template <int NT_, int S_, int WARPS_, int L_ = kSelTile>
struct SelShape {
    static constexpr int NT = NT_, S = S_, WARPS = WARPS_;
    static constexpr int L = L_;                 // tokens staged together (S divides it)
    static constexpr int CW = 32 / S;            // channels of a warp
    static constexpr int CB = CW * WARPS;        // channels of a block
    static constexpr int NP = NT * S;            // states, padded
    static constexpr int THREADS = 32 * WARPS;
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

// B and C of tokens t0 .. t0 + L - 1 as floats in sm[L][2][NP]; tokens at or past `end` and
// states past N read zero.
template <typename IO, int NP, int L, int THREADS>
__device__ __forceinline__ void sel_stage_bc(const SelArgs& a, const SelPlace& p, int t0, int end,
                                             float* sm) {
    const IO* pb = static_cast<const IO*>(a.B.p) + p.b * a.B.bs + (long long)p.g * a.N;
    const IO* pc = static_cast<const IO*>(a.C.p) + p.b * a.C.bs + (long long)p.g * a.N;
#pragma unroll 4
    for (int i = threadIdx.x; i < L * 2 * NP; i += THREADS) {
        const int n = i % NP, which = (i / NP) & 1, t = t0 + i / (2 * NP);
        float v = 0.f;
        if (t < end && n < a.N)
            v = to_f(which ? pc[t * a.C.ts + n] : pb[t * a.B.ts + n]);
        sm[i] = v;
    }
}

}  // namespace m3
