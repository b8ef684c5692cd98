// norm.cu -- RMS norm with the residual's addition, outputs in the io type or in e4m3 with one
// scale for each 128 values, and its backward (m3_norm_*).
//
// Memory alone bounds it: a row is read once, stays in registers between the two passes over
// its values, and is written once.  A row is spread over TPR threads (a warp to a block of 1024);
// thread k of a row holds the vectors k, k + TPR, .. of 8 neighbouring values, so the 128 values
// of an e4m3 group lie in 16 neighbouring lanes.
//
// 32768 rows of 2048, bf16 in, fp32 residual, e4m3 out: 120 us, one call after another (6.2 TB/s; the
// bytes take 113 at the copy rate).  Backward of 16384 rows: 96 us (5.6 TB/s; 82): the next row's
// vectors on their way while a row is summed took 30 % off.
#include <cuda_fp8.h>

#include "block_internal.h"
#include "block_common.cuh"

namespace m3 {

namespace {

constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100
constexpr float kE4m3Max = 448.f;

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sum over the TPR threads of a row of M values each; every thread gets the sums.  `sm` holds
// M floats for each warp of the block.
template <int TPR, int M>
__device__ __forceinline__ void row_sum(float (&v)[M], float* sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int m = 0; m < M; m++) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int wid = threadIdx.x >> 5, first = wid / W * W;
        __syncthreads();            // the sums of the row before have been read
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int m = 0; m < M; m++) sm[wid * M + m] = v[m];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < M; m++) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; w++) s += sm[(first + w) * M + m];
            v[m] = s;
        }
    }
}

__device__ __forceinline__ uint2 to_e4m3(const float (&q)[8]) {
    union { __nv_fp8x2_storage_t h[4]; uint2 v; } out;
#pragma unroll
    for (int j = 0; j < 4; j++)
        out.h[j] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * j], q[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    return out.v;
}

// Eight values of a row in e4m3, with the scale of their group of 128 (16 neighbouring lanes): every
// value the nearest step, ties to even.
//
// A value next to the middle of two steps lands on the other step for an error of one ulp (y / scale
// from rounded y and scale: 40 of 67 million).  The reciprocal root is a factor of y and of max |y|
// alike, so the quotient is 448 r w / max |r w|; with the products, the reciprocal of their largest
// and the quotient each rounded once, t is within 2^-23 of it.  Where t (1 - 2^-22) and t (1 + 2^-22)
// go to the same step, so does the quotient.
// Else the value is open, and the warp (one in six hundred) comes again with EXACT: it is compared
// with g, the nearest value of five significant bits (every step and every middle of two is one).
// The sign of 448 r w - g max |r w|, formed by FMA with the products' low parts (to 2^-44, exactly
// where there are none), says on which side of g the quotient is rounded.
// few_bits: r of 8 significant bits (bf16) and weights of 4 at most (none, or ones) give products
// that lie in the middle itself in most warps, else 2^-17 from it (7 a and g b are integers below
// 2^17 for 12-bit a and b): one remainder step makes t the quotient where that is representable,
// and the conversion does the rest (32768 rows of 2048 without a residual: 72 us; 115 by the
// comparison).
template <bool EXACT, bool WIDE>
__device__ __forceinline__ bool store_e4m3(const float (&r)[8], const float (&w)[8], bool few_bits, float mean,
                                           float rstd, uint8_t* o, int n, float* scale_out) {
    // rstd = ratio 2^e: the power of two keeps the products in range and rounds nothing
    const uint32_t bits = __float_as_uint(rstd);
    const float pow2 = __uint_as_float(bits & 0x7f800000u);
    const float ratio = __uint_as_float((bits & 0x007fffffu) | 0x3f800000u);
    float hi[8], top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        hi[j] = __fmul_rn(r[j] * pow2, w[j]);
        top = max_nan(top, fabsf(hi[j]));        // padding is 0
    }
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, s));
    // what the reciprocal root lacks (one Newton step on mean rstd^2 = 1, by FMA), for the scale
    const float p = mean * rstd, e = fmaf(mean, rstd, -p);
    float low = 0.5f * ratio * (fmaf(-p, rstd, 1.f) - e * rstd);
    if (!(fabsf(low) < ratio)) low = 0.f;      // a mean of 0, infinity or NaN has no remainder
    const float product = top * ratio;
    float amax = product + fmaf(top, low, fmaf(top, ratio, -product));
    const bool tiny = amax < kAmaxFloor, finite = amax < __int_as_float(0x7f800000);
    float inv = tiny ? ratio * (kE4m3Max / kAmaxFloor) : kE4m3Max / top;
    if (!finite) amax = inv = __int_as_float(0x7fffffff);
    union { uint8_t b[8]; uint2 v; } out;
    bool open = false;
    float q[8];
    if constexpr (EXACT) {
        float top_lo = -3.4e38f;      // the low part of the largest product
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (fabsf(hi[j]) == top) top_lo = fmaxf(top_lo, fmaf(fabsf(r[j] * pow2), fabsf(w[j]), -top));
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) top_lo = fmaxf(top_lo, __shfl_xor_sync(0xffffffffu, top_lo, s));
        if (tiny) {
            top = kAmaxFloor / ratio;
            top_lo = 0.f;
        }
        if (!finite) return false;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            // 2^-9 on both sides keeps the products in range
            const float h = fabsf(hi[j]);
            const uint32_t g = (__float_as_uint(h * inv) + 0x40000u) & ~0x7ffffu;
            const float step = __uint_as_float(g) * 0.001953125f, x = __fmul_rn(step, top);
            const float gap = fmaf(0.875f, h, -x) - fmaf(step, top, -x) +
                              fmaf(0.875f, fmaf(fabsf(r[j] * pow2), fabsf(w[j]), -h), -(step * top_lo));
            q[j] = copysignf(__uint_as_float(gap > 0.f ? g + 1u : gap < 0.f ? g - 1u : g), hi[j]);
        }
        out.v = to_e4m3(q);
    } else {
        if (scale_out) *scale_out = max_nan(amax, kAmaxFloor) / kE4m3Max;
        if (few_bits && top < 1e35f) {      // 448 hi stays finite
            const float back = tiny ? 0.f : inv * (1.f / kE4m3Max);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float t = __fmul_rn(hi[j], inv);
                q[j] = fmaf(fmaf(-t, top, kE4m3Max * hi[j]), back, t);
            }
            out.v = to_e4m3(q);
        } else {
            constexpr float kSpread = 2.384185791015625e-07f;      // 2^-22
            float above[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float t = __fmul_rn(hi[j], inv);
                q[j] = t * (1.f - kSpread);
                above[j] = t * (1.f + kSpread);
            }
            out.v = to_e4m3(q);
            const uint2 other = to_e4m3(above);
            open = out.v.x != other.x || out.v.y != other.y;
        }
    }
    if constexpr (WIDE) {
        if (n > 0) *reinterpret_cast<uint2*>(o) = out.v;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) o[j] = out.b[j];
    }
    return open;
}

// Rows of up to 16384 values in e4m3: 1152 threads an SM, 56 registers (32768 rows of 2048, bf16 without
// a residual: 73 us; 77 with the 64 that it takes by itself, and at 48 they spill).
template <int OUT, int NV, int THREADS>
constexpr int fwd_blocks = OUT == M3_OUT_E4M3 && NV == 2 ? 1152 / THREADS : 1;

template <typename IO, typename RES, int OUT, int TPR, int NV, bool WIDE>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, fwd_blocks<OUT, NV, TPR < 128 ? 128 : TPR>)
norm_fwd_kernel(const NormArgs a) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    __shared__ float sm[32];
    const int k = threadIdx.x % TPR;
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    const bool live = row < a.rows;
    if (!live) row = a.rows - 1;       // a spare row group joins the barriers and writes nothing
    const IO* x = static_cast<const IO*>(a.x) + row * a.xs;
    const RES* res = static_cast<const RES*>(a.res) + row * a.rs;
    float r[NV][8];
    float ss[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; v++) {
        const int i = (k + v * TPR) * 8, n = min(max(a.d - i, 0), 8);
        Vec<IO, 8>::template load<WIDE>(r[v], x + i, n);
        if (a.res) {
            float q[8];
            Vec<RES, 8>::template load<WIDE>(q, res + i, n);
#pragma unroll
            for (int j = 0; j < 8; j++) r[v][j] = to_f(from_f<RES>(r[v][j] + q[j]));
        }
#pragma unroll
        for (int j = 0; j < 8; j++) ss[0] = fmaf(r[v][j], r[v][j], ss[0]);
    }
    row_sum<TPR>(ss, sm);
    const float mean = ss[0] / (float)a.d + a.eps, rstd = 1.f / sqrtf(mean);
    bool open = false;
    auto values = [&](auto exact, int v) {
        const int i = (k + v * TPR) * 8, n = live ? min(max(a.d - i, 0), 8) : 0;
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] = 1.f;
        bool few_bits = sizeof(RES) == 2;
        if (a.weight) {
            Vec<float, 8>::load<WIDE>(w, a.weight + i, min(max(a.d - i, 0), 8));
            if constexpr (sizeof(RES) == 2) {
                uint32_t tail = 0;
#pragma unroll
                for (int j = 0; j < 8; j++) tail |= __float_as_uint(w[j]);
                few_bits = !__any_sync(0xffffffffu, tail & 0xfffffu);
            }
        }
        uint8_t* o = static_cast<uint8_t*>(a.y) + row * a.ys + i;
        float* scale = n > 0 && i % 128 == 0 ? a.scales + row * ((a.d + 127) / 128) + i / 128 : nullptr;
        open |= store_e4m3<decltype(exact)::value, WIDE>(r[v], w, few_bits, mean, rstd, o, n, scale);
    };
#pragma unroll
    for (int v = 0; v < NV; v++) {
        const int i = (k + v * TPR) * 8, n = live ? min(max(a.d - i, 0), 8) : 0;
        if (a.res_out)
            Vec<RES, 8>::template store<WIDE>(r[v], static_cast<RES*>(a.res_out) + row * a.ros + i, n);
        if constexpr (OUT == M3_OUT_IO) {
            float y[8], w[8];
            if (a.weight) Vec<float, 8>::load<WIDE>(w, a.weight + i, min(max(a.d - i, 0), 8));
#pragma unroll
            for (int j = 0; j < 8; j++) {
                y[j] = r[v][j] * rstd;
                if (a.weight) y[j] *= w[j];
            }
            Vec<IO, 8>::template store<WIDE>(y, static_cast<IO*>(a.y) + row * a.ys + i, n);
        } else {
            values(std::false_type{}, v);
        }
    }
    if constexpr (OUT == M3_OUT_E4M3) {
        if (__any_sync(0xffffffffu, open))
#pragma unroll
            for (int v = 0; v < NV; v++) values(std::true_type{}, v);
    }
}

// Backward: a block walks rows (row group `blockIdx.x`, then every gridDim.x-th) and keeps its
// columns' share of dweight in registers.  With one vector a thread (rows of up to 8192 values)
// the next row's r, dy and dres are on their way while a row is summed and written; longer rows
// are read again for the second pass (from L2), as registers hold dweight alone.
template <typename IO, typename RES>
struct BwdVec {
    typename Vec<RES, 8>::Raw r, q;
    typename Vec<IO, 8>::Raw g;
};

template <typename T, bool WIDE>
__device__ __forceinline__ void load_raw(typename Vec<T, 8>::Raw& v, const T* p, int n) {
    if constexpr (WIDE) {
        if (n > 0) v = *reinterpret_cast<const typename Vec<T, 8>::Raw*>(p);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) v.v[j] = p[j];
    }
}

template <typename IO, typename RES, int TPR, int NV, bool WIDE>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_bwd_kernel(const NormArgs a) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    constexpr bool AHEAD = NV == 1;
    __shared__ float sm[64];
    const int k = threadIdx.x % TPR;
    float dw[NV][8];
#pragma unroll
    for (int v = 0; v < NV; v++)
#pragma unroll
        for (int j = 0; j < 8; j++) dw[v][j] = 0.f;
    const float inv_d = 1.f / (float)a.d;
    const long long step = (long long)gridDim.x * RPB;
    auto request = [&](long long row, int v, BwdVec<IO, RES>& to, bool second) {
        const int i = (k + v * TPR) * 8, n = row < a.rows ? min(max(a.d - i, 0), 8) : 0;
        load_raw<RES, WIDE>(to.r, static_cast<const RES*>(a.x) + row * a.xs + i, n);
        load_raw<IO, WIDE>(to.g, static_cast<const IO*>(a.dy) + row * a.dys + i, n);
        if (second && a.dres)
            load_raw<RES, WIDE>(to.q, static_cast<const RES*>(a.dres) + row * a.drs + i, n);
    };
    auto weights = [&](int v, float (&w)[8]) {
        const int i = (k + v * TPR) * 8;
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] = 1.f;
        if (a.weight) Vec<float, 8>::load<WIDE>(w, a.weight + i, min(max(a.d - i, 0), 8));
    };
    const BwdVec<IO, RES> none = {};
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    BwdVec<IO, RES> next = none;
    float w0[8];
    weights(0, w0);
    if (AHEAD) request(row, 0, next, true);
    // every thread of a block makes the same number of turns: the barriers are the block's
    for (long long row0 = (long long)blockIdx.x * RPB; row0 < a.rows; row0 += step, row += step) {
        const bool live = row < a.rows;
        const BwdVec<IO, RES> cur = next;
        if (AHEAD) {
            next = none;
            request(row + step, 0, next, true);
        }
        float s[2] = {0.f, 0.f};      // sum r^2, sum dy w r
#pragma unroll
        for (int v = 0; v < NV; v++) {
            BwdVec<IO, RES> c = AHEAD ? cur : none;
            float w[8];
            if (!AHEAD) {
                request(row, v, c, false);
                weights(v, w);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float r = to_f(c.r.v[j]);
                s[0] = fmaf(r, r, s[0]);
                s[1] = fmaf(to_f(c.g.v[j]) * (AHEAD ? w0[j] : w[j]), r, s[1]);
            }
        }
        row_sum<TPR>(s, sm);
        const float rstd = 1.f / sqrtf(s[0] * inv_d + a.eps);
        const float back = s[1] * inv_d * rstd * rstd;      // mean(dy w u) rstd
        if (!live) continue;
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int i = (k + v * TPR) * 8, n = min(max(a.d - i, 0), 8);
            BwdVec<IO, RES> c = AHEAD ? cur : none;
            float w[8], o[8];
            if (!AHEAD) {
                request(row, v, c, true);
                weights(v, w);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float r = to_f(c.r.v[j]), g = to_f(c.g.v[j]);
                o[j] = rstd * (g * (AHEAD ? w0[j] : w[j]) - r * back);
                if (a.dres) o[j] += to_f(c.q.v[j]);
                dw[v][j] = fmaf(g, r * rstd, dw[v][j]);
            }
            Vec<IO, 8>::template store<WIDE>(o, static_cast<IO*>(a.dx) + row * a.dxs + i, n);
            if (a.dresidual)
                Vec<RES, 8>::template store<WIDE>(o, static_cast<RES*>(a.dresidual) + row * a.dros + i, n);
        }
    }
    if (a.part) {
        float* o = a.part + (long long)blockIdx.x * a.d;
        if constexpr (RPB > 1) {
            // the row groups of a block add up, in order
            __shared__ float sums[RPB][TPR][9];
#pragma unroll
            for (int j = 0; j < 8; j++) sums[threadIdx.x / TPR][k][j] = dw[0][j];
            __syncthreads();
            if (threadIdx.x >= TPR) return;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                dw[0][j] = 0.f;
#pragma unroll
                for (int g = 0; g < RPB; g++) dw[0][j] += sums[g][k][j];
            }
        }
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int i = (k + v * TPR) * 8;
            Vec<float, 8>::store<WIDE>(dw[v], o + i, min(max(a.d - i, 0), 8));
        }
    }
}

__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float* part, int shares, int d,
                                                            float* dweight) {
    const int c = blockIdx.x * 32 + (threadIdx.x & 31);
    const float v = column_sum(part + c, shares, d, c < d);
    if (threadIdx.x < 32 && c < d) dweight[c] = v;
}

// Threads of a row: the fewest that hold it with two vectors each (1024 hold four).
int row_threads(int d) {
    int t = 32;
    while (t < 1024 && t * 8 * 2 < d) t *= 2;
    return t;
}

template <typename IO, typename RES, int OUT, bool WIDE>
cudaError_t fwd_t(const NormArgs& a, cudaStream_t s) {
    auto go = [&](auto kernel, int tpr) {
        const int rpb = tpr < 128 ? 128 / tpr : 1;
        kernel<<<(unsigned)(((long long)a.rows + rpb - 1) / rpb), tpr < 128 ? 128 : tpr, 0, s>>>(a);
        return cudaGetLastError();
    };
    switch (row_threads(a.d)) {
        case 32: return go(norm_fwd_kernel<IO, RES, OUT, 32, 2, WIDE>, 32);
        case 64: return go(norm_fwd_kernel<IO, RES, OUT, 64, 2, WIDE>, 64);
        case 128: return go(norm_fwd_kernel<IO, RES, OUT, 128, 2, WIDE>, 128);
        case 256: return go(norm_fwd_kernel<IO, RES, OUT, 256, 2, WIDE>, 256);
        case 512: return go(norm_fwd_kernel<IO, RES, OUT, 512, 2, WIDE>, 512);
    }
    if (a.d <= 1024 * 16) return go(norm_fwd_kernel<IO, RES, OUT, 1024, 2, WIDE>, 1024);
    return go(norm_fwd_kernel<IO, RES, OUT, 1024, 4, WIDE>, 1024);
}

// The backward holds four times as much of a row: one vector a thread up to 8192 values.
int bwd_threads(int d) {
    int t = 32;
    while (t < 1024 && t * 8 < d) t *= 2;
    return t;
}

template <typename IO, typename RES, bool WIDE>
cudaError_t bwd_t(const NormArgs& a, cudaStream_t s) {
    auto go = [&](auto kernel, int tpr) {
        kernel<<<a.blocks, tpr < 128 ? 128 : tpr, 0, s>>>(a);
        if (a.part) {
            norm_bwd_sum_kernel<<<(a.d + 31) / 32, column_threads(a.d), 0, s>>>(a.part, a.blocks, a.d, a.dweight);
        }
        return cudaGetLastError();
    };
    switch (bwd_threads(a.d)) {
        case 32: return go(norm_bwd_kernel<IO, RES, 32, 1, WIDE>, 32);
        case 64: return go(norm_bwd_kernel<IO, RES, 64, 1, WIDE>, 64);
        case 128: return go(norm_bwd_kernel<IO, RES, 128, 1, WIDE>, 128);
        case 256: return go(norm_bwd_kernel<IO, RES, 256, 1, WIDE>, 256);
        case 512: return go(norm_bwd_kernel<IO, RES, 512, 1, WIDE>, 512);
    }
    if (a.d <= 1024 * 8) return go(norm_bwd_kernel<IO, RES, 1024, 1, WIDE>, 1024);
    if (a.d <= 1024 * 16) return go(norm_bwd_kernel<IO, RES, 1024, 2, WIDE>, 1024);
    return go(norm_bwd_kernel<IO, RES, 1024, 4, WIDE>, 1024);
}

template <typename F>
cudaError_t by_type(int io, int res, bool wide, F f) {
    using bf = __nv_bfloat16;
    auto w = [&](auto i, auto r) {
        return wide ? f(i, r, std::true_type{}) : f(i, r, std::false_type{});
    };
    if (io == M3_BF16) return res == M3_BF16 ? w(bf{}, bf{}) : w(bf{}, float{});
    return res == M3_BF16 ? w(float{}, bf{}) : w(float{}, float{});
}

}  // namespace

int norm_bwd_blocks(int rows, int d) {
    const int tpr = bwd_threads(d), rpb = tpr < 128 ? 128 / tpr : 1, threads = tpr < 128 ? 128 : tpr;
    const long long groups = ((long long)rows + rpb - 1) / rpb;
    const int most = 148 * (1024 / threads);
    return (int)(groups < most ? (groups < 1 ? 1 : groups) : most);
}

cudaError_t launch_norm_fwd(const NormArgs& a, int io, int res, int out, cudaStream_t s) {
    return by_type(io, res, a.wide, [&](auto i, auto r, auto w) {
        using I = decltype(i);
        using R = decltype(r);
        constexpr bool W = decltype(w)::value;
        return out == M3_OUT_E4M3 ? fwd_t<I, R, M3_OUT_E4M3, W>(a, s) : fwd_t<I, R, M3_OUT_IO, W>(a, s);
    });
}

cudaError_t launch_norm_bwd(const NormArgs& a, int io, int res, cudaStream_t s) {
    return by_type(io, res, a.wide, [&](auto i, auto r, auto w) {
        return bwd_t<decltype(i), decltype(r), decltype(w)::value>(a, s);
    });
}

}  // namespace m3
