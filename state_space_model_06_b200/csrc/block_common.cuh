// block_common.cuh -- shared pieces of the block operators (conv.cu, sel_*.cu, norm.cu): strided
// row views, vectors of io values, the activations and the lane reductions.
#pragma once

#include "m3_internal.h"

namespace m3 {

// Device-side form of m3_rows: element (b, t, i) at p[b * bs + t * ts + i].
template <typename T>
struct Rows {
    T* p;
    long long bs, ts;
    __device__ __forceinline__ T* at(long long b, long long t) const { return p + b * bs + t * ts; }
};

// Tokens of sequence b: its entry of seqlens clamped to [0, T], or T.
__device__ __forceinline__ int tokens_of(const int32_t* seqlens, int b, int T) {
    return seqlens ? min(max(seqlens[b], 0), T) : T;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Logistic function.  bf16 results round at 2^-8 (relative), so they take the hardware exp2
// and reciprocal (a few 2^-22); fp32 results take expf and a rounded division.
template <typename IO>
__device__ __forceinline__ float sigmoid_f(float v) {
    if constexpr (sizeof(IO) == 2) return rcp(1.f + ex2(-kLog2e * v));
    return 1.f / (1.f + expf(-v));
}

// Softplus: max(v, 0) + log(1 + u), u = e^-|v| in (0, 1], in fp32 for every io type.  With
// s = u / (2 + u) in (0, 1/3], log(1 + u) = 2 atanh(s) = 2 s (1 + s^2/3 + s^4/5 + ..): the four
// coefficients are a minimax fit of the series over s^2 in [0, 1/9] (relative error 5e-9), good for
// small u, where log(1 + u) from a rounded 1 + u is not.  The rounding of |v| log2(e) becomes a
// relative error of u, so the step is good to (1.33 |v| + 12) 2^-24: some 20 2^-24 where it is 0.001.
// The remainder of that product is not carried: it would take four instructions more, where step
// and gate take 49.
__device__ __forceinline__ float softplus_f(float v) {
    const float u = ex2(-fabsf(v) * kLog2e);
    const float s = u * rcp(2.f + u), q = s * s;
    float r = 0.1400599330663681f;
    r = fmaf(r, q, 0.1400090307f);
    r = fmaf(r, q, 0.2001076341f);
    r = fmaf(r, q, 0.3333320916f);
    const float t = s + s;
    return fmaxf(v, 0.f) + fmaf(r * q, t, t);
}

// A kernel may use `bytes` of dynamic shared memory (above the 48 KiB that every kernel may).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// ------------------------------------------------------------------ packed pairs
// Two fp32 values in a 64-bit register pair: one FFMA2 does the work of two FFMAs in one issue
// slot, and these kernels are short of issue slots.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// ------------------------------------------------------------------ asynchronous copies
// Global to shared memory, without a register in between.  16 bytes (`on` false: zeros).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int bytes = on ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes)
                 : "memory");
}
// The same of 4 bytes.
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool on) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int bytes = on ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(bytes)
                 : "memory");
}
// N = 8 or 16 bytes.
template <int N>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// V consecutive io values as floats.  WIDE: one aligned vector access of V * sizeof(IO) bytes
// (8 or 16, or 32 as two); otherwise element by element, the first n of them (the rest read 0
// and are not written).
template <typename IO, int V>
struct Vec {
    static constexpr int BYTES = V * (int)sizeof(IO);
    struct alignas(BYTES < 16 ? BYTES : 16) Raw {
        IO v[V];
    };
    template <bool WIDE>
    static __device__ __forceinline__ void load(float (&f)[V], const IO* p, int n) {
        if constexpr (WIDE) {
            if (n > 0) {
                const Raw r = *reinterpret_cast<const Raw*>(p);
#pragma unroll
                for (int i = 0; i < V; i++) f[i] = to_f(r.v[i]);
                return;
            }
#pragma unroll
            for (int i = 0; i < V; i++) f[i] = 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) f[i] = i < n ? to_f(p[i]) : 0.f;
        }
    }
    template <bool WIDE>
    static __device__ __forceinline__ void store(const float (&f)[V], IO* p, int n) {
        if constexpr (WIDE) {
            if (n > 0) {
                Raw r;
#pragma unroll
                for (int i = 0; i < V; i++) r.v[i] = from_f<IO>(f[i]);
                *reinterpret_cast<Raw*>(p) = r;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (i < n) p[i] = from_f<IO>(f[i]);
        }
    }
};

// Sums v[0..M) over the L lanes that differ in the bits LO, 2 LO, .. L LO / 2 of the lane
// number.  Each halving step keeps half of the values and sends the other half, so the lanes
// end with max(M / L, 1) sums each: M (1 - 1/L) shuffles instead of M log2 L.  With L >= M the
// last steps add whole values.  Returns in v[0..max(M/L,1)) the sums of the values whose number
// starts at the returned offset; lanes that differ only in the adding steps hold the same ones.
template <int M, int L, int LO, int K>
__device__ __forceinline__ int lane_sum(float (&v)[K], int lane) {
    if constexpr (L == 1) {
        return 0;
    } else if constexpr (M > 1) {
        constexpr int H = M / 2, BIT = LO * L / 2;
        const bool up = lane & BIT;
#pragma unroll
        for (int i = 0; i < H; i++) {
            const float send = up ? v[i] : v[i + H];
            const float keep = up ? v[i + H] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, BIT);
        }
        return (up ? H : 0) + lane_sum<H, L / 2, LO>(v, lane);
    } else {
#pragma unroll
        for (int o = LO * L / 2; o >= LO; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        return 0;
    }
}

// Sum of a column of shares, p[r * stride] for r < rows, by a block of which lane l of every warp
// passes the same column: each warp takes every so many rows, then the warps' sums add up in
// order.  The result is valid in the first warp.
__device__ __forceinline__ float column_sum(const float* p, int rows, long long stride, bool on) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float s = 0.f;
    if (on)
#pragma unroll 8
        for (int r = wid; r < rows; r += warps) s += p[r * stride];
    sm[wid][lane] = s;
    __syncthreads();
    float v = 0.f;
    if (wid == 0)
        for (int i = 0; i < warps; i++) v += sm[i][lane];
    return v;
}
// Threads of such a block: eight warps where the columns alone fill the GPU, else 32.
inline int column_threads(long long columns) { return columns >= 32 * 148 * 4 ? 256 : 1024; }

}  // namespace m3
