// block_internal.h -- launchers between the block operators' entry points (block_api.cu) and
// their kernels.  Everything is validated before it comes here.
#pragma once

#include <cuda_runtime.h>

#include "m3_common.cuh"

namespace m3 {

struct View {          // m3_rows, device side
    const void* p;
    long long bs, ts;
};

// ------------------------------------------------------------------ convolution
struct ConvArgs {
    View x, dy;            // inputs [b][T][C] io
    struct { void* p; long long bs, ts; } y, dx;
    const float* weight;   // [C][W]
    const float* bias;     // [C] or null
    const int32_t* seqlens;
    void* state;           // [b][W-1][C] io (backward: read only)
    float* dweight;
    float* dbias;
    float* dstate;
    float* part;           // workspace: [b * nseg][W + 1][C]
    int batch, T, C, W;
    int seg, nseg;         // tokens per run, runs per sequence
    bool silu, wide;
};
enum class ConvCall { fwd, step, bwd };
cudaError_t launch_conv(const ConvArgs& a, ConvCall call, int io_dtype, cudaStream_t s);

// ------------------------------------------------------------------ selective scan
struct SelArgs {
    View x, dt, B, C, z;   // z.p null: no gate
    View dy;
    struct { void* p; long long bs, ts; } y, dx, ddt, dB, dC, dz;
    const float* A;        // [D][N]
    const float* Dskip;    // [D] or null
    const float* dt_bias;  // [D] or null
    const int32_t* seqlens;
    float* h;              // [b][D][N] in / out (backward: h0, read only)
    const float* dhT;
    float *dA, *dD, *ddt_bias, *dh;
    // workspace
    float* hseg;           // [b][nseg][D][N]: forward: each segment's own end state, then its entry
                           // state; backward: its entry state
    float* dsum;           // forward [b][nseg][D]: sum of delta over the segment; backward
                           // [b][ntile][D]: from the segment's start through the tile
    float* hloc;           // [b][ntile][D][N]: backward: the segment's own state after the tile
    float* gseg;           // [b][nseg][D][N]: own entry adjoint, then the leaving adjoint
    float* pBC;            // [b][T][channel blocks][2][states padded]: shares of dB and dC
    float* pA;             // [b * nseg][D][N]
    float* pD;             // [b * nseg][2][D]: dD, ddt_bias
    int batch, T, D, G, N;
    int seg, nseg;         // tokens per segment (a multiple of the tile), segments
    int tile, ntile;       // backward: tokens per tile, tiles
    bool softplus;
    bool wide;             // rows of channels: 16-byte copies, pairs of channels in one access
    bool wide_bc;          // the same of B and C
    bool step_rows;
};
// Tokens of one staged tile: segments are multiples of it.
constexpr int kSelTile = 32;
int sel_fwd_segments(int batch, int T, int D, int G, int N, int* seg);
size_t sel_fwd_workspace(int batch, int T, int D, int G, int N);
size_t sel_fwd_most(int batch, int T, int D, int G, int N);      // of any length up to T
cudaError_t launch_sel_fwd(const SelArgs& a, int io_dtype, cudaStream_t s);
cudaError_t launch_sel_step(const SelArgs& a, int io_dtype, cudaStream_t s);
// Fills in seg, nseg and the workspace pointers (relative to a null workspace: sizes alone).
size_t sel_bwd_plan(SelArgs* a, char* ws);
size_t sel_bwd_most(SelArgs a);      // the largest size of any length up to a.T
cudaError_t launch_sel_bwd(const SelArgs& a, int io_dtype, cudaStream_t s);

// ------------------------------------------------------------------ norm
struct NormArgs {
    const void *x, *res, *dy, *dres;
    void *y, *res_out, *dx, *dresidual;
    long long xs, rs, ys, ros, dys, drs, dxs, dros;   // row strides in elements
    const float* weight;
    float* scales;
    float* dweight;
    float* part;           // workspace: [blocks][d]
    int rows, d, blocks;
    float eps;
    bool wide;
};
int norm_bwd_blocks(int rows, int d);
cudaError_t launch_norm_fwd(const NormArgs& a, int io_dtype, int res_dtype, int out, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, int io_dtype, int res_dtype, cudaStream_t s);

}  // namespace m3
