// swiglu.hip -- silu(gate) * up between the experts' two products (or a dense
// layer's), written as the A operand and scales of the second.
//
//   y = g / (1 + exp(-g)) * u       binary32, not rounded before the encoder
//   code = enc(y / s)               s by the GEMM's scale rule
//
// Bound by memory: 4 bytes read and 1 written an output.  The block forms
// (scales per 32 or 128 elements) need nothing of the rest of the row: a wave
// takes any 64 consecutive pieces of 8 outputs.  The row forms keep a row in
// the registers of a workgroup or, where there are many short rows, of a wave.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../layer/norm_dev.hpp"
#include "experts.hpp"

namespace qgemm {

namespace {

// silu(g) u.  exp(-g) as a power of two: t = -g log2(e) rounded, and what the
// rounding left out as a factor 1 + r ln 2, which keeps the result within a few
// units in the last place for any g; past 2^126 the power alone (infinity or
// zero: silu is -0 or g).
__device__ __forceinline__ float swiglu(float g, float u)
{
    constexpr float L2E = 1.44269502162933349609375f, L2E_LO = 1.92596299112661746887e-8f, LN2 = 0.693147180559945f;
    const float t = -g * L2E;
    float e = __builtin_amdgcn_exp2f(t);
    if (fabsf(t) < 126.0f) {
        const float r = fmaf(-g, L2E, -t) - g * L2E_LO;
        e = fmaf(e, r * LN2, e);
    }
    return g / (1.0f + e) * u;
}

__device__ __forceinline__ Piece load_y(const u32x4 *g, const u32x4 *u, int p)
{
    const u32x4 a = __builtin_nontemporal_load(&g[p]), b = __builtin_nontemporal_load(&u[p]);
    Piece y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y.v[2 * i] = swiglu(lo_bf16(a[i]), lo_bf16(b[i]));
        y.v[2 * i + 1] = swiglu(hi_bf16(a[i]), hi_bf16(b[i]));
    }
    return y;
}

// Block forms: piece g of the launch is piece g % np of row g / np; np is a
// multiple of a block's pieces, so that a block lies on adjacent lanes.
template <int OUT>
__global__ void __launch_bounds__(256) swiglu_block_kernel(SwigluArgs a)
{
    const int64_t rows = a.count ? min<int64_t>(max(*a.count - a.row0, (int64_t)0), a.M) : a.M;
    const unsigned np = a.I / 8;
    const uint64_t g = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    const uint64_t total = (uint64_t)rows * np;
    if (g - threadIdx.x >= total)
        return;
    const bool live = g < total;
    const uint64_t row = live ? g / np : 0;
    const int p = live ? (int)(g - row * np) : (int)(threadIdx.x & 15);
    const u32x4 *x = (const u32x4 *)(a.X + row * a.ldx);
    Piece y{};
    if (live)
        y = load_y(x, x + np, p);
    emit<OUT>(y, 1.0f, 0.0f, p, live, a.Q + row * a.ldq, (uint8_t *)a.S + row * a.lds * (OUT == NORM_F8_BLOCK ? 4 : 1));
}

// Row forms.
template <int OUT, int THREADS, int KEEP>
__global__ void __launch_bounds__(256) swiglu_row_kernel(SwigluArgs a)
{
    constexpr int ROWS = 256 / THREADS;                 // rows a workgroup
    constexpr int WAVES = THREADS / 64;
    const int64_t rows = a.count ? min<int64_t>(max(*a.count - a.row0, (int64_t)0), a.M) : a.M;
    const int t = threadIdx.x % THREADS;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS;
    if (row >= rows)
        return;                                         // (a workgroup of several rows has no barrier)
    const int np = a.I / 8;
    const u32x4 *g = (const u32x4 *)(a.X + row * a.ldx), *u = g + np;
    uint8_t *q = a.Q + row * a.ldq;

    Piece keep[KEEP];
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int p = t + THREADS * c;
        keep[c] = Piece{};
        if (p < np)
            keep[c] = load_y(g, u, p);
        top = max_nan(top, max_abs(keep[c]));
    }
    for (int p = t + THREADS * KEEP; p < np; p += THREADS)
        top = max_nan(top, max_abs(load_y(g, u, p)));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        top = max_nan(top, __shfl_xor(top, off));
    if constexpr (WAVES > 1) {
        __shared__ float wtop[WAVES];
        if ((t & 63) == 0)
            wtop[t >> 6] = top;
        __syncthreads();
        top = wtop[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            top = max_nan(top, wtop[w]);
    }
    const float s = top / (OUT == NORM_I8_ROW ? 127.0f : 448.0f);
    if (t == 0)
        ((float *)a.S)[row] = s;
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int p = t + THREADS * c;
        emit<OUT>(keep[c], 1.0f, s, p, p < np, q, nullptr);
    }
    for (int p = t + THREADS * KEEP; p < np; p += THREADS)
        emit<OUT>(load_y(g, u, p), 1.0f, s, p, true, q, nullptr);
}

template <int OUT, int THREADS, int KEEP>
hipError_t launch_row(const SwigluArgs &a, hipStream_t s)
{
    constexpr int ROWS = 256 / THREADS;
    hipLaunchKernelGGL((swiglu_row_kernel<OUT, THREADS, KEEP>), dim3((unsigned)((a.M + ROWS - 1) / ROWS)), dim3(256), 0,
                       s, a);
    return hipGetLastError();
}

template <int OUT>
hipError_t launch_rows(const SwigluArgs &a, hipStream_t s)
{
    const int np = a.I / 8;
    if (np <= 256)
        return launch_row<OUT, 256, 1>(a, s);
    if (np <= 512)
        return launch_row<OUT, 256, 2>(a, s);
    return launch_row<OUT, 256, 4>(a, s);
}

template <int OUT>
hipError_t launch_block(const SwigluArgs &a, hipStream_t s)
{
    const uint64_t pieces = (uint64_t)a.M * (a.I / 8);
    hipLaunchKernelGGL((swiglu_block_kernel<OUT>), dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu_quant(int out, const SwigluArgs &all, hipStream_t s)
{
    // a launch holds fewer than 2^32 threads: more rows than that go in several
    const int64_t per = std::max<int64_t>(1, std::min<int64_t>(1 << 23, ((int64_t)1 << 31) / (all.I / 8)));
    hipError_t e = hipSuccess;
    for (int64_t row = 0; row < all.M && e == hipSuccess; row += per) {
        SwigluArgs a = all;
        a.row0 = row;
        a.M = (int)std::min<int64_t>(per, all.M - row);
        a.X += row * a.ldx;
        a.Q += row * a.ldq;
        const int64_t scale = out <= NORM_F8_ROW ? 4 : a.lds * (out == NORM_F8_BLOCK ? 4 : 1);   // bytes a row
        a.S = (uint8_t *)a.S + row * scale;
        switch (out) {
        case NORM_I8_ROW: e = launch_rows<NORM_I8_ROW>(a, s); break;
        case NORM_F8_ROW: e = launch_rows<NORM_F8_ROW>(a, s); break;
        case NORM_F8_BLOCK: e = launch_block<NORM_F8_BLOCK>(a, s); break;
        case NORM_MX_E4M3: e = launch_block<NORM_MX_E4M3>(a, s); break;
        default: e = launch_block<NORM_MX_E2M1>(a, s); break;
        }
    }
    return e;
}

}  // namespace qgemm
