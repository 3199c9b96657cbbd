// swiglu.hip -- silu(gate) * up between the experts' two products (or a dense
// layer's), written as the A operand and scales of the second.
//
//   y = g / (1 + exp(-g)) * u       binary32, not rounded before the encoder
//   code = enc(y / s)               s by the GEMM's scale rule
//
// Bound by memory: 4 bytes read and 1 written an output (one MI355X: 30001 x
// 2112 to MXFP8 53 us, 6.0 TB/s; 512 x 2048 with row scales 3.3 us).  The block forms
// (scales per 32 or 128 elements) need nothing of the rest of the row: a wave
// takes any 64 consecutive pieces of 8 outputs.  The row forms keep a row in
// the registers of a workgroup or, where there are many short rows, of a wave.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../layer/norm_dev.hpp"
#include "experts.hpp"

namespace qgemm {

namespace {

// silu(g) u by the hardware's exp2 and reciprocal, each good to a unit in the
// last place.  The exponent -g log2(e) is rounded once, an error of up to |g|
// half units in exp(-g): far below what the encoder resolves wherever silu(g)
// is not itself negligible.  (A correctly rounded exponential and division are 30
// instructions an element more: the kernel waited for the vector units, 67 us
// for 30001 rows of 2112 to MXFP8.)  exp(-g) = inf gives g * 0 = -0, as the
// formula does.
__device__ __forceinline__ float swiglu(float g, float u)
{
    const float e = __builtin_amdgcn_exp2f(-1.44269504088896340736f * g);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

__device__ __forceinline__ Piece product(u32x4 a, u32x4 b)
{
    Piece y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y.v[2 * i] = swiglu(lo_bf16(a[i]), lo_bf16(b[i]));
        y.v[2 * i + 1] = swiglu(hi_bf16(a[i]), hi_bf16(b[i]));
    }
    return y;
}

__device__ __forceinline__ Piece load_y(const u32x4 *g, const u32x4 *u, int p)
{
    return product(__builtin_nontemporal_load(&g[p]), __builtin_nontemporal_load(&u[p]));
}

// Block forms: piece g of the launch is piece g % np of row g / np; np is a
// multiple of a block's pieces, so that a block lies on adjacent lanes.  A thread
// takes PER pieces, 256 apart, all loaded first.
constexpr int PER = 2;

template <int OUT>
__global__ void __launch_bounds__(256) swiglu_block_kernel(SwigluArgs a)
{
    const int64_t rows = a.count ? min<int64_t>(max(*a.count - a.row0, (int64_t)0), a.M) : a.M;
    const unsigned np = a.I / 8;
    const uint64_t total = (uint64_t)rows * np, g0 = (uint64_t)blockIdx.x * (256 * PER);
    if (g0 >= total)
        return;
    u32x4 gate[PER], up[PER];
    int64_t row[PER];
    int p[PER];
    bool live[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint64_t g = g0 + 256 * i + threadIdx.x;
        live[i] = g < total;
        row[i] = live[i] ? (int64_t)(g / np) : 0;
        p[i] = live[i] ? (int)(g - row[i] * np) : (int)(threadIdx.x & 15);
        const u32x4 *x = (const u32x4 *)(a.X + row[i] * a.ldx) + p[i];
        gate[i] = up[i] = u32x4{};
        if (live[i]) {
            gate[i] = __builtin_nontemporal_load(x);
            up[i] = __builtin_nontemporal_load(x + np);
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        emit<OUT>(product(gate[i], up[i]), 1.0f, 0.0f, p[i], live[i], a.Q + row[i] * a.ldq,
                  (uint8_t *)a.S + row[i] * a.lds * (OUT == NORM_F8_BLOCK ? 4 : 1));
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
    hipLaunchKernelGGL((swiglu_block_kernel<OUT>), dim3((unsigned)((pieces + 256 * PER - 1) / (256 * PER))),
                       dim3(256), 0, s, a);
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
