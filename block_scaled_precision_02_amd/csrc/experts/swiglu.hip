// swiglu.hip -- silu(gate) * up between the experts' two products (or a dense
// layer's), written as the A operand and scales of the second.
//
//   y = g / (1 + exp(-g)) * u       binary32, not rounded before the encoder
//   code = enc(y / s)               s by the GEMM's scale rule
//
// Bound by memory, 4 bytes read and 1 written an output, and close behind it by
// the vector units (one MI355X: 30001 x 2112 to MXFP8 53 us, 6.0 TB/s; 30001 x 2048 to
// blockscale 57, to e4m3 with row scales 60; 512 x 2048 with row scales 4).  Quotients by
// a scale are the divided ones, as after the norms: 4 us of the 60.  The block forms
// (scales per 32 or 128 elements) need nothing of the rest of the row: a wave
// takes any 64 consecutive pieces of 8 outputs.  The row forms keep a row in
// the registers of a workgroup of 256 threads, however short it is.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../layer/norm_dev.hpp"
#include "experts.hpp"

namespace qgemm {

namespace {

// silu(g) u within a few units in the last place for every g: with a =
// exp(-|g|) <= 1, silu is g / (1 + a) or g a / (1 + a), so that nothing
// overflows and a small silu keeps a's relative error.  a = 2^n 2^z, n + z =
// -|g| log2(e): g has 8 bits and HI, the logarithm's first part, 16, so that
// their product is exact, n is what is whole in it and z, within a half, takes
// the rest with the second part.  Past 400 a is 0 in any case.  1 + a lies in
// [1, 2]; its reciprocal takes one Newton step on the hardware's.  (By one exp2
// of the rounded exponent and the reciprocal as it comes, 11 instructions less an
// element, the error is |g| + 4 units; 30001 x 2048 to e4m3 with row scales 50 us, by
// this 56, to MXFP8 51 by either.)
__device__ __forceinline__ float swiglu(float g, float u)
{
    constexpr float HI = 1.44268798828125f, LO = 7.052607543e-6f;   // log2(e)
    const float m = __builtin_amdgcn_fmed3f(fabsf(g), 0.0f, 400.0f);   // (NaN: any; g brings it back)
    const float t = m * -HI, n = __builtin_rintf(t);
    const float a = __builtin_ldexpf(__builtin_amdgcn_exp2f(fmaf(m, -LO, t - n)), (int)n);
    const float d = 1.0f + a, r0 = __builtin_amdgcn_rcpf(d);
    const float r = fmaf(fmaf(-d, r0, 1.0f), r0, r0);
    return g * (g < 0.0f ? a : 1.0f) * r * u;
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
    // (a launch has at most 2^31 pieces)
    const unsigned np = a.I / 8, total = (unsigned)rows * np, g0 = blockIdx.x * (256u * PER);
    if (g0 >= total)
        return;
    u32x4 gate[PER], up[PER];
    int64_t row[PER];
    int p[PER];
    bool live[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const unsigned g = g0 + 256 * i + threadIdx.x;
        live[i] = g < total;
        const unsigned h = live[i] ? g : threadIdx.x & 3, r = __umulhi(h, a.row_mul) >> a.row_shift;   // (any piece that is there)
        row[i] = r;
        p[i] = (int)(h - r * np);
        const u32x4 *x = (const u32x4 *)(a.X + row[i] * a.ldx) + p[i];
        gate[i] = __builtin_nontemporal_load(x);
        up[i] = __builtin_nontemporal_load(x + np);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        emit<OUT, true>(product(gate[i], up[i]), 1.0f, 0.0f, p[i], live[i], a.Q + row[i] * a.ldq,
                  (uint8_t *)a.S + row[i] * a.lds * (OUT == NORM_F8_BLOCK ? 4 : 1));
}

// Row forms.
constexpr int THREADS = 256, WAVES = THREADS / 64;

template <int OUT, int KEEP>
__global__ void __launch_bounds__(THREADS) swiglu_row_kernel(SwigluArgs a)
{
    const int64_t rows = a.count ? min<int64_t>(max(*a.count - a.row0, (int64_t)0), a.M) : a.M;
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x;
    if (row >= rows)
        return;
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
    __shared__ float wtop[WAVES];
    if ((t & 63) == 0)
        wtop[t >> 6] = top;
    __syncthreads();
    top = wtop[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
        top = max_nan(top, wtop[w]);
    const float s = top / (OUT == NORM_I8_ROW ? 127.0f : 448.0f);
    if (t == 0)
        ((float *)a.S)[row] = s;
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int p = t + THREADS * c;
        if (p < np)                                     // (the row forms exchange nothing between lanes)
            emit<OUT, true>(keep[c], 1.0f, s, p, true, q, nullptr);
    }
    for (int p = t + THREADS * KEEP; p < np; p += THREADS)
        emit<OUT, true>(load_y(g, u, p), 1.0f, s, p, true, q, nullptr);
}

template <int OUT>
hipError_t launch_rows(const SwigluArgs &a, hipStream_t s)
{
    const int np = a.I / 8;
    const dim3 grid((unsigned)a.M), block(THREADS);
    if (np <= 256)
        hipLaunchKernelGGL((swiglu_row_kernel<OUT, 1>), grid, block, 0, s, a);
    else if (np <= 512)
        hipLaunchKernelGGL((swiglu_row_kernel<OUT, 2>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((swiglu_row_kernel<OUT, 4>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int OUT>
hipError_t launch_block(SwigluArgs a, hipStream_t s)
{
    // n / d for n < 2^31, 2^(b-1) < d <= 2^b: m = ceil(2^(31+b) / d) has 32 bits, and
    // n m / 2^(31+b) is above n / d by less than n / 2^31 of 1 / d
    const unsigned np = a.I / 8, b = 32 - __builtin_clz(np - 1);   // (np >= 4)
    a.row_mul = (unsigned)((((uint64_t)1 << (31 + b)) + np - 1) / np);
    a.row_shift = b - 1;
    const uint64_t pieces = (uint64_t)a.M * np;
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
