// norm.hip -- root-mean-square norm of x + residual, written as the A operand
// and scales of the GEMM that follows.
//
//   h = x + r                       binary32 (exact sum rounded once)
//   r' = bf16(h)                    the residual stream, handed on
//   y = (h * g) * rsqrt(mean(h^2) + eps)
//   code = enc(y / s)               s by the GEMM's scale rule
//
// h goes into the norm unrounded and y into the encoder unrounded: the only
// roundings to fewer bits are the outputs themselves.  Multiplying by g
// before the row's factor makes the row's max |y| the factor times max |h g|
// (rounding is monotone), so one reduction carries both the sum of squares
// and the maximum, and the row is read once.
//
// Bound by memory: 4 bytes read and 3 written an element (1 + 2 without the
// residual).  A row belongs to one workgroup and stays in registers as h * g
// (KEEP pieces of 8 elements a thread; longer rows read the rest again).
// On one MI355X: 16383x8192 to MXFP8 160 us, 5.9 TB/s of the bytes it needs (a
// copy runs at 5.1); 4096x7168 to e4m3 per 128 40 us, 5.1 TB/s; one row of 7168
// 4.2 us, which is a launch and two trips to memory.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "norm_dev.hpp"

namespace qgemm {

namespace {

// The h of piece p (8 elements) of the row.
template <bool RES>
__device__ __forceinline__ Piece load_h(const u32x4 *x, const u32x4 *r, int p)
{
    Piece h;
    const u32x4 a = __builtin_nontemporal_load(&x[p]);
    if constexpr (RES) {
        const u32x4 b = __builtin_nontemporal_load(&r[p]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h.v[2 * i] = lo_bf16(a[i]) + lo_bf16(b[i]);
            h.v[2 * i + 1] = hi_bf16(a[i]) + hi_bf16(b[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h.v[2 * i] = lo_bf16(a[i]);
            h.v[2 * i + 1] = hi_bf16(a[i]);
        }
    }
    return h;
}

template <int OUT, int THREADS, int KEEP, bool RES>
__global__ void __launch_bounds__(THREADS) rmsnorm_quant_kernel(NormArgs a)
{
    constexpr int WAVES = THREADS / 64;
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x;
    const u32x4 *x = (const u32x4 *)(a.X + row * a.ldx);
    const u32x4 *r = RES ? (const u32x4 *)(a.R + row * a.ldr) : nullptr;
    u32x4 *o = a.Rout ? (u32x4 *)(a.Rout + row * a.ldo) : nullptr;
    const u32x4 *g = (const u32x4 *)a.gamma;
    uint8_t *q = a.Q + row * a.ldq;
    const int np = a.K / 8;

    Piece keep[KEEP];
    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int p = t + THREADS * c;
        keep[c] = Piece{};
        if (p < np)
            keep[c] = load_h<RES>(x, r, p);
    }
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int p = t + THREADS * c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = fmaf(keep[c].v[i], keep[c].v[i], sum);
        if (p < np) {
            if (o)
                store_h(o, p, keep[c]);
            times_gamma(keep[c], g, p);
        }
        top = max_nan(top, max_abs(keep[c]));
    }
    for (int p = t + THREADS * KEEP; p < np; p += THREADS) {
        Piece h = load_h<RES>(x, r, p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = fmaf(h.v[i], h.v[i], sum);
        times_gamma(h, g, p);
        top = max_nan(top, max_abs(h));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        sum += __shfl_xor(sum, off);
        top = max_nan(top, __shfl_xor(top, off));
    }
    if constexpr (WAVES > 1) {
        __shared__ float wsum[WAVES], wtop[WAVES];
        if ((t & 63) == 0) {
            wsum[t >> 6] = sum;
            wtop[t >> 6] = top;
        }
        __syncthreads();
        sum = wsum[0];
        top = wtop[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            sum += wsum[w];
            top = max_nan(top, wtop[w]);
        }
    }
    const float rstd = inv_sqrt(sum / (float)a.K + a.eps);
    float row_scale = 0.0f;
    uint8_t *srow = (uint8_t *)a.S;
    if constexpr (OUT == NORM_I8_ROW || OUT == NORM_F8_ROW) {
        row_scale = (top * rstd) / (OUT == NORM_I8_ROW ? 127.0f : 448.0f);
        if (t == 0)
            ((float *)a.S)[row] = row_scale;
    } else {
        srow += row * a.lds * (OUT == NORM_F8_BLOCK ? 4 : 1);
    }
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int p = t + THREADS * c;
        emit<OUT>(keep[c], rstd, row_scale, p, p < np, q, srow);
    }
    // the rest of a long row: the loop's trip count is the workgroup's, so that
    // the lanes of a block stay together
    for (int p0 = THREADS * KEEP; p0 < np; p0 += THREADS) {
        const int p = p0 + t;
        Piece h{};
        if (p < np) {
            h = load_h<RES>(x, r, p);
            if (o)
                store_h(o, p, h);   // after the last read of r: o may be r or x
            times_gamma(h, g, p);
        }
        emit<OUT>(h, rstd, row_scale, p, p < np, q, srow);
    }
}

template <int OUT, int THREADS, int KEEP>
hipError_t launch_res(const NormArgs &a, hipStream_t s)
{
    if (a.R)
        hipLaunchKernelGGL((rmsnorm_quant_kernel<OUT, THREADS, KEEP, true>), dim3((unsigned)a.M), dim3(THREADS), 0, s, a);
    else
        hipLaunchKernelGGL((rmsnorm_quant_kernel<OUT, THREADS, KEEP, false>), dim3((unsigned)a.M), dim3(THREADS), 0, s, a);
    return hipGetLastError();
}

template <int OUT>
hipError_t launch_out(const NormArgs &a, hipStream_t s)
{
    const int np = a.K / 8;
    if (np <= 256)
        return launch_res<OUT, 256, 1>(a, s);
    if (np <= 512)
        return launch_res<OUT, 256, 2>(a, s);
    if (np <= 1024)
        return launch_res<OUT, 256, 4>(a, s);
    return launch_res<OUT, 256, 8>(a, s);
}

}  // namespace

hipError_t launch_rmsnorm_quant(int out, const NormArgs &all, hipStream_t s)
{
    // a launch holds fewer than 2^32 threads: more rows than that go in several
    constexpr int ROWS = 1 << 23;
    hipError_t e = hipSuccess;
    for (int64_t row = 0; row < all.M && e == hipSuccess; row += ROWS) {
        NormArgs a = all;
        a.M = (int)std::min<int64_t>(ROWS, all.M - row);
        a.X += row * a.ldx;
        a.R = a.R ? a.R + row * a.ldr : nullptr;
        a.Rout = a.Rout ? a.Rout + row * a.ldo : nullptr;
        a.Q += row * a.ldq;
        const int64_t scale = out <= NORM_F8_ROW ? 4 : a.lds * (out == NORM_F8_BLOCK ? 4 : 1);   // bytes a row
        a.S = (uint8_t *)a.S + row * scale;
        switch (out) {
        case NORM_I8_ROW: e = launch_out<NORM_I8_ROW>(a, s); break;
        case NORM_F8_ROW: e = launch_out<NORM_F8_ROW>(a, s); break;
        case NORM_F8_BLOCK: e = launch_out<NORM_F8_BLOCK>(a, s); break;
        case NORM_MX_E4M3: e = launch_out<NORM_MX_E4M3>(a, s); break;
        default: e = launch_out<NORM_MX_E2M1>(a, s); break;
        }
    }
    return e;
}

}  // namespace qgemm
