// postnorm.hip -- the norm after a block, its gate and residual scale, and the
// norm before the next block, written as the A operand and scales of the GEMM
// that follows.
//
//   n = y * rsqrt(mean(y^2) + eps) * gp      the block's output, normalised
//   h = r + alpha * (gate * n)               binary32
//   r' = bf16(h)                             the residual stream, handed on
//   z = (h * g) * rsqrt(mean(h^2) + eps)
//   code = enc(z / s)                        s by the GEMM's scale rule
//
// Nothing is rounded to fewer bits on the way but the outputs.  Two sums
// follow one another (h needs the first), so a row stays in the registers of
// its workgroup from y to the codes: y and r are read once, as bf16 (KEEP
// pieces of 8 elements a thread; longer rows read the rest again).  Bound by memory
// (one MI355X: 8191 x 5376 to blockscale 59 us, 5.2 TB/s, a copy's rate; one row of
// 7168 4.9 us, two sums' latency).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "norm_dev.hpp"

namespace qgemm {

namespace {

// h of a piece: y and r as loaded, p its place in the row.
template <bool GATE>
__device__ __forceinline__ Piece gated_sum(u32x4 y, u32x4 r, const u32x4 *gpost, const u32x4 *gate, float rstd,
                                           float alpha, int p)
{
    Piece h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h.v[2 * i] = lo_bf16(y[i]) * rstd;
        h.v[2 * i + 1] = hi_bf16(y[i]) * rstd;
    }
    times_gamma(h, gpost, p);
    if constexpr (GATE)
        times_gamma(h, gate, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h.v[2 * i] = lo_bf16(r[i]) + alpha * h.v[2 * i];
        h.v[2 * i + 1] = hi_bf16(r[i]) + alpha * h.v[2 * i + 1];
    }
    return h;
}

__device__ __forceinline__ float sum_squares(u32x4 y, float sum)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = fmaf(lo_bf16(y[i]), lo_bf16(y[i]), sum);
        sum = fmaf(hi_bf16(y[i]), hi_bf16(y[i]), sum);
    }
    return sum;
}

template <int OUT, int THREADS, int KEEP, bool GATE>
__global__ void __launch_bounds__(THREADS) postnorm_quant_kernel(PostnormArgs a)
{
    constexpr int WAVES = THREADS / 64;
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x;
    const u32x4 *y = (const u32x4 *)(a.Y + row * a.ldy);
    const u32x4 *r = (const u32x4 *)(a.R + row * a.ldr);
    u32x4 *o = a.Rout ? (u32x4 *)(a.Rout + row * a.ldo) : nullptr;
    const u32x4 *gp = (const u32x4 *)a.gpost, *gt = (const u32x4 *)a.gate, *g = (const u32x4 *)a.gamma;
    uint8_t *q = a.Q + row * a.ldq;
    const int np = a.K / 8;
    __shared__ float wsum[2][WAVES], wtop[WAVES];

    u32x4 ky[KEEP], kr[KEEP];
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int p = t + THREADS * c;
        ky[c] = kr[c] = u32x4{};
        if (p < np) {
            ky[c] = __builtin_nontemporal_load(&y[p]);
            kr[c] = __builtin_nontemporal_load(&r[p]);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < KEEP; ++c)
        sum = sum_squares(ky[c], sum);
    for (int p = t + THREADS * KEEP; p < np; p += THREADS)
        sum = sum_squares(y[p], sum);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        sum += __shfl_xor(sum, off);
    if ((t & 63) == 0)
        wsum[0][t >> 6] = sum;
    __syncthreads();
    sum = wsum[0][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
        sum += wsum[0][w];
    const float rpost = inv_sqrt(sum / (float)a.K + a.eps);

    Piece keep[KEEP];
    float top = 0.0f;
    sum = 0.0f;
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int p = t + THREADS * c;
        keep[c] = Piece{};
        if (p < np) {
            keep[c] = gated_sum<GATE>(ky[c], kr[c], gp, gt, rpost, a.alpha, p);
            if (o)
                store_h(o, p, keep[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum = fmaf(keep[c].v[i], keep[c].v[i], sum);
            times_gamma(keep[c], g, p);
        }
        top = max_nan(top, max_abs(keep[c]));
    }
    for (int p = t + THREADS * KEEP; p < np; p += THREADS) {
        Piece h = gated_sum<GATE>(y[p], r[p], gp, gt, rpost, a.alpha, p);
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
    if ((t & 63) == 0) {
        wsum[1][t >> 6] = sum;
        wtop[t >> 6] = top;
    }
    __syncthreads();
    sum = wsum[1][0];
    top = wtop[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        sum += wsum[1][w];
        top = max_nan(top, wtop[w]);
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
        emit<OUT, true>(keep[c], rstd, row_scale, p, p < np, q, srow);
    }
    // the rest of a long row: the loop's trip count is the workgroup's, so that
    // the lanes of a block stay together
    for (int p0 = THREADS * KEEP; p0 < np; p0 += THREADS) {
        const int p = p0 + t;
        Piece h{};
        if (p < np) {
            h = gated_sum<GATE>(y[p], r[p], gp, gt, rpost, a.alpha, p);
            if (o)
                store_h(o, p, h);   // after the last read of r and y: o may be either
            times_gamma(h, g, p);
        }
        emit<OUT, true>(h, rstd, row_scale, p, p < np, q, srow);
    }
}

template <int OUT, int THREADS, int KEEP>
hipError_t launch_gate(const PostnormArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)a.M), block(THREADS);
    if (a.gate)
        hipLaunchKernelGGL((postnorm_quant_kernel<OUT, THREADS, KEEP, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((postnorm_quant_kernel<OUT, THREADS, KEEP, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int OUT>
hipError_t launch_out(const PostnormArgs &a, hipStream_t s)
{
    const int np = a.K / 8;
    if (np <= 256)
        return launch_gate<OUT, 256, 1>(a, s);
    if (np <= 512)
        return launch_gate<OUT, 256, 2>(a, s);
    return launch_gate<OUT, 256, 4>(a, s);
}

}  // namespace

hipError_t launch_postnorm_quant(int out, const PostnormArgs &all, hipStream_t s)
{
    // a launch holds fewer than 2^32 threads: more rows than that go in several
    constexpr int ROWS = 1 << 23;
    hipError_t e = hipSuccess;
    for (int64_t row = 0; row < all.M && e == hipSuccess; row += ROWS) {
        PostnormArgs a = all;
        a.M = (int)std::min<int64_t>(ROWS, all.M - row);
        a.Y += row * a.ldy;
        a.R += row * a.ldr;
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
