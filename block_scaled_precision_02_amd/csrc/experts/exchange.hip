// exchange.hip -- tokens' rows to their experts and back, and the gradients.
//
//   gather    xs[position[t,j]] = x[t]
//   combine   out[t] = residual[t] + sum_j w[t,j] y[position[t,j]]
//   gradient  dy[position[t,j]] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[position[t,j]]>
//
// (the gather's gradient is the combine without weights).  All three go by
// tokens: a token's row is read once, however many experts it has, and a row
// of the experts' order is touched by one token alone, so that no sum needs an
// atomic and every result is the same on every call.  Sums are binary32, in
// the order of j; each output is rounded once.
//
// Positions outside [0, rows) stand for no expert.
//
// Bound by memory (one MI355X: 8192 x 8 rows of 7168, gather and combine 215 us
// each, 5.2 TB/s, a copy's rate; 4095 x 6 of 5376, half of them here, gradient 63
// and gather's gradient 31 us, 5.1 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../layer/layer_dev.hpp"
#include "experts.hpp"

namespace qgemm {

namespace {

constexpr int THREADS = 256;

__global__ void __launch_bounds__(THREADS) moe_gather_kernel(ExchangeArgs a)
{
    const int64_t t = blockIdx.x;
    const int p = blockIdx.y * THREADS + threadIdx.x;
    if (p >= a.H / 8)
        return;
    const int32_t *pos = a.position + t * a.k;
    const u32x4 v = __builtin_nontemporal_load((const u32x4 *)(a.X + t * a.ldx) + p);
    for (int j = 0; j < a.k; ++j) {
        const int r = pos[j];
        if (r >= 0 && r < a.rows)
            __builtin_nontemporal_store(v, (u32x4 *)(a.O + (int64_t)r * a.ldo) + p);
    }
}

template <bool RES, bool WEIGHTS>
__global__ void __launch_bounds__(THREADS) moe_combine_kernel(ExchangeArgs a)
{
    const int64_t t = blockIdx.x;
    const int p = blockIdx.y * THREADS + threadIdx.x;
    if (p >= a.H / 8)
        return;
    const int32_t *pos = a.position + t * a.k;
    float acc[8] = {};
    if constexpr (RES) {
        const u32x4 v = __builtin_nontemporal_load((const u32x4 *)(a.X + t * a.ldx) + p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] = lo_bf16(v[i]);
            acc[2 * i + 1] = hi_bf16(v[i]);
        }
    }
    // four rows in flight
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        u32x4 v[4];
        float w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = j0 + u < a.k ? pos[j0 + u] : -1;
            const bool in = r >= 0 && r < a.rows;
            v[u] = u32x4{};
            w[u] = 0.0f;
            if (in) {
                v[u] = __builtin_nontemporal_load((const u32x4 *)(a.Y + (int64_t)r * a.ldy) + p);
                w[u] = WEIGHTS ? a.W[t * a.k + j0 + u] : 1.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * i] = fmaf(w[u], lo_bf16(v[u][i]), acc[2 * i]);
                acc[2 * i + 1] = fmaf(w[u], hi_bf16(v[u][i]), acc[2 * i + 1]);
            }
    }
    const u32x4 o = {pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]),
                     pack_bf16(acc[6], acc[7])};
    __builtin_nontemporal_store(o, (u32x4 *)(a.O + t * a.ldo) + p);
}

// A workgroup takes a token; dout's row stays in registers, KEEP pieces of 8
// elements a thread (longer rows in several passes over the experts' rows).
constexpr int KEEP = 4;

__global__ void __launch_bounds__(THREADS) moe_combine_grad_kernel(ExchangeArgs a)
{
    constexpr int WAVES = THREADS / 64;
    __shared__ float dots[WAVES][MOE_MAX_K];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int np = a.H / 8;
    const int32_t *pos = a.position + t * a.k;
    for (int p0 = 0; p0 < np; p0 += THREADS * KEEP) {
        u32x4 d[KEEP];
#pragma unroll
        for (int c = 0; c < KEEP; ++c) {
            const int p = p0 + THREADS * c + tid;
            d[c] = p < np ? __builtin_nontemporal_load((const u32x4 *)(a.X + t * a.ldx) + p) : u32x4{};
        }
        for (int j = 0; j < a.k; ++j) {
            const int r = pos[j];
            float dot = 0.0f;
            if (r >= 0 && r < a.rows) {
                const float w = a.W[t * a.k + j];
                const u32x4 *y = (const u32x4 *)(a.Y + (int64_t)r * a.ldy);
                u32x4 *o = (u32x4 *)(a.O + (int64_t)r * a.ldo);
                u32x4 v[KEEP];
#pragma unroll
                for (int c = 0; c < KEEP; ++c) {
                    const int p = p0 + THREADS * c + tid;
                    v[c] = p < np ? __builtin_nontemporal_load(&y[p]) : u32x4{};
                }
#pragma unroll
                for (int c = 0; c < KEEP; ++c) {
                    const int p = p0 + THREADS * c + tid;
                    u32x4 s;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        dot = fmaf(lo_bf16(d[c][i]), lo_bf16(v[c][i]), dot);
                        dot = fmaf(hi_bf16(d[c][i]), hi_bf16(v[c][i]), dot);
                        s[i] = pack_bf16(w * lo_bf16(d[c][i]), w * hi_bf16(d[c][i]));
                    }
                    if (p < np)
                        __builtin_nontemporal_store(s, &o[p]);   // after y's loads: o may be y
                }
            }
#pragma unroll
            for (int off = 32; off > 0; off >>= 1)
                dot += __shfl_xor(dot, off);
            if (lane == 0)
                dots[wave][j] = p0 == 0 ? dot : dots[wave][j] + dot;
        }
    }
    __syncthreads();
    if (tid < a.k) {
        float s = dots[0][tid];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            s += dots[w][tid];
        a.dW[t * a.k + tid] = s;
    }
}

// A launch holds fewer than 2^32 threads: f(a) on slices of the tokens.
template <class F>
hipError_t by_tokens(ExchangeArgs a, bool x_rows, bool o_rows, F &&f)
{
    const int per = std::max(1, (int)((1 << 23) / ((a.H / 8 + THREADS - 1) / THREADS)));
    hipError_t e = hipSuccess;
    for (int left = a.tokens; left > 0 && e == hipSuccess; left -= per) {
        a.tokens = std::min(left, per);
        e = f(a);
        a.position += (int64_t)per * a.k;
        if (a.W)
            a.W += (int64_t)per * a.k;
        if (a.dW)
            a.dW += (int64_t)per * a.k;
        if (a.X && x_rows)
            a.X += (int64_t)per * a.ldx;
        if (o_rows)
            a.O += (int64_t)per * a.ldo;
    }
    return e;
}

dim3 grid_of(const ExchangeArgs &a)
{
    return dim3((unsigned)a.tokens, (unsigned)((a.H / 8 + THREADS - 1) / THREADS));
}

}  // namespace

hipError_t launch_moe_gather(const ExchangeArgs &all, hipStream_t s)
{
    return by_tokens(all, true, false, [&](const ExchangeArgs &a) {
        hipLaunchKernelGGL(moe_gather_kernel, grid_of(a), dim3(THREADS), 0, s, a);
        return hipGetLastError();
    });
}

hipError_t launch_moe_combine(const ExchangeArgs &all, hipStream_t s)
{
    return by_tokens(all, true, true, [&](const ExchangeArgs &a) {
        const dim3 grid = grid_of(a), block(THREADS);
        if (a.X && a.W)
            hipLaunchKernelGGL((moe_combine_kernel<true, true>), grid, block, 0, s, a);
        else if (a.X)
            hipLaunchKernelGGL((moe_combine_kernel<true, false>), grid, block, 0, s, a);
        else if (a.W)
            hipLaunchKernelGGL((moe_combine_kernel<false, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((moe_combine_kernel<false, false>), grid, block, 0, s, a);
        return hipGetLastError();
    });
}

hipError_t launch_moe_combine_grad(const ExchangeArgs &all, hipStream_t s)
{
    return by_tokens(all, true, false, [&](const ExchangeArgs &a) {
        hipLaunchKernelGGL(moe_combine_grad_kernel, dim3((unsigned)a.tokens), dim3(THREADS), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace qgemm
