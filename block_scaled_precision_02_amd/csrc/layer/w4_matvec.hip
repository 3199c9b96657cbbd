// w4_matvec.hip -- a few rows of bf16 activations times 4-bit weights with
// group scales, the projections of a decode step.
//
//   i4:  y[m,n] = sum_G s[n,G] ( sum_{k in G} x[m,k] w[n,k] - z[n,G] sum_{k in G} x[m,k] ) (+ bias[n])
//   mx:  y[m,n] = sum_k x[m,k] e2m1(w[n,k]) 2^(s[n,k/32] - 127) (+ bias[n])
//
// Bound by memory: half a byte a weight and its scales.  The weights go from
// memory to matrix-core operands; the matrix cores' 16-row product does the
// sums also for one row of x, because the vector units are busy enough turning
// 4-bit codes into bf16 (both exact):
//  * e2m1: the conversion instruction takes the scale along (a power of two).
//  * int4: a nibble OR-ed into the mantissa of 128 is the bf16 value 128 + w,
//    two a bit operation (nibbles j and j + 4 of a dword; x is taken in the
//    same order).  The 128 goes with the zero point: the sum of x over the
//    group comes from one more product, with ones.
// A wave's load is 16 bytes of each of 16 rows and 4 lane groups: 128 weights
// of a row side by side.  A product sums over 8 elements of every lane group,
// so that where a scale group is shorter than 128 the dwords are exchanged
// between the lane groups first (a 4x4 transposition, 4 lane swaps): product u
// then holds elements 32 u .. 32 u + 31.
// The workgroup's 8 waves split K and meet in LDS; the order of the sums is
// fixed.
#include <hip/hip_runtime.h>

#include "layer.hpp"
#include "layer_dev.hpp"

namespace qgemm {

namespace {

constexpr int W4_WAVES = 8;
constexpr int CHUNK = 128;   // weights of a row a wave takes at a time

// The four dwords of lane groups 0..3 transposed: lane group g ends with dword
// g of each lane group's four.
__device__ __forceinline__ u32x4 swap4(u32x4 w)
{
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

// Eight nibbles as 128 + w, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 nibbles_bf16(unsigned w)
{
    constexpr unsigned M = 0x000f000fu, B = 0x43004300u;
    return __builtin_bit_cast(bf16x8, u32x4{(w & M) | B, ((w >> 4) & M) | B, ((w >> 8) & M) | B, ((w >> 12) & M) | B});
}

// Eight e2m1 codes times scale (a power of two).
__device__ __forceinline__ bf16x8 e2m1_bf16(unsigned w, float scale)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// x in the nibbles' order.
__device__ __forceinline__ bf16x8 x_order(u32x4 x)
{
    return __builtin_bit_cast(bf16x8, u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u),
                                            __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                                            __builtin_amdgcn_perm(x[3], x[1], 0x05040100u),
                                            __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)});
}

// GROUP 0: mx; else i4 with that group.  MT 16-row tiles of x, of which RI of
// every 4 accumulators hold rows (row t of a tile stands in product row
// 4 (t % 4) + t / 4, so that 4 RI rows need RI of them).  NT 16-row tiles of
// weights a wave.
template <int GROUP, int MT, int RI, int NT>
__global__ void __launch_bounds__(W4_WAVES * 64) w4_matvec_kernel(W4Args a)
{
    constexpr bool MX = GROUP == 0;
    constexpr bool SWAP = GROUP == 32 || GROUP == 64;
    constexpr int SC = MX ? 1 : CHUNK / GROUP;   // scales of a chunk
    constexpr int U = 4 / NT;                    // chunks loaded ahead together
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * (16 * NT);
    const int chunks = (a.K + CHUNK - 1) / CHUNK, groups = a.K / (MX ? 32 : GROUP);
    const int c0 = chunks * wave / W4_WAVES, c1 = chunks * (wave + 1) / W4_WAVES;

    const uint8_t *w[NT];
    const uint8_t *sb[NT];
    const uint8_t *zb[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t n = min(n0 + 16 * t + r16, a.N - 1);
        w[t] = a.W + n * a.ldw + 16 * g;
        sb[t] = (const uint8_t *)a.S + (MX ? n / a.srows * groups : n * groups * 2);
        zb[t] = a.Z ? a.Z + n * groups : nullptr;
    }
    const uint16_t *x[MT];
    bool has[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int row = 16 * t + (r16 >> 2) + 4 * (r16 & 3);
        has[t] = row < a.M;
        x[t] = a.X + (int64_t)(has[t] ? row : 0) * a.ldx + (SWAP ? 8 : 32) * g;
    }

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            acc[i][t] = f32x4{0, 0, 0, 0};
    const u32x4 one4 = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, one4);

    for (int cb = c0; cb < c1; cb += U) {
        u32x4 wv[U][NT];
        unsigned sv[U][NT][SC], zv[U][NT][SC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = min(cb + u, c1 - 1);
            // a lane's weights past K (a last chunk of 32, 64 or 96): any that
            // are there, as x is zero for them
            const int64_t off = min((int64_t)c * (CHUNK / 2), (int64_t)(a.K / 2) - 16 * g - 16);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                wv[u][t] = __builtin_nontemporal_load((const u32x4 *)(w[t] + off));
                if constexpr (MX) {
                    sv[u][t][0] = sb[t][min(4 * c + g, groups - 1)];
                } else {
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        const int at = min(c * SC + j, groups - 1);
                        sv[u][t][j] = *(const uint16_t *)(sb[t] + 2 * at);
                        zv[u][t][j] = a.Z ? zb[t][at] : 8;
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = cb + u;
            if (c >= c1)
                break;
            u32x4 xv[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int k = c * CHUNK + (SWAP ? 32 * p : 8 * p);
                    const bool in = has[i] && (SWAP ? k < a.K : c * CHUNK + 32 * g < a.K);
                    xv[i][p] = in ? *(const u32x4 *)(x[i] + k) : u32x4{0, 0, 0, 0};
                }
            if constexpr (MX) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const unsigned s = sv[u][t][0];
                    const float scale = __uint_as_float(s == 255u ? 0x7fc00000u : s ? s << 23 : 0x00400000u);
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const bf16x8 wf = e2m1_bf16(wv[u][t][p], scale);
#pragma unroll
                        for (int i = 0; i < MT; ++i)
                            acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[i][p]),
                                                                                wf, acc[i][t], 0, 0, 0);
                    }
                }
            } else {
                constexpr int PG = 4 / SC;   // products of a scale group
                bf16x8 wf[NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const u32x4 v = SWAP ? swap4(wv[u][t]) : wv[u][t];
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        wf[t][p] = nibbles_bf16(v[p]);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        f32x4 xs = {0, 0, 0, 0}, part[NT];
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            part[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int p = j * PG; p < (j + 1) * PG; ++p) {
                            const bf16x8 xf = x_order(xv[i][p]);
                            xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, ones, xs, 0, 0, 0);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                part[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, wf[t][p], part[t], 0, 0, 0);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const float s = lo_bf16(sv[u][t][j]), z = 128.0f + (float)(int)zv[u][t][j];
#pragma unroll
                            for (int r = 0; r < RI; ++r)
                                acc[i][t][r] = fmaf(fmaf(-z, xs[r], part[t][r]), s, acc[i][t][r]);
                        }
                    }
                }
            }
        }
    }

    // the waves' sums, a tile at a time: [wave][product row][column]
    __shared__ float red[W4_WAVES][16][17];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (i || t)
                __syncthreads();
#pragma unroll
            for (int r = 0; r < RI; ++r)
                red[wave][4 * g + r][r16] = acc[i][t][r];
            __syncthreads();
            const int pr = threadIdx.x >> 4, col = threadIdx.x & 15;   // 16 x 16 of the 512 threads
            const int row = 16 * i + (pr >> 2) + 4 * (pr & 3), n = n0 + 16 * t + col;
            if (pr < 16 && row < a.M && n < a.N) {
                float y = 0.0f;
#pragma unroll
                for (int v = 0; v < W4_WAVES; ++v)
                    y += red[v][pr][col];
                if (a.bias)
                    y += lo_bf16(a.bias[n]);
                a.Y[(int64_t)row * a.ldy + n] = (uint16_t)pack_bf16(y, 0.0f);
            }
        }
}

template <int GROUP, int MT, int RI>
hipError_t launch_nt(const W4Args &a, hipStream_t s)
{
    constexpr int NT = 1;
    const unsigned grid = (unsigned)((a.N + 16 * NT - 1) / (16 * NT));
    hipLaunchKernelGGL((w4_matvec_kernel<GROUP, MT, RI, NT>), dim3(grid), dim3(W4_WAVES * 64), 0, s, a);
    return hipGetLastError();
}

template <int GROUP>
hipError_t launch_rows(const W4Args &a, hipStream_t s)
{
    if (a.M <= 4)
        return launch_nt<GROUP, 1, 1>(a, s);
    if (a.M <= 16)
        return launch_nt<GROUP, 1, 4>(a, s);
    if (a.M <= 32)
        return launch_nt<GROUP, 2, 4>(a, s);
    return launch_nt<GROUP, 4, 4>(a, s);
}

}  // namespace

hipError_t launch_w4_matvec(const W4Args &a, hipStream_t s)
{
    switch (a.group) {
    case 0: return launch_rows<0>(a, s);
    case 32: return launch_rows<32>(a, s);
    case 64: return launch_rows<64>(a, s);
    default: return launch_rows<128>(a, s);
    }
}

}  // namespace qgemm
