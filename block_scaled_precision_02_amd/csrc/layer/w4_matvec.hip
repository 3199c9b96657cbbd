// w4_matvec.hip -- a few rows of bf16 activations times 4-bit weights with
// group scales, the projections of a decode step.
//
//   i4:  y[m,n] = sum_G s[n,G] sum_{k in G} x[m,k] (w[n,k] - z[n,G]) (+ bias[n])
//   mx:  y[m,n] = sum_k x[m,k] e2m1(w[n,k]) 2^(s[n,k/32] - 127) (+ bias[n])
//
// Bound by memory: half a byte a weight and its scales.  The weights go from
// memory to matrix-core operands; the matrix cores' 16-row product does the
// sums also for one row of x, because the vector units are busy enough turning
// 4-bit codes into bf16 (both exact):
//  * e2m1: the conversion instruction takes the scale along (a power of two).
//  * int4: two masked nibbles of a dword (j and j + 4; x is taken in the same
//    order) are two subnormal binary16 numbers, which a mixed-precision fused
//    multiply-add turns into w - z in binary32; its upper half is the bf16
//    value (|w - z| <= 255 has 8 bits).  The products are the definition's own:
//    a weight at its zero point adds nothing, an infinite x gives infinities.
//    (Products with 128 + w, from which 128 + z times the sum of x was taken, need
//    one operation a weight in place of two, but round 17 times coarser and have
//    neither: 1x21504x5376 18.4 us in place of 20.4, 16x8192x8192 in groups of 32
//    26.4 in place of 25.3.)
// A wave's load is 16 bytes of each of 16 rows and 4 lane groups: 128 weights
// of a row side by side.  A product sums over 8 elements of every lane group,
// so that where a scale group is shorter than 128 the dwords are exchanged
// between the lane groups first (a 4x4 transposition, 4 lane swaps): product u
// then holds elements 32 u .. 32 u + 31.
// The workgroup's 8 waves split K and meet in LDS; the order of the sums is
// fixed.
// On one MI355X, weights not in a cache: 1x21504x5376 int4 in groups of 128 with
// zero points 20.4 us, 3.0 TB/s, 10 of them vector instructions, of which the
// nibbles are three in five; 1x8192x8192 MXFP4 11.4 us, 3.1 TB/s; 16x8192x8192
// MXFP4 20.5 us, in which the vector units issue for 4.4 and a wave waits for
// three quarters of its time: every workgroup lays out all of x for itself.
#include <hip/hip_runtime.h>

#include <algorithm>

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

// Eight nibbles less the zero point, in the order 0 4 1 5 2 6 3 7.  As the
// mantissa of a binary16 number a nibble w is w 2^-24, or w 2^-20 four bits up.
__device__ __forceinline__ bf16x8 nibbles_bf16(unsigned w, float z)
{
    constexpr unsigned M = 0x000f000fu;
    const unsigned part[4] = {w & M, w & (M << 4), (w >> 8) & M, (w >> 8) & (M << 4)};
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f16x2 h = __builtin_bit_cast(f16x2, part[i]);
        const float unit = i & 1 ? 0x1p20f : 0x1p24f;
        const float lo = fmaf((float)h[0], unit, -z), hi = fmaf((float)h[1], unit, -z);
        v[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
    return __builtin_bit_cast(bf16x8, v);
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

// The x of a chunk as product operands, from four loads of which number p holds
// elements 32 p + 8 g .. + 7 (the four lane groups side by side: 64 bytes of a
// row an instruction; a lane's own 32 elements would be 64 separate pieces).
// Where the weights are not exchanged between the lane groups, x is: product p
// then takes elements 32 g + 8 p of lane group g.
template <bool SWAP>
__device__ __forceinline__ void x_operands(u32x4 (&v)[4])
{
    if constexpr (!SWAP) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32x4 t = swap4(u32x4{v[0][i], v[1][i], v[2][i], v[3][i]});
#pragma unroll
            for (int p = 0; p < 4; ++p)
                v[p][i] = t[p];
        }
    }
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
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
        x[t] = a.X + (int64_t)(has[t] ? row : 0) * a.ldx + 8 * g;
    }

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            acc[i][t] = f32x4{0, 0, 0, 0};

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
                wv[u][t] = *(const u32x4 *)(w[t] + off);
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
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int k = c * CHUNK + 32 * p;
                    const bool in = has[i] && k < a.K;
                    xv[i][p] = *(const u32x4 *)(in ? x[i] + k : a.X);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        xv[i][p][e] = in ? xv[i][p][e] : 0u;
                }
                x_operands<SWAP>(xv[i]);
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
                        wf[t][p] = nibbles_bf16(v[p], (float)zv[u][t][p / PG]);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        f32x4 part[NT];
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            part[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int p = j * PG; p < (j + 1) * PG; ++p) {
                            const bf16x8 xf = x_order(xv[i][p]);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                part[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, wf[t][p], part[t], 0, 0, 0);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const float s = lo_bf16(sv[u][t][j]);
#pragma unroll
                            for (int r = 0; r < RI; ++r)
                                acc[i][t][r] = fmaf(part[t][r], s, acc[i][t][r]);
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

// The same for up to 16 rows and K up to 8192, the ordinary decode step: a
// workgroup stays and walks over 16-row tiles of weights.  Wave v's chunks are
// the same for every tile, so that x (XR rows of it) is laid out once in LDS in
// the order of the products' operands; a product's rows without a row of x repeat others, as nobody reads their sums.
// Up to four rows that leaves room for two workgroups a CU.  Where x is too
// long for LDS, K goes in parts, one walk each, with the tiles' sums kept in
// LDS between them.  A chunk's register takes the next tile's weights as soon
// as it is used.  A tile's scales lie side by side in memory: the workgroup
// fetches them 16 bytes a thread, a tile ahead, and takes them from LDS (a byte
// or two at a time from memory took 6 of 19 us at 1x8192x8192).
// CPW: chunks a wave and part, at most.
constexpr int LDS_BYTES = 160 * 1024;   // a workgroup's, at most

// A walk's LDS: the arrays of a fixed size, x, and the tiles' sums that are kept
// between the parts of a long K (1024 bytes a tile), for which the first two
// leave room for KEPT tiles a workgroup.
template <int GROUP, int XR, int CPW, bool ZERO>
struct WalkLds {
    static constexpr int W = W4_WAVES, SC = GROUP == 0 ? 4 : CHUNK / GROUP, ESZ = GROUP == 0 ? 1 : 2;
    static constexpr int RI = XR == 16 ? 4 : XR == 8 ? 2 : 1;   // accumulators that hold rows of x
    // a tile's scales and zero points: rows of K <= 8192, 16 bytes further apart
    // where they are whole 16-byte pieces (rows 256 bytes apart are one bank)
    static constexpr int KC = XR >= 8 ? 64 : W * CPW;           // chunks of a row, at most
    static constexpr int SB = 16 * (KC * SC * ESZ + 16), ZB = ZERO ? 16 * (KC * SC + 16) : 0;
    struct Fixed {
        float red[2][W][16][17];
        alignas(16) uint8_t tab[2][SB + ZB];
    };
    static constexpr int X = W * CPW * 16 * XR * 16, ROOM = (LDS_BYTES - X - (int)sizeof(Fixed)) / 1024;
    static constexpr int KEPT = ROOM < 8 ? ROOM : 8;
    static_assert(KEPT >= 1 && X + (int)sizeof(Fixed) + 1024 * KEPT <= LDS_BYTES, "a workgroup's LDS");
};

template <int GROUP, int XR, int CPW, bool ZERO>
__global__ void __launch_bounds__(W4_WAVES * 64, XR <= 4 ? 4 : 2) w4_walk_kernel(W4Args a)
{
    using Lds = WalkLds<GROUP, XR, CPW, ZERO>;
    constexpr int W = W4_WAVES;
    constexpr bool MX = GROUP == 0;
    constexpr bool SWAP = GROUP == 32 || GROUP == 64;
    constexpr int RI = Lds::RI;
    constexpr int SC = Lds::SC;                          // scales of a chunk
    constexpr int PG = 4 / SC;                           // products of a scale
    constexpr int ESZ = Lds::ESZ;                        // bytes of a scale
    constexpr int SB = Lds::SB;
    constexpr int NX = (CPW * XR + 3) / 4;               // 16-byte pieces of x a thread lays out
    extern __shared__ u32x4 xl[];                        // [chunk][product][lane group][XR], then the tiles' sums
    __shared__ typename Lds::Fixed fixed;
    auto &red = fixed.red;
    auto &tab = fixed.tab;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int chunks = (a.K + CHUNK - 1) / CHUNK, groups = a.K / (MX ? 32 : GROUP);
    const int parts = (chunks + W * CPW - 1) / (W * CPW);
    const int tiles = (a.N + 15) / 16, step = gridDim.x;
    const int pr = threadIdx.x >> 4, col = threadIdx.x & 15, xr = (pr >> 2) + 4 * (pr & 3);   // a result's place
    float *const kept = (float *)(xl + W * CPW * 16 * XR) + threadIdx.x;                      // 256 a tile

    // bytes of a row's scales, of a tile's (a 32-row scale: one row, for two
    // tiles), of the whole arrays; the pitch and this thread's place in LDS
    const int srows = MX ? a.srows : 1, row_b = groups * ESZ, lim = (srows == 1 ? 16 : 1) * row_b;
    const int at_t = 16 * threadIdx.x;
    const int s_pitch = row_b + (row_b % 16 ? 0 : 16), z_pitch = groups + (groups % 16 ? 0 : 16);
    const int s_to = row_b % 16 ? at_t : at_t + 16 * (at_t / row_b);
    [[maybe_unused]] const int z_to = SB + (groups % 16 ? at_t : at_t + 16 * (at_t / groups));
    const int64_t s_all = (int64_t)((a.N + srows - 1) / srows) * row_b;
    const auto start = [&](int tile) { return (int64_t)(tile * 16 / srows) * row_b; };
    u32x4 wv[CPW], sv, zv;   // the weights, and this thread's 16 bytes of scales and zero points
    const auto load_scales = [&](int tile) {
        const int64_t at = start(tile) + at_t;
        sv = *(const u32x4 *)((const uint8_t *)a.S + (at_t < lim && at + 16 <= s_all ? at : 0));
        if constexpr (ZERO) {
            const int64_t az = start(tile) / 2 + at_t;
            zv = *(const u32x4 *)(a.Z + (at_t < lim / 2 && az + 16 <= s_all / 2 ? az : 0));
        }
    };
    // the scales to LDS; what lies past the arrays' last whole 16 bytes comes
    // byte by byte
    const auto stage = [&](int tile, uint8_t *to) {
        const int64_t at = start(tile) + at_t;
        if (at_t < lim) {
            if (at + 16 <= s_all)
                *(u32x4 *)(to + s_to) = sv;
            else
                for (int i = 0; i < 16 && at + i < s_all; ++i)
                    to[s_to + i] = ((const uint8_t *)a.S)[at + i];
        }
        if constexpr (ZERO) {
            const int64_t az = start(tile) / 2 + at_t;
            if (at_t < lim / 2) {
                if (az + 16 <= s_all / 2)
                    *(u32x4 *)(to + z_to) = zv;
                else
                    for (int i = 0; i < 16 && az + i < s_all / 2; ++i)
                        to[z_to + i] = a.Z[az + i];
            }
        }
    };
    const auto weights = [&](int tile) { return a.W + (int64_t)min(tile * 16 + r16, a.N - 1) * a.ldw + 16 * g; };
    // the row of x that stands in a product's row
    const int xslot = XR == 1 ? 0 : XR == 4 ? r16 >> 2 : XR == 8 ? (r16 >> 2) + 4 * (r16 & 1) : (r16 >> 2) + 4 * (r16 & 3);

    for (int part = 0; part < parts; ++part) {
        const int p0 = chunks * part / parts, pn = chunks * (part + 1) / parts - p0;   // W <= pn <= W * CPW
        const int l0 = pn * wave / W, c0 = p0 + l0, nc = pn * (wave + 1) / W - l0;     // 1 <= nc <= CPW
        // every wave loads CPW chunks, its last one again past its own count;
        // weights past K (a last chunk of 32, 64 or 96) are any that are there,
        // as x is zero for them
        const auto load_chunk = [&](const uint8_t *w, int c) {
            const int off = min((c0 + min(c, nc - 1)) * (CHUNK / 2), a.K / 2 - 16 * g - 16);
            return *(const u32x4 *)(w + off);
        };
        const auto operand = [&](int c, int p) {
            return __builtin_bit_cast(bf16x8, xl[(((l0 + c) * 4 + p) * 4 + g) * XR + xslot]);
        };
        if (part)
            __syncthreads();   // x and the tables of the part before are done with
        // x first: what is loaded first is there first
        u32x4 xp[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int at = threadIdx.x + i * (W * 64);
            const int row = at % XR, pg = at / XR % 16, c = p0 + at / XR / 16;
            const int k = c * CHUNK + (SWAP ? 8 * pg : 32 * (pg & 3) + 8 * (pg >> 2));
            const bool in = row < a.M && k < a.K;
            xp[i] = *(const u32x4 *)(in ? a.X + (int64_t)row * a.ldx + k : a.X);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                xp[i][e] = in ? xp[i][e] : 0u;
        }
        __builtin_amdgcn_sched_barrier(0);
        load_scales(blockIdx.x);
        {
            const uint8_t *w = weights(blockIdx.x);
#pragma unroll
            for (int c = 0; c < CPW; ++c)
                wv[c] = load_chunk(w, c);
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int at = threadIdx.x + i * (W * 64);
            if (at < pn * 16 * XR)
                xl[at] = MX ? xp[i] : __builtin_bit_cast(u32x4, x_order(xp[i]));
        }
        stage(blockIdx.x, tab[0]);
        __syncthreads();
        // A tile: its sums, with the next one's loads; the next one's scales to
        // LDS; one barrier (a buffer's last readers have passed the barrier of
        // the tile between); the result.
        int flip = 0, nth = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += step, flip ^= 1, ++nth) {
            const int next = min(tile + step, tiles - 1);
            const bool more = tile + step < tiles;   // weights past the last tile cost 3 of 14 us at 1x8192x8192, MXFP4
            const uint8_t *w = weights(next), *sz = tab[flip];
            load_scales(next);
            // x is the same for every tile: an offset that the compiler cannot see
            // through keeps it in LDS and out of the registers
            int here = 0;
            asm volatile("" : "+s"(here));
            f32x4 acc = {0, 0, 0, 0};
            const int row = min(r16, a.N - 1 - tile * 16);
            const uint8_t *srow = sz + (srows == 1 ? row * s_pitch : 0);
            [[maybe_unused]] const uint8_t *zrow = sz + SB + row * z_pitch;
#pragma unroll
            for (int c = 0; c < CPW; ++c) {
                if (c >= nc)
                    break;
                const u32x4 wc = wv[c];
                if (more)
                    wv[c] = load_chunk(w, c);
                const int at = (c0 + c) * SC;
                if constexpr (MX) {
                    // a group past K (x is zero there) takes any scale of the row
                    const unsigned s = srow[min(at + g, groups - 1)];
                    const float scale = __uint_as_float(s == 255u ? 0x7fc00000u : s ? s << 23 : 0x00400000u);
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(c + here, p), e2m1_bf16(wc[p], scale), acc, 0,
                                                                      0, 0);
                } else {
                    const u32x4 v = SWAP ? swap4(wc) : wc;
                    struct alignas(2 * SC) Scales {
                        uint16_t s[SC];
                    };
                    struct alignas(SC) Zeros {
                        uint8_t z[SC];
                    };
                    const Scales s4 = *(const Scales *)(srow + 2 * at);
                    [[maybe_unused]] Zeros z4;
                    if constexpr (ZERO)
                        z4 = *(const Zeros *)(zrow + at);
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        const float z = ZERO ? (float)z4.z[j] : 8.0f;
                        f32x4 part_sum = {0, 0, 0, 0};
#pragma unroll
                        for (int p = j * PG; p < (j + 1) * PG; ++p)
                            part_sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(c + here, p),
                                                                               nibbles_bf16(v[p], z), part_sum, 0, 0, 0);
                        const float s = __uint_as_float((unsigned)s4.s[j] << 16);
#pragma unroll
                        for (int r = 0; r < RI; ++r)
                            acc[r] = fmaf(part_sum[r], s, acc[r]);
                    }
                }
            }
            stage(next, tab[flip ^ 1]);
#pragma unroll
            for (int r = 0; r < RI; ++r)
                red[flip][wave][4 * g + r][r16] = acc[r];
            __syncthreads();
            const int n = tile * 16 + col;
            if (pr < 16 && xr < a.M && n < a.N) {
                float y = 0.0f;
#pragma unroll
                for (int v = 0; v < W; ++v)
                    y += red[flip][v][pr][col];
                if (part)
                    y += kept[256 * nth];   // this thread's own
                if (part + 1 < parts) {
                    kept[256 * nth] = y;
                } else {
                    if (a.bias)
                        y += lo_bf16(a.bias[n]);
                    a.Y[(int64_t)xr * a.ldy + n] = (uint16_t)pack_bf16(y, 0.0f);
                }
            }
        }
    }
}

template <int GROUP, int MT, int RI, int NT>
hipError_t launch_tiles(const W4Args &all, hipStream_t s)
{
    // a launch holds fewer than 2^32 threads: more rows of weights than that go
    // in several (a multiple of 32, an MX scale's rows)
    constexpr int ROWS = 1 << 26;
    hipError_t e = hipSuccess;
    for (int64_t n = 0; n < all.N && e == hipSuccess; n += ROWS) {
        W4Args a = all;
        a.N = (int)std::min<int64_t>(ROWS, all.N - n);
        a.W += n * a.ldw;
        a.S = (const uint8_t *)a.S + n / a.srows * (a.K / (GROUP ? GROUP : 32)) * (GROUP ? 2 : 1);
        a.Z = a.Z ? a.Z + n * (a.K / (GROUP ? GROUP : 32)) : nullptr;
        a.bias = a.bias ? a.bias + n : nullptr;
        a.Y += n;
        hipLaunchKernelGGL((w4_matvec_kernel<GROUP, MT, RI, NT>), dim3((unsigned)((a.N + 16 * NT - 1) / (16 * NT))),
                           dim3(W4_WAVES * 64), 0, s, a);
        e = hipGetLastError();
    }
    return e;
}

template <int GROUP, int MT, int RI>
hipError_t launch_wide(const W4Args &a, hipStream_t s)
{
    // two tiles of weights a wave halve the loads of x, where that leaves a
    // workgroup a CU (MXFP4, 64 rows, 8192x8192: 42 us against 67; 32 rows,
    // 2112x7168: 23 against 19)
    if constexpr (MT > 1) {
        if (a.N >= 8192)
            return launch_tiles<GROUP, MT, RI, 2>(a, s);
    }
    return launch_tiles<GROUP, MT, RI, 1>(a, s);
}

template <int GROUP, int XR, int CPW, bool ZERO>
hipError_t launch_zeros(const W4Args &a, hipStream_t s)
{
    using Lds = WalkLds<GROUP, XR, CPW, ZERO>;
    constexpr int NUM_CU = 256;
    const int tiles = (a.N + 15) / 16, chunks = (a.K + CHUNK - 1) / CHUNK;
    // as many workgroups as are resident: two a CU while LDS has room for both
    // (int4 in groups of 64, one and two: 4x8192x8192, 64 KB of x, 15.4 us and
    // 19.7; 1x20000x2048 10.9 and 9.1; 1x21504x5376 23.0 and 21.8)
    int wgs = Lds::X <= 32768 && XR <= 4 ? 2 * NUM_CU : NUM_CU, kept = 0;
    if (chunks > W4_WAVES * CPW) {   // K in parts: no more tiles a workgroup than have room for their sums
        wgs = std::max(wgs, (tiles + Lds::KEPT - 1) / Lds::KEPT);
        kept = (tiles + wgs - 1) / wgs;
    }
    hipLaunchKernelGGL((w4_walk_kernel<GROUP, XR, CPW, ZERO>), dim3((unsigned)std::min(tiles, wgs)),
                       dim3(W4_WAVES * 64), Lds::X + kept * 1024, s, a);
    return hipGetLastError();
}

template <int GROUP, int XR, int CPW>
hipError_t launch_cpw(const W4Args &a, hipStream_t s)
{
    if constexpr (GROUP != 0) {
        if (a.Z)
            return launch_zeros<GROUP, XR, CPW, true>(a, s);
    }
    return launch_zeros<GROUP, XR, CPW, false>(a, s);
}

template <int GROUP, int XR>
hipError_t launch_walk(const W4Args &a, hipStream_t s)
{
    // 64 KB of x a part, or 128 where the scales leave room; longer K in parts
    constexpr int MOST = XR == 16 ? (GROUP == 0 ? 4 : 3) : XR == 8 ? 4 : 8;
    const int cpw = ((a.K + CHUNK - 1) / CHUNK + W4_WAVES - 1) / W4_WAVES;
    if (cpw <= 1)
        return launch_cpw<GROUP, XR, 1>(a, s);
    if (cpw <= 2)
        return launch_cpw<GROUP, XR, 2>(a, s);
    if constexpr (MOST == 8) {
        if (cpw <= 4)
            return launch_cpw<GROUP, XR, 4>(a, s);
        if (cpw <= 6)
            return launch_cpw<GROUP, XR, 6>(a, s);
    }
    return launch_cpw<GROUP, XR, MOST>(a, s);
}

template <int GROUP>
hipError_t launch_rows(const W4Args &a, hipStream_t s)
{
    const int chunks = (a.K + CHUNK - 1) / CHUNK;
    const int64_t groups = a.K / (GROUP ? GROUP : 32);
    // the walk has a chunk for every wave, eight at most, and reads scales 16
    // bytes at a time; int4's groups a chunk at a time
    const bool walk = a.M <= 16 && (GROUP == 0 || a.K % CHUNK == 0) && chunks >= W4_WAVES && chunks <= 8 * W4_WAVES && (uintptr_t)a.S % 16 == 0 &&
                      (uintptr_t)a.Z % 16 == 0 && (a.srows == 1 || groups % 16 == 0) &&
                      a.N * groups >= 16 * a.srows;
    if (walk) {
        if (a.M == 1)
            return launch_walk<GROUP, 1>(a, s);
        if (a.M <= 4)
            return launch_walk<GROUP, 4>(a, s);
        return a.M <= 8 ? launch_walk<GROUP, 8>(a, s) : launch_walk<GROUP, 16>(a, s);
    }
    if (a.M <= 4)
        return launch_wide<GROUP, 1, 1>(a, s);
    if (a.M <= 16)
        return launch_wide<GROUP, 1, 4>(a, s);
    if (a.M <= 32)
        return launch_wide<GROUP, 2, 4>(a, s);
    return launch_wide<GROUP, 4, 4>(a, s);
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
