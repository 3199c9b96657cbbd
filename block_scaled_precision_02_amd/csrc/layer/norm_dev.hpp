// norm_dev.hpp -- what the operators with quantised output share on the
// device: eight elements of a row in registers, the scale rules of the GEMMs'
// A operand, and the reciprocal square root.
#pragma once
#include "layer.hpp"
#include "layer_dev.hpp"

namespace qgemm {

struct Piece {
    float v[8];
};

__device__ __forceinline__ void store_h(u32x4 *o, int p, const Piece &h)
{
    const u32x4 v = {pack_bf16(h.v[0], h.v[1]), pack_bf16(h.v[2], h.v[3]), pack_bf16(h.v[4], h.v[5]),
                     pack_bf16(h.v[6], h.v[7])};
    __builtin_nontemporal_store(v, &o[p]);
}

__device__ __forceinline__ void times_gamma(Piece &h, const u32x4 *g, int p)
{
    const u32x4 w = g[p];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h.v[2 * i] *= lo_bf16(w[i]);
        h.v[2 * i + 1] *= hi_bf16(w[i]);
    }
}

// The larger one, NaN where either is: what is not a number in a row shows in
// its scale.
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ float max_abs(const Piece &h)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max_nan(m, fabsf(h.v[i]));
    return m;
}

// y / s for a piece.  The quotient by one reciprocal differs from the divided
// one by a unit in the last place at most, as y itself does from the formula's;
// where the reciprocal would overflow (a scale near the bottom of the range),
// the division itself.  DIVIDED: the divided one, by one step of correction (its
// residue is exact), where the scale is a number: two instructions an element,
// in the norm after a block hidden behind memory (8191 x 5376: 59 us with and
// without; the codes' distance from those of float32 division 5.8e-5 without, 8.5e-6
// with), in SwiGLU 4 to 7% (swiglu.hip).
template <bool DIVIDED = false>
__device__ __forceinline__ void over_scale(Piece &y, float s)
{
    if (s >= 0x1p-120f) {
        const float inv = 1.0f / s;
        if (DIVIDED && s < 0x1p120f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = y.v[i] * inv;
                y.v[i] = fmaf(fmaf(-q, s, y.v[i]), inv, q);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y.v[i] *= inv;
    } else if (s > 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y.v[i] /= s;
    }
}

// Codes and, for the block forms, scales of piece p, whose y is a * rstd.
// Every lane of the wave comes here (the block forms exchange maxima between
// lanes); live: whether the piece is in the row.
template <int OUT, bool DIVIDED = false>
__device__ __forceinline__ void emit(Piece y, float rstd, float row_scale, int p, bool live, uint8_t *q, uint8_t *srow)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y.v[i] *= rstd;
    if constexpr (OUT == NORM_I8_ROW || OUT == NORM_F8_ROW) {
        over_scale<DIVIDED>(y, row_scale);
    } else if constexpr (OUT == NORM_F8_BLOCK) {
        float m = live ? max_abs(y) : 0.0f;
#pragma unroll
        for (int off = 1; off < 16; off <<= 1)
            m = max_nan(m, __shfl_xor(m, off));
        const float s = m / 448.0f;
        over_scale<DIVIDED>(y, s);
        if (live && (p & 15) == 0)
            ((float *)srow)[p >> 4] = s;
    } else {
        constexpr unsigned EMAX = OUT == NORM_MX_E4M3 ? 8u : 2u;
        float m = live ? max_abs(y) : 0.0f;
        m = max_nan(m, __shfl_xor(m, 1));
        m = max_nan(m, __shfl_xor(m, 2));
        const unsigned E = (__float_as_uint(m) >> 23) & 0xffu;
        const unsigned code = E == 255u ? 255u : E > EMAX ? E - EMAX : 0u;   // 255: NaN
        const float mul = __uint_as_float((254u - code) << 23);   // 2^(127 - code), exact (255: any)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y.v[i] *= mul;
        if (live && (p & 3) == 0)
            srow[p >> 2] = (uint8_t)code;
    }
    if (!live)
        return;
    if constexpr (OUT == NORM_MX_E2M1) {
        __builtin_nontemporal_store(enc8_e2m1(y.v), (unsigned *)q + p);
    } else if constexpr (OUT == NORM_I8_ROW) {
        const u32x2 c = {enc4_i8(y.v[0], y.v[1], y.v[2], y.v[3]), enc4_i8(y.v[4], y.v[5], y.v[6], y.v[7])};
        __builtin_nontemporal_store(c, (u32x2 *)q + p);
    } else {
        const u32x2 c = {enc4_e4m3(y.v[0], y.v[1], y.v[2], y.v[3]), enc4_e4m3(y.v[4], y.v[5], y.v[6], y.v[7])};
        __builtin_nontemporal_store(c, (u32x2 *)q + p);
    }
}

// 1/sqrt(v), v >= 0, to half a unit in the last place (0 for 0: a zero row
// with eps 0 stays zero; NaN for NaN).  One Newton step on the hardware's estimate r,
// r + r (1 - v r^2) / 2, with the residual formed exactly: v r = t + u.
__device__ __forceinline__ float inv_sqrt(float v)
{
    if (!(v > 1e-30f && v < 1e30f))
        return v == 0.0f ? 0.0f : 1.0f / __builtin_sqrtf(v);
    const float r = __builtin_amdgcn_rsqf(v);
    const float t = v * r, u = fmaf(v, r, -t);
    const float e = fmaf(-u, r, fmaf(-t, r, 1.0f));
    return fmaf(0.5f * r, e, r);
}

}  // namespace qgemm
