// kv8_dev.hpp -- the 8-bit cache on the device: its layout, the exact code
// conversions, and what both attention kernels share.
//
// Layout, per physical block of bs tokens (16, 32, 64 or 128) and kv head:
//   K codes [bs][D] -- a token's row is what a matrix-core operand takes along
//     the head dimension
//   V codes [D][bs] -- transposed, so that a lane's 16-byte load is 16 tokens
//     of one channel: the operand of the product with the probabilities,
//     whose sum runs over tokens, without a transposition through LDS
//   one fp32 scale each for the block's K and V of that head
#pragma once
#include "layer.hpp"
#include "layer_dev.hpp"

namespace qgemm {

// Four codes (a dword) as four bf16; both conversions are exact.
template <int FMT>
__device__ __forceinline__ u32x2 codes4_bf16(unsigned w)
{
    if constexpr (FMT == KV8_E4M3) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
        return u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
    } else {
        // (the compiler would take the dword apart where it is loaded, and hold
        // four registers for one until it is used)
        asm("" : "+v"(w));
        // an int8 has at most 7 significant bits besides its sign: the upper
        // half of its binary32 form is the bf16 value
        const unsigned a = __float_as_uint((float)(int8_t)w), b = __float_as_uint((float)(int8_t)(w >> 8));
        const unsigned c = __float_as_uint((float)(int8_t)(w >> 16)), d = __float_as_uint((float)(int8_t)(w >> 24));
        return u32x2{__builtin_amdgcn_perm(b, a, 0x07060302u), __builtin_amdgcn_perm(d, c, 0x07060302u)};
    }
}

// Eight codes as a matrix-core operand register group.
template <int FMT>
__device__ __forceinline__ bf16x8 codes8_bf16(unsigned w0, unsigned w1)
{
    const u32x2 a = codes4_bf16<FMT>(w0), b = codes4_bf16<FMT>(w1);
    return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
}

// The same in binary16 (exact too: e4m3 spans 2^-9 .. 448, int8 has 7 bits).
template <int FMT>
__device__ __forceinline__ u32x2 codes4_f16(unsigned w)
{
    if constexpr (FMT == KV8_E4M3) {
        const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
        const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
        return u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
    } else {
        asm("" : "+v"(w));
        const auto lo = __builtin_amdgcn_cvt_pkrtz((float)(int8_t)w, (float)(int8_t)(w >> 8));
        const auto hi = __builtin_amdgcn_cvt_pkrtz((float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24));
        return u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
    }
}

template <int FMT>
__device__ __forceinline__ f16x8 codes8_f16(unsigned w0, unsigned w1)
{
    const u32x2 a = codes4_f16<FMT>(w0), b = codes4_f16<FMT>(w1);
    return __builtin_bit_cast(f16x8, u32x4{a[0], a[1], b[0], b[1]});
}

// Four codes as binary32.
template <int FMT>
__device__ __forceinline__ void codes4_f32(unsigned w, float (&v)[4])
{
    const u32x2 a = codes4_bf16<FMT>(w);
    v[0] = lo_bf16(a[0]);
    v[1] = hi_bf16(a[0]);
    v[2] = lo_bf16(a[1]);
    v[3] = hi_bf16(a[1]);
}

template <int FMT>
__device__ __forceinline__ unsigned enc4(float a, float b, float c, float d)
{
    if constexpr (FMT == KV8_E4M3)
        return enc4_e4m3(a, b, c, d);
    else
        return enc4_i8(a, b, c, d);
}

// What a block's V scale does to a probability, see kv8_stream.hip: its log2
// and its reciprocal.  Where the scale is zero the codes are cleared
// and the last other scale stands in (held: per lane, starts at 1).
struct VScale {
    float log2, inv;
};
__device__ __forceinline__ VScale v_scale(float s, float &held)
{
    if (s > 0.0f)
        held = fmaxf(s, 0x1p-100f);
    return VScale{__builtin_amdgcn_logf(held), __builtin_amdgcn_rcpf(held)};
}

// What a block's scores are multiplied by.  A NaN V scale makes it NaN, and so
// the weights of the rows that see the block, and theirs alone.
__device__ __forceinline__ float score_scale(float sk, float sv, float scale2) { return fmaf(sk, scale2, sv - sv); }

// The weights enter the second product as binary16 between 0 and 2^15.
constexpr float W_TOP = 15.0f;

// A row's sum of weights (up to 2^15) over their V scales is kept in units of
// 2^19: 2^31 tokens at the smallest scale, 2^-100, add up to 2^127 units, and one
// at the largest that bf16 values lead to, 2^121, is 2^-125 of them (the tiled
// kernel's weights may be 2^8 smaller: 16 bits of a subnormal number).
constexpr float SUM_UNIT = 0x1p-19f;

// A row's result is its accumulators times pre over sum: pre is a power of two
// that keeps the reciprocal and the products in range, sum infinite where the
// row has seen nothing (its accumulators are 0 and stay so).  A sum that is not
// a number (a query's NaN) stays one.
struct RowSum {
    float pre, sum;
};
__device__ __forceinline__ RowSum row_sum(float units)
{
    const float e = units < 1.0f ? 0x1p32f : 0x1p-32f;
    return RowSum{SUM_UNIT * e, units == 0.0f ? __builtin_inff() : units * e};
}

// The keys that a sequence's new token t (of q, the cache holding n tokens
// with them) sees: [lo, hi).
struct Span {
    int lo, hi;
};
__device__ __forceinline__ Span span_of(int t, int q, int n, int causal, int window)
{
    if (!causal)
        return Span{0, n};
    const int hi = max(min(n - q + t + 1, n), 0);
    return Span{window > 0 ? max(hi - window, 0) : 0, hi};
}

}  // namespace qgemm
