// layer_dev.hpp -- device helpers shared by the decoder-layer operators
// (norm, 8-bit cache, 4-bit matvec).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace qgemm {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float lo_bf16(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(unsigned w) { return __uint_as_float(w & 0xffff0000u); }

// Two binary32 values as a dword of bf16, nearest even.
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi)
{
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(unsigned, v);
}

// Two binary32 values as a dword of binary16, nearest even.
__device__ __forceinline__ unsigned pack_f16(float lo, float hi)
{
    const f16x2 v = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(unsigned, v);
}

// Four e4m3fn codes, nearest even.  The conversion instruction turns
// magnitudes past 448 into NaN, so they are clamped first; over every finite
// binary32 input the clamped form equals the library's software encoder.
__device__ __forceinline__ unsigned enc4_e4m3(float a, float b, float c, float d)
{
    a = __builtin_amdgcn_fmed3f(a, -448.0f, 448.0f);
    b = __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f);
    c = __builtin_amdgcn_fmed3f(c, -448.0f, 448.0f);
    d = __builtin_amdgcn_fmed3f(d, -448.0f, 448.0f);
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// Four int8 codes, nearest even, clamped to +-127: added to 3 * 2^22, a value
// is rounded to a whole number whose low byte is the code.
__device__ __forceinline__ unsigned enc4_i8(float a, float b, float c, float d)
{
    constexpr float ROUND = 12582912.0f;
    const unsigned ia = __float_as_uint(__builtin_amdgcn_fmed3f(a, -127.0f, 127.0f) + ROUND);
    const unsigned ib = __float_as_uint(__builtin_amdgcn_fmed3f(b, -127.0f, 127.0f) + ROUND);
    const unsigned ic = __float_as_uint(__builtin_amdgcn_fmed3f(c, -127.0f, 127.0f) + ROUND);
    const unsigned id = __float_as_uint(__builtin_amdgcn_fmed3f(d, -127.0f, 127.0f) + ROUND);
    const unsigned lo = __builtin_amdgcn_perm(ib, ia, 0x0c0c0400u), hi = __builtin_amdgcn_perm(id, ic, 0x0c0c0400u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// Eight e2m1 codes in a dword, element i in bits 4i .. 4i+3 (the conversion
// saturates by itself; equal to the software encoder on every finite input).
__device__ __forceinline__ unsigned enc8_e2m1(const float (&v)[8])
{
    unsigned w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
    return w;
}

}  // namespace qgemm
