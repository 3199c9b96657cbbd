// kv8_append.hip -- new keys and values into the 8-bit cache.
//
// For each block of tokens that a sequence's new tokens touch, and each head,
// K and V apart:
//   s' = max(s, amax(new) * (1 / qmax))   s counts only where the block already
//                                         holds older tokens of the sequence
//   code = enc(x / s')                nearest even, the IEEE quotient
//   older codes become enc(code * s / s') where s' > s, and stay otherwise
// Bound by memory (2 bytes read, 1 written an element) for prompts, by
// latency for single tokens.  One workgroup a block, head and operand: it owns
// all bytes that its scale governs, so that no scale is seen half updated and
// no atomics are needed.  A NaN or an infinity among the new values makes the
// scale NaN, which the maximum hands on to later appends.  On one MI355X: 64 single tokens of 8 heads of 128
// 6.2 to 6.7 us (5.2 the shortest); six prompts, 19002 tokens in all, 36 to 39 us,
// 3.1 TB/s of the bytes they need: a workgroup's loads, maximum, quotients and
// stores follow one another (waves wait for two thirds of their time, the vector
// units issue for 16 us), and five workgroups a CU cover for each other only in part (workgroups of 512
// threads 41 us, registers held to 6 waves a SIMD 58).  Bytes of tokens at or past the sequence's length
// keep what they held.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv8_dev.hpp"

namespace qgemm {

namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_KEEP = 2;   // 16-byte pieces of new rows a thread keeps

// x / s, correctly rounded: with inv the correctly rounded reciprocal, a
// residual step on a quotient within a unit in the last place gives the
// rounded one (Markstein, 1990), while nothing leaves the normal range; else
// the division itself.  x * inv alone can be off by more than a unit, so that
// it takes two steps.  The residual of a zero is +0: the sign is x's (SIGNED:
// the code keeps a zero's).
template <bool SIGNED>
struct Divider {
    float s, inv;
    bool fast;
    __device__ __forceinline__ explicit Divider(float scale)
    {
        s = scale > 0.0f ? scale : 1.0f;   // scale 0: all values are zeros and keep their signs
        fast = s > 0x1p-60f && s < 0x1p60f;
        inv = 1.0f / s;
    }
    __device__ __forceinline__ float operator()(float x) const
    {
        if (!fast)
            return x / s;
        float q = x * inv;
        q = fmaf(fmaf(-q, s, x), inv, q);
        q = fmaf(fmaf(-q, s, x), inv, q);
        return SIGNED ? __builtin_copysignf(q, x) : q;
    }
};

template <int FMT>
__device__ __forceinline__ u32x2 enc_piece(u32x4 w, const Divider<FMT == KV8_E4M3> &d)
{
    return u32x2{enc4<FMT>(d(lo_bf16(w[0])), d(hi_bf16(w[0])), d(lo_bf16(w[1])), d(hi_bf16(w[1]))),
                 enc4<FMT>(d(lo_bf16(w[2])), d(hi_bf16(w[2])), d(lo_bf16(w[3])), d(hi_bf16(w[3])))};
}

template <int FMT>
__device__ __forceinline__ unsigned requantise(unsigned w, float was, const Divider<FMT == KV8_E4M3> &d)
{
    float v[4];
    codes4_f32<FMT>(w, v);
    return enc4<FMT>(d(v[0] * was), d(v[1] * was), d(v[2] * was), d(v[3] * was));
}

// The larger one, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// The byte mask of the tokens [lo, hi) among the four from t0 on.
__device__ __forceinline__ unsigned byte_mask(int t0, int lo, int hi)
{
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (t0 + i >= lo && t0 + i < hi)
            m |= 0xffu << (8 * i);
    return m;
}

// Rows of four codes (channels 4c .. 4c+3 of four tokens) to four columns.
__device__ __forceinline__ u32x4 transpose4(unsigned a, unsigned b, unsigned c, unsigned d)
{
    const unsigned ab_lo = __builtin_amdgcn_perm(b, a, 0x05010400u);   // a0 b0 a1 b1
    const unsigned cd_lo = __builtin_amdgcn_perm(d, c, 0x05010400u);
    const unsigned ab_hi = __builtin_amdgcn_perm(b, a, 0x07030602u);   // a2 b2 a3 b3
    const unsigned cd_hi = __builtin_amdgcn_perm(d, c, 0x07030602u);
    return u32x4{__builtin_amdgcn_perm(cd_lo, ab_lo, 0x05040100u), __builtin_amdgcn_perm(cd_lo, ab_lo, 0x07060302u),
                 __builtin_amdgcn_perm(cd_hi, ab_hi, 0x05040100u), __builtin_amdgcn_perm(cd_hi, ab_hi, 0x07060302u)};
}

template <int D, int FMT>
__global__ void __launch_bounds__(AP_THREADS) kv8_append_kernel(Kv8Append a)
{
    constexpr int PR = D / 8;             // pieces a row
    constexpr int PITCH = D / 4 + 1;      // dwords a staged row
    extern __shared__ unsigned stage[];   // V only: [bs][PITCH] codes of the new tokens
    __shared__ float wtop[AP_THREADS / 64];
    const int t = threadIdx.x, bs = a.bs;
    const int head = blockIdx.y >> 1, is_v = blockIdx.y & 1, b = blockIdx.z;
    const int c0 = a.cu[b], q = a.cu[b + 1] - c0, len = a.lens[b];
    const int start = len - q;
    if (q <= 0 || len <= 0)
        return;
    const int64_t blk = (int64_t)(max(start, 0) / bs) + a.at + blockIdx.x;
    if (blk >= a.width || blk * bs >= len)
        return;
    const int first = (int)(blk * bs);
    const int lo = max(start, first), hi = min(len, first + bs);   // new tokens of this block
    if (lo >= hi)
        return;
    const int id = a.table[b * a.ldt + blk];
    const int64_t src = (int64_t)c0 + (lo - start);                // the first one's row of K / V
    const int n = hi - lo;
    if ((unsigned)id >= (unsigned)a.blocks || src < 0 || src + n > a.tokens)
        return;
    const int64_t ld = is_v ? a.ldv : a.ldk;
    const uint16_t *x = (is_v ? a.V : a.K) + src * ld + head * D;
    const int64_t unit = (int64_t)id * a.kv_heads + head;
    uint8_t *codes = (is_v ? a.cv : a.ck) + unit * ((int64_t)bs * D);
    float *scale = (is_v ? a.sv : a.sk) + unit;

    const int np = n * PR;
    u32x4 keep[AP_KEEP];
    float top = 0.0f;
    const auto piece = [&](int p) { return *(const u32x4 *)(x + (int64_t)(p / PR) * ld + (p % PR) * 8); };
    const auto widen = [&](u32x4 w) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = max_nan(top, max_nan(fabsf(lo_bf16(w[i])), fabsf(hi_bf16(w[i]))));
    };
#pragma unroll
    for (int c = 0; c < AP_KEEP; ++c) {
        const int p = t + AP_THREADS * c;
        keep[c] = p < np ? piece(p) : u32x4{0, 0, 0, 0};
    }
    const int old = lo - first;            // older tokens of the block
    const float was = old > 0 ? *scale : 0.0f;
#pragma unroll
    for (int c = 0; c < AP_KEEP; ++c)
        widen(keep[c]);
    for (int p = t + AP_THREADS * AP_KEEP; p < np; p += AP_THREADS)
        widen(piece(p));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        top = max_nan(top, __shfl_xor(top, off));
    if ((t & 63) == 0)
        wtop[t >> 6] = top;
    __syncthreads();                        // also: every thread has read the scale
#pragma unroll
    for (int w = 0; w < AP_THREADS / 64; ++w)
        top = max_nan(top, wtop[w]);
    float now = max_nan(was, top * (FMT == KV8_E4M3 ? 1.0f / 448.0f : 1.0f / 127.0f));
    if (!(now < __builtin_inff()))
        now = __builtin_nanf("");
    const bool grown = old > 0 && now > was;
    const Divider<FMT == KV8_E4M3> div(now);
    if (t == 0)
        *scale = now;

    if (!is_v) {
        u32x2 *dst = (u32x2 *)codes;
        const int at = old * PR;
#pragma unroll
        for (int c = 0; c < AP_KEEP; ++c) {
            const int p = t + AP_THREADS * c;
            if (p < np)
                dst[at + p] = enc_piece<FMT>(keep[c], div);
        }
        for (int p = t + AP_THREADS * AP_KEEP; p < np; p += AP_THREADS)
            dst[at + p] = enc_piece<FMT>(piece(p), div);
        if (grown)
            for (int p = t; p < at; p += AP_THREADS) {
                const u32x2 w = dst[p];
                dst[p] = u32x2{requantise<FMT>(w[0], was, div), requantise<FMT>(w[1], was, div)};
            }
        return;
    }

    // V: the new rows' codes to LDS, then columns of tokens out
    const auto put = [&](int p, u32x4 w) {
        const u32x2 c = enc_piece<FMT>(w, div);
        unsigned *row = stage + (old + p / PR) * PITCH + (p % PR) * 2;
        row[0] = c[0];
        row[1] = c[1];
    };
#pragma unroll
    for (int c = 0; c < AP_KEEP; ++c) {
        const int p = t + AP_THREADS * c;
        if (p < np)
            put(p, keep[c]);
    }
    for (int p = t + AP_THREADS * AP_KEEP; p < np; p += AP_THREADS)
        put(p, piece(p));
    __syncthreads();
    // a few tokens whose block keeps its scale: byte stores, which wait for
    // nothing, where reading the 16 bytes around them costs a trip to memory
    if (!grown && n < 4) {
        for (int i = t; i < n * D; i += AP_THREADS) {
            const int tok = old + i / D, d = i % D;
            codes[(int64_t)d * bs + tok] = ((const uint8_t *)(stage + tok * PITCH))[d];
        }
        return;
    }
    // item: four channels of 16 tokens; the tokens of a row of the block on
    // neighbouring lanes
    const int groups = bs / 16, lo_b = old, hi_b = old + n;
    for (int item = t; item < (D / 4) * groups; item += AP_THREADS) {
        const int dq = item / groups, t0 = (item % groups) * 16;
        if (t0 >= hi_b || (!grown && t0 + 16 <= lo_b))
            continue;
        u32x4 col[4];   // [channel] of four dwords of four tokens
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned *row = stage + (t0 + 4 * k) * PITCH + dq;
            const u32x4 c = transpose4(row[0], row[PITCH], row[2 * PITCH], row[3 * PITCH]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                col[i][k] = c[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4 *dst = (u32x4 *)(codes + (int64_t)(4 * dq + i) * bs + t0);
            if (t0 >= lo_b && t0 + 16 <= hi_b) {
                *dst = col[i];
                continue;
            }
            u32x4 w = *dst;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const unsigned fresh = byte_mask(t0 + 4 * k, lo_b, hi_b), older = byte_mask(t0 + 4 * k, 0, lo_b);
                unsigned v = (w[k] & ~fresh) | (col[i][k] & fresh);
                if (grown && older)
                    v = (v & ~older) | (requantise<FMT>(w[k], was, div) & older);
                w[k] = v;
            }
            *dst = w;
        }
    }
}

template <int D>
hipError_t launch_fmt(const Kv8Append &a, dim3 grid, hipStream_t s)
{
    const size_t lds = (size_t)a.bs * (D / 4 + 1) * 4;
    if (a.fmt == KV8_E4M3)
        hipLaunchKernelGGL((kv8_append_kernel<D, KV8_E4M3>), grid, dim3(AP_THREADS), lds, s, a);
    else
        hipLaunchKernelGGL((kv8_append_kernel<D, KV8_I8>), grid, dim3(AP_THREADS), lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv8_append(const Kv8Append &all, hipStream_t s)
{
    // q tokens touch at most (q + bs - 2) / bs + 1 blocks, whatever they start at;
    // a launch holds fewer than 2^32 threads along an axis: more go in several
    constexpr int64_t BLOCKS = 1 << 23;
    const int64_t n = ((int64_t)all.max_q + all.bs - 2) / all.bs + 1;
    hipError_t e = hipSuccess;
    for (int64_t at = 0; at < n && e == hipSuccess; at += BLOCKS) {
        Kv8Append a = all;
        a.at = (int)at;
        const dim3 grid((unsigned)std::min(BLOCKS, n - at), (unsigned)a.kv_heads * 2, (unsigned)a.batch);
        switch (a.dim) {
        case 64: e = launch_fmt<64>(a, grid, s); break;
        case 128: e = launch_fmt<128>(a, grid, s); break;
        case 192: e = launch_fmt<192>(a, grid, s); break;
        default: e = launch_fmt<256>(a, grid, s); break;
        }
    }
    return e;
}

}  // namespace qgemm
