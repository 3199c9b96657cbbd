// kv8_stream.hip -- attention of few query rows over the 8-bit cache: single
// tokens, and a few at a time.
//
//   x[j,r] = log2(e) scale sk[blk(j)] sum_d kc[j,d] q[r,d] + log2 sv[blk(j)]   over the visible j
//   w = 2^(x - max_j x)
//   o[r,:] = sum_j w vc[j,:] / sum_j (w / sv[blk(j)])          0 where nothing is visible
//
// which is the softmax with the V scale drawn into the exponent: w is the
// probability times its scale, so that the second product takes the bare codes
// and the largest weight is 1 whatever the scales are.  That lets w be
// binary16 (times 2^15: what is below 2^-29 of the largest is subnormal), whose
// rounding, 2^-11, disappears in that of the bf16 result; bf16 weights doubled
// the error of the result where few keys hold the weight.
//
// The rows of a kv head are its new tokens times the query heads that share
// it, in tiles of 16 (NT tiles a wave).  Each wave runs alone over steps of 64
// tokens with its own running maximum and sum (binary32); the waves of a
// workgroup, and the splits of a long cache, are joined at the end.
//
// Bound by memory: 2 D bytes a cached token and kv head.  Codes go from memory
// to matrix-core operands with no LDS and no transposition:
//  * S is formed transposed, tokens along the rows of the product (operand A =
//    K) and query rows along its columns, so that a lane's results belong to
//    one query row (lane % 16) and the softmax's maximum and sum need two
//    exchanges between lanes.
//  * Which token stands in which row of the four 16-token products is free:
//    row 4 g + i of product j is token 16 g + 4 j + i of the step.  Lane group
//    g = lane / 16 then holds the probabilities of tokens 16 g .. 16 g + 15, in
//    order, which is the operand layout (8 sum elements a lane) of the second
//    product O^T = V^T P^T, and its V operand is one 16-byte load of 16
//    tokens of a channel.  No value changes lanes.
//  * 16 tokens never cross a block (bs >= 16), so that a lane group's scales
//    are one pair a step.
// Q and the codes of K enter the first product as bf16, the codes of V the
// second as binary16, all exactly; the sums are binary32.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv8_dev.hpp"

namespace qgemm {

namespace {

constexpr int STEP = 64;
constexpr float NEG_INF = -__builtin_inff();

__device__ __forceinline__ float xor16(float v) { return __shfl_xor(v, 16); }
__device__ __forceinline__ float xor32(float v) { return __shfl_xor(v, 32); }

template <int DC, int NT, int WAVES, int FMT>
__global__ void __launch_bounds__(WAVES * 64) kv8_stream_kernel(Kv8Attn a)
{
    constexpr int D = DC * 64, DT = D / 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n16 = lane & 15, g = lane >> 4;
    const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
    const int head = blockIdx.y, b = blockIdx.z;
    const int c0 = a.cu[b], q = a.cu[b + 1] - c0;
    const int rows = q * a.group, row0 = tile * (16 * NT);
    if (q <= 0 || row0 >= rows || c0 < 0 || (int64_t)c0 + q > a.tokens)
        return;
    const int len = max(min(a.lens[b], (int)min((int64_t)a.width * a.bs, (int64_t)0x7fffffc0)), 0);
    const int qlen_pos = a.lens[b];   // positions go by the sequence's own length

    // the tile's rows and what they see
    Span span[NT];
    const int t_first = row0 / a.group, t_last = min(row0 + 16 * NT - 1, rows - 1) / a.group;
    const Span s_first = span_of(t_first, q, qlen_pos, a.causal, a.window);
    const Span s_last = span_of(t_last, q, qlen_pos, a.causal, a.window);
    const int lo_all = s_first.lo, hi_all = min(s_last.hi, len);   // any row sees
    const int lo_in = s_last.lo, hi_in = min(s_first.hi, len);     // every row sees
    bf16x8 qf[NT][2 * DC];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = min(row0 + 16 * t + n16, rows - 1);
        span[t] = span_of(r / a.group, q, qlen_pos, a.causal, a.window);
        span[t].hi = min(span[t].hi, len);
        const uint16_t *p = a.Q + (int64_t)(c0 + r / a.group) * a.ldq + (head * a.group + r % a.group) * D + 16 * g;
#pragma unroll
        for (int c = 0; c < DC; ++c) {
            qf[t][2 * c] = *(const bf16x8 *)(p + 64 * c);
            qf[t][2 * c + 1] = *(const bf16x8 *)(p + 64 * c + 8);
        }
    }

    const int step_lo = lo_all / STEP, step_hi = (hi_all + STEP - 1) / STEP;
    const int s0 = step_lo + split * a.split_steps, s1 = min(s0 + a.split_steps, step_hi);
    const int bshift = __builtin_ctz(a.bs);
    const int32_t *table = a.table + b * a.ldt;
    const int64_t unit_bytes = (int64_t)a.bs * D;

    f32x4 o[NT][DT];
    float m[NT], l[NT], held = 1.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t] = NEG_INF;
        l[t] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
            o[t][d] = f32x4{0, 0, 0, 0};
    }

    // this lane's K rows of a step: tokens 16 kg + 4 j + (lane & 3)
    const int kg = n16 >> 2;
    for (int s = s0 + wave; s < s1; s += WAVES) {
        const int base = s * STEP;
        // the block of a 16-token group, or -1 where no row sees it
        const auto block_at = [&](int tok) {
            int id = -1;
            if (tok < hi_all && tok + 16 > lo_all)
                id = table[tok >> bshift];
            return (unsigned)id < (unsigned)a.blocks ? id : -1;
        };
        const int ktok = base + 16 * kg, vtok = base + 16 * g;
        const int kid = block_at(ktok), vid = block_at(vtok);
        const int64_t kunit = (int64_t)max(kid, 0) * a.kv_heads + head, vunit = (int64_t)max(vid, 0) * a.kv_heads + head;
        const uint8_t *kp = a.ck + kunit * unit_bytes + (int64_t)((ktok & (a.bs - 1)) + (lane & 3)) * D + 16 * g;
        const uint8_t *vp = a.cv + vunit * unit_bytes + (int64_t)n16 * a.bs + (vtok & (a.bs - 1));
        u32x4 kw[4][DC], vw[DT];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < DC; ++c)
                kw[j][c] = *(const u32x4 *)(kp + 4 * j * D + 64 * c);
#pragma unroll
        for (int d = 0; d < DT; ++d)
            vw[d] = *(const u32x4 *)(vp + (int64_t)(16 * d) * a.bs);
        const float sk = vid >= 0 ? a.sk[vunit] * a.scale2 : 0.0f;
        const float raw = vid >= 0 ? a.sv[vunit] : 0.0f;
        const VScale sv = v_scale(raw, held);

        f32x4 sc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sc[t][j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < DC; ++c) {
                const bf16x8 k0 = codes8_bf16<FMT>(kw[j][c][0], kw[j][c][1]);
                const bf16x8 k1 = codes8_bf16<FMT>(kw[j][c][2], kw[j][c][3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    sc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[t][2 * c], sc[t][j], 0, 0, 0);
                    sc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[t][2 * c + 1], sc[t][j], 0, 0, 0);
                }
            }

        // a step that every row sees whole needs no mask; elsewhere the codes
        // of V that no row sees (0 * NaN), or whose scale is zero, are cleared
        const bool whole = base >= lo_in && base + STEP <= hi_in && __all(raw > 0.0f);
        if (!whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unsigned keep = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = vtok + 4 * k + i;
                    if (raw > 0.0f && tok >= lo_all && tok < hi_all)
                        keep |= 0xffu << (8 * i);
                }
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    vw[d][k] &= keep;
            }
        }
        f16x8 pf[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float x[16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[4 * j + i] = fmaf(sc[t][j][i], sk, sv.log2);
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (vid < 0 || vtok + i < span[t].lo || vtok + i >= span[t].hi)
                        x[i] = NEG_INF;
            }
            float top = x[0];
#pragma unroll
            for (int i = 1; i < 16; ++i)
                top = fmaxf(top, x[i]);
            top = fmaxf(top, xor16(top));
            top = fmaxf(top, xor32(top));
            const float now = fmaxf(m[t], top);
            const float ref = now == NEG_INF ? 0.0f : now;
            const float fade = __builtin_amdgcn_exp2f(m[t] - ref), zero = ref - W_TOP;
            m[t] = now;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = __builtin_amdgcn_exp2f(x[i] - zero);
                sum += x[i];
            }
            l[t] = fmaf(l[t], fade, sum * sv.inv);
            if (!__all(fade == 1.0f)) {
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[t][d][i] *= fade;
            }
            u32x4 w[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[u][i] = pack_f16(x[8 * u + 2 * i], x[8 * u + 2 * i + 1]);
            pf[t][0] = __builtin_bit_cast(f16x8, w[0]);
            pf[t][1] = __builtin_bit_cast(f16x8, w[1]);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const f16x8 v0 = codes8_f16<FMT>(vw[d][0], vw[d][1]), v1 = codes8_f16<FMT>(vw[d][2], vw[d][3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[t][0], o[t][d], 0, 0, 0);
                o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[t][1], o[t][d], 0, 0, 0);
            }
        }
    }

    // join the waves, a tile at a time: in LDS, [wave][row][D + 4], and the
    // (maximum, sum) pairs
    constexpr int PITCH = D + 4;
    __shared__ float ow[WAVES][16][PITCH];
    __shared__ float om[WAVES][16], ol[WAVES][16];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float sum = l[t];
        sum += xor16(sum);
        sum += xor32(sum);
        if (t)
            __syncthreads();
        if (g == 0) {
            om[wave][n16] = m[t];
            ol[wave][n16] = sum;
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *(f32x4 *)&ow[wave][n16][16 * d + 4 * g] = o[t][d];
        __syncthreads();
        for (int item = threadIdx.x; item < 16 * (D / 4); item += WAVES * 64) {
            const int r = item / (D / 4), d = item % (D / 4) * 4;
            const int row = row0 + 16 * t + r;
            if (row >= rows)
                continue;
            float top = om[0][r];
#pragma unroll
            for (int w = 1; w < WAVES; ++w)
                top = fmaxf(top, om[w][r]);
            const float ref = top == NEG_INF ? 0.0f : top;
            f32x4 acc = {0, 0, 0, 0};
            float all = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const float f = __builtin_amdgcn_exp2f(om[w][r] - ref);
                const f32x4 v = *(const f32x4 *)&ow[w][r][d];
                all = fmaf(ol[w][r], f, all);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] = fmaf(v[i], f, acc[i]);
            }
            const int64_t tok = c0 + row / a.group;
            const int hq = head * a.group + row % a.group;
            if (a.splits == 1) {
                const float inv = all > 0.0f ? 1.0f / all : 0.0f;
                *(u32x2 *)(a.O + tok * a.ldo + hq * D + d) =
                    u32x2{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
            } else {
                const int64_t at = (tok * a.kv_heads * a.group + hq) * a.splits + split;
                *(f32x4 *)(a.part + at * D + d) = acc;
                if (d == 0) {
                    a.stat[2 * at] = top;
                    a.stat[2 * at + 1] = all;
                }
            }
        }
    }
}

// The splits of one row joined: a wave a row.
template <int DC>
__global__ void __launch_bounds__(256) kv8_join_kernel(Kv8Attn a)
{
    constexpr int D = DC * 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int heads = a.kv_heads * a.group;
    const int b = blockIdx.z, hq = blockIdx.y * 4 + wave, t = blockIdx.x;
    const int c0 = a.cu[b], q = a.cu[b + 1] - c0;
    if (hq >= heads || t >= q || c0 < 0 || (int64_t)c0 + q > a.tokens)
        return;
    const int64_t row = (int64_t)(c0 + t) * heads + hq;
    const float *stat = a.stat + 2 * row * a.splits, *part = a.part + row * a.splits * D + lane * DC;
    float top = NEG_INF;
    for (int s = lane; s < a.splits; s += 64)
        top = fmaxf(top, stat[2 * s]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        top = fmaxf(top, __shfl_xor(top, off));
    const float ref = top == NEG_INF ? 0.0f : top;
    float all = 0.0f, acc[DC] = {};
    for (int s = 0; s < a.splits; ++s) {
        const float f = __builtin_amdgcn_exp2f(stat[2 * s] - ref);
        all = fmaf(stat[2 * s + 1], f, all);
#pragma unroll
        for (int i = 0; i < DC; ++i)
            acc[i] = fmaf(part[(int64_t)s * D + i], f, acc[i]);
    }
    const float inv = all > 0.0f ? 1.0f / all : 0.0f;
    uint16_t *o = a.O + (int64_t)(c0 + t) * a.ldo + hq * D + lane * DC;
#pragma unroll
    for (int i = 0; i < DC; ++i)
        o[i] = (uint16_t)pack_bf16(acc[i] * inv, 0.0f);
}

template <int DC, int NT>
hipError_t launch_nt(const Kv8Attn &a, hipStream_t s)
{
    const dim3 grid((unsigned)(a.row_tiles * a.splits), (unsigned)a.kv_heads, (unsigned)a.batch);
    if (a.fmt == KV8_E4M3)
        hipLaunchKernelGGL((kv8_stream_kernel<DC, NT, 4, KV8_E4M3>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((kv8_stream_kernel<DC, NT, 4, KV8_I8>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int DC>
hipError_t launch_dim(const Kv8Attn &a, hipStream_t s)
{
    hipError_t e = a.kernel == 1 ? launch_kv8_tile(a, s) : a.nt == 1 ? launch_nt<DC, 1>(a, s) : launch_nt<DC, 2>(a, s);
    if (e == hipSuccess && a.splits > 1) {
        const dim3 join((unsigned)a.max_q, (unsigned)((a.kv_heads * a.group + 3) / 4), (unsigned)a.batch);
        hipLaunchKernelGGL((kv8_join_kernel<DC>), join, dim3(256), 0, s, a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

int64_t kv8_plan(Kv8Attn &a)
{
    const int64_t rows = (int64_t)a.max_q * a.group;
    // steps that a row tile can cover; a window starts anywhere in its first one
    int64_t steps = ((int64_t)a.max_kv + STEP - 1) / STEP;
    if (a.causal && a.window > 0)
        steps = std::min(steps, ((int64_t)a.window + a.max_q + 2 * STEP - 2) / STEP);
    steps = std::max<int64_t>(steps, 1);
    int64_t want, per;
    if (rows > 32) {
        a.kernel = 1;
        a.waves = rows > 128 && a.dim <= 128 ? 8 : 4;
        a.row_tiles = (int)((rows + 32 * a.waves - 1) / (32 * a.waves));
        const int64_t units = (int64_t)a.row_tiles * a.kv_heads * a.batch;
        want = units >= 256 ? 1 : (256 + units - 1) / units;
        per = std::max<int64_t>((steps + want - 1) / want, 8);
    } else {
        a.kernel = 0;
        a.nt = rows > 16 ? 2 : 1;
        a.row_tiles = (int)((rows + 16 * a.nt - 1) / (16 * a.nt));
        const int64_t units = (int64_t)a.row_tiles * a.kv_heads * a.batch;
        want = (2048 + units - 1) / units;
        per = (steps + want - 1) / want;
        per = per < 4 ? 4 : (per + 3) / 4 * 4;
        if (steps <= 8)
            per = steps;
    }
    a.split_steps = (int)std::min(per, steps);
    a.splits = (int)((steps + per - 1) / per);
    if (a.splits == 1)
        return 0;
    return a.tokens * a.kv_heads * a.group * a.splits * (a.dim + 2) * 4;
}

hipError_t launch_kv8_attention(const Kv8Attn &a, hipStream_t s)
{
    switch (a.dim) {
    case 64: return launch_dim<1>(a, s);
    case 128: return launch_dim<2>(a, s);
    case 192: return launch_dim<3>(a, s);
    default: return launch_dim<4>(a, s);
    }
}

}  // namespace qgemm
