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
// On one MI355X: 64 sequences of up to 8192 tokens, 64 heads over 8 of 128, e4m3,
// 152 us, 5.3 TB/s (reading alone: 6.5); three of 65537, 64 heads over 4, int8,
// 44 us (vector units issuing for 14 of them, waves waiting for three quarters of
// their time, 1.4 of them a SIMD) and 4.8 for the joining; one of 1001 11 us, which is latency (a chain of
// lengths, block number, codes, and two turns of a wave).
// Q and the codes of K enter the first product as bf16, the codes of V the
// second as binary16, all exactly; the sums are binary32.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv8_dev.hpp"

namespace qgemm {

namespace {

constexpr int STEP = 64;
constexpr float NEG_INF = -__builtin_inff();

// max / sum over the four lane groups
__device__ __forceinline__ float groups_max(float v)
{
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float groups_sum(float v)
{
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Waves a SIMD that the registers are held to, and that the plan counts on (the
// 168 registers of D = 128 with one tile would let in a third one).
constexpr int stream_occupancy(int dc, int nt)
{
    return nt == 1 ? (dc == 1 ? 4 : dc <= 3 ? 2 : 1) : dc <= 2 ? 2 : 1;
}

template <int DC, int NT, int WAVES, int FMT>
__global__ void __launch_bounds__(WAVES * 64, stream_occupancy(DC, NT)) kv8_stream_kernel(Kv8Attn a)
{
    constexpr int D = DC * 64, DT = D / 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n16 = lane & 15, g = lane >> 4;
    const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
    const int head = blockIdx.y, b = blockIdx.z;
    const int c0 = a.cu[b], q = a.cu[b + 1] - c0;
    const int rows = min(q, a.max_q) * a.group, row0 = tile * (16 * NT);
    if (q <= 0 || row0 >= rows || c0 < 0 || (int64_t)c0 + q > a.tokens)
        return;
    const int len = max(min(a.lens[b], (int)min((int64_t)a.width * a.bs, (int64_t)min(a.max_kv, 0x7fff0000))), 0);
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

    // this lane's K rows of a step: tokens 16 kg + 4 j + (lane & 3); its V tokens
    // and scales: 16 g .. 16 g + 15.  K's registers take the next step as soon as
    // the first product is done, V's after the second: one or the other is always
    // under way.  Block numbers come a step earlier still.
    const int kg = n16 >> 2;
    const auto block_at = [&](int tok) {   // -1 where no row sees the 16 tokens from tok on
        int id = -1;
        if (tok < hi_all && tok + 16 > lo_all)
            id = table[tok >> bshift];
        return (unsigned)id < (unsigned)a.blocks ? id : -1;
    };
    u32x4 kw[4][DC], vw[DT];
    float sk = 0.0f, raw = 0.0f;
    const auto load_k = [&](int s, int id) {
        const int tok = s * STEP + 16 * kg;
        const int64_t unit = (int64_t)max(id, 0) * a.kv_heads + head;
        const uint8_t *p = a.ck + unit * unit_bytes + (int64_t)((tok & (a.bs - 1)) + (lane & 3)) * D + 16 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < DC; ++c)
                kw[j][c] = *(const u32x4 *)(p + 4 * j * D + 64 * c);
    };
    const auto load_v = [&](int s, int id) {
        const int tok = s * STEP + 16 * g;
        const int64_t unit = (int64_t)max(id, 0) * a.kv_heads + head;
        const uint8_t *p = a.cv + unit * unit_bytes + (int64_t)n16 * a.bs + (tok & (a.bs - 1));
        sk = a.sk[unit];
        raw = a.sv[unit];
#pragma unroll
        for (int d = 0; d < DT; ++d)
            vw[d] = *(const u32x4 *)(p + (int64_t)(16 * d) * a.bs);
    };
    int vid = -1, next_k = -1, next_v = -1;
    if (s0 + wave < s1) {
        const int s = s0 + wave;
        const int kid = block_at(s * STEP + 16 * kg);
        vid = block_at(s * STEP + 16 * g);
        load_k(s, kid);
        load_v(s, vid);
        next_k = block_at((s + WAVES) * STEP + 16 * kg);
        next_v = block_at((s + WAVES) * STEP + 16 * g);
    }
    for (int s = s0 + wave; s < s1; s += WAVES) {
        const int base = s * STEP, vtok = base + 16 * g;
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
        const bool more = s + WAVES < s1;
        if (more)
            load_k(s + WAVES, next_k);
        // (a scale of a block that is not there may be anything)
        const float k_scale = vid >= 0 ? score_scale(sk, raw, a.scale2) : 0.0f, v_raw = vid >= 0 ? raw : 0.0f;
        const VScale sv = v_scale(v_raw, held);

        // a step that every row sees whole needs no mask; elsewhere the codes
        // of V that no row sees (0 * NaN), or whose scale is zero, are cleared
        const bool whole = base >= lo_in && base + STEP <= hi_in && __all(v_raw > 0.0f);
        if (!whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unsigned keep = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = vtok + 4 * k + i;
                    if (v_raw > 0.0f && tok >= lo_all && tok < hi_all)
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
                    x[4 * j + i] = fmaf(sc[t][j][i], k_scale, sv.log2);
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
            top = groups_max(top);
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
            l[t] = fmaf(l[t], fade, sum * SUM_UNIT * sv.inv);
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
        if (more) {
            load_v(s + WAVES, next_v);
            vid = next_v;
            next_k = block_at((s + 2 * WAVES) * STEP + 16 * kg);
            next_v = block_at((s + 2 * WAVES) * STEP + 16 * g);
        }
    }

    // join the waves, a tile at a time: in LDS, [wave][row][D + 4], and the
    // (maximum, sum) pairs
    constexpr int PITCH = D + 4;
    __shared__ float ow[WAVES][16][PITCH];
    __shared__ float om[WAVES][16], ol[WAVES][16];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float sum = groups_sum(l[t]);
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
                const RowSum f = row_sum(all);
                const float inv = 1.0f / f.sum;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] = acc[i] * f.pre * inv;
                *(u32x2 *)(a.O + tok * a.ldo + hq * D + d) = u32x2{pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3])};
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

// The splits of one row joined: WPR waves a row, taking turns over the splits,
// in a fixed order.
template <int DC, int WPR>
__global__ void __launch_bounds__(256) kv8_join_kernel(Kv8Attn a)
{
    constexpr int D = DC * 64;
    [[maybe_unused]] __shared__ float part_o[WPR][D], part_l[WPR];
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wid % WPR;
    const int heads = a.kv_heads * a.group;
    const int b = blockIdx.z, hq = blockIdx.y * (4 / WPR) + wid / WPR, t = blockIdx.x;
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
#pragma unroll 4
    for (int s = wave; s < a.splits; s += WPR) {
        const float f = __builtin_amdgcn_exp2f(stat[2 * s] - ref);
        all = fmaf(stat[2 * s + 1], f, all);
#pragma unroll
        for (int i = 0; i < DC; ++i)
            acc[i] = fmaf(part[(int64_t)s * D + i], f, acc[i]);
    }
    uint16_t *out = a.O + (int64_t)(c0 + t) * a.ldo + hq * D;
    if constexpr (WPR == 1) {
        const RowSum f = row_sum(all);
        const float inv = 1.0f / f.sum;
#pragma unroll
        for (int i = 0; i < DC; ++i)
            out[lane * DC + i] = (uint16_t)pack_bf16(acc[i] * f.pre * inv, 0.0f);
        return;
    }
#pragma unroll
    for (int i = 0; i < DC; ++i)
        part_o[wave][lane * DC + i] = acc[i];
    if (lane == 0)
        part_l[wave] = all;
    __syncthreads();
    if (threadIdx.x < D) {
        const int d = threadIdx.x;
        float l = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            l += part_l[w];
            v += part_o[w][d];
        }
        const RowSum f = row_sum(l);
        out[d] = (uint16_t)pack_bf16(v * f.pre / f.sum, 0.0f);
    }
}

template <int DC, int NT, int WAVES>
hipError_t launch_waves(const Kv8Attn &a, hipStream_t s)
{
    const dim3 grid((unsigned)(a.row_tiles * a.splits), (unsigned)a.kv_heads, (unsigned)a.batch);
    if (a.fmt == KV8_E4M3)
        hipLaunchKernelGGL((kv8_stream_kernel<DC, NT, WAVES, KV8_E4M3>), grid, dim3(WAVES * 64), 0, s, a);
    else
        hipLaunchKernelGGL((kv8_stream_kernel<DC, NT, WAVES, KV8_I8>), grid, dim3(WAVES * 64), 0, s, a);
    return hipGetLastError();
}

template <int DC, int NT>
hipError_t launch_nt(const Kv8Attn &a, hipStream_t s)
{
    if constexpr (stream_occupancy(DC, NT) > 1)
        if (a.waves == 8)
            return launch_waves<DC, NT, 8>(a, s);
    return launch_waves<DC, NT, 4>(a, s);
}

template <int DC>
hipError_t launch_dim(const Kv8Attn &a, hipStream_t s)
{
    hipError_t e = a.kernel == 1 ? launch_kv8_tile(a, s) : a.nt == 1 ? launch_nt<DC, 1>(a, s) : launch_nt<DC, 2>(a, s);
    if (e == hipSuccess && a.splits > 1) {
        const unsigned heads = (unsigned)(a.kv_heads * a.group);
        if (a.splits > 4)
            hipLaunchKernelGGL((kv8_join_kernel<DC, 4>), dim3((unsigned)a.max_q, heads, (unsigned)a.batch), dim3(256), 0,
                               s, a);
        else
            hipLaunchKernelGGL((kv8_join_kernel<DC, 1>), dim3((unsigned)a.max_q, (heads + 3) / 4, (unsigned)a.batch),
                               dim3(256), 0, s, a);
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
    // Waves a workgroup and splits: the fewest turns of the loop over steps from
    // first to last, with the workgroups that are resident together as one round;
    // a workgroup's start and end count as `ends` turns, joining splits as `ends`
    // more.  (Single tokens: 64 x 8192 tokens, 512 units: no split 157 us, two
    // 169, four 184; 131072 tokens, 8 units: splits of 32 steps 58 us, of 16 60,
    // of 8 67.)
    a.kernel = rows > 32;
    a.nt = rows > 16 ? 2 : 1;
    const int dc = a.dim / 64, ends = a.kernel ? 4 : 1;
    int64_t best = -1, per = steps;
    for (int waves = 8; waves >= 4; waves -= 4) {
        const int per_cu = 4 * (a.kernel ? kv8_tile_occupancy(dc, waves) : stream_occupancy(dc, a.nt)) / waves;
        if (per_cu == 0)
            continue;
        const int tile_rows = a.kernel ? 32 * waves : 16 * a.nt;
        const int64_t tiles = (rows + tile_rows - 1) / tile_rows, units = tiles * a.kv_heads * a.batch;
        for (int64_t w = 1; w <= 64 && w <= steps; ++w) {
            if (a.kernel && w > 1 && units * w > 256 * per_cu)
                break;   // many rows: their sums cost more than an uneven last round
            const int64_t p = (steps + w - 1) / w, turns = a.kernel ? p : (p + waves - 1) / waves;
            const int64_t cost = (units * w + 256 * per_cu - 1) / (256 * per_cu) * (turns + ends) + (w > 1 ? ends : 0);
            if (best < 0 || cost < best) {
                best = cost;
                per = p;
                a.waves = waves;
                a.row_tiles = (int)tiles;
            }
        }
    }
    a.split_steps = (int)per;
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
