// kv8_tile.hip -- attention of many query rows (prompts) over the 8-bit cache.
//
// The mathematics of kv8_stream.hip, bound by the matrix cores and, as closely,
// by the exponentials: for 32 rows, 64 tokens and D = 128 a wave's products
// take 1024 cycles of its matrix core and the softmax about 900 of its vector
// unit.  Hence
//  * codes are turned into bf16 (K) and binary16 (V) once a workgroup, on their
//    way into LDS, a step of 64 tokens ahead of the products, in two buffers
//    with one barrier a step;
//  * 32x32x16 products, whose operands come out of LDS at half the bytes a
//    product of 16x16x32, tokens again along the rows of the first: token 16 h +
//    i of a 32-token tile stands in row 8 (i / 4) + 4 h + i % 4, so that lane
//    half h ends with 16 tokens in order, in one block of the cache, and its
//    results are the second product's operand as they are;
//  * two waves a SIMD, so that one's products run beside the other's softmax;
//  * the running maximum moves only when a weight would pass 2^15 (a binary16's
//    range): weights are 2^(x - reference + 7) with the reference up to 2^8 out
//    of date, and most steps neither fade the sums nor touch the accumulators.
// On one MI355X: a chunk of 4096 tokens over 8192, 32 heads over 8 of 128, e4m3,
// 454 to 480 us, 860 to 910 TFLOP/s (a bf16 library product of 8192^3: 1323; 512 us
// with the block numbers loaded together with the codes, which waited for them).
// Counters there: matrix cores busy 36% of the cycles, vector instructions (262 a
// wave and step besides the 32 products; the softmax is about 225 of them) 41%, two
// waves a SIMD, LDS 28%.  So the two overlap little: the barrier a step keeps both
// waves of a SIMD in the same phase, and they wait for 44% of their time.  Five
// prompts of up to 1777 tokens, 16 heads of 64, int8, window 1024, 69 us, 340
// TFLOP/s: matrix cores 13%, vector instructions 40% (365 a wave and step, for
// half the products), 1.8 of three waves a SIMD there, waiting 45% of their
// time (928 workgroups on 768 places, a barrier a step).  192 and 256 channels,
// whose accumulators leave one wave a SIMD, 375 and 354 TFLOP/s.
// The rows of a kv head (its tokens times the heads that share it) are cut into
// tiles of 32 a wave; a split of the keys, where there are few tiles, leaves
// sums for kv8_join_kernel.
#include <hip/hip_runtime.h>

#include "kv8_dev.hpp"

namespace qgemm {

namespace {

constexpr int STEP = 64;
constexpr float NEG_INF = -__builtin_inff();
constexpr float TOP = 7.0f, LIMIT = 15.0f;   // log2 of a fresh maximum's weight and of the largest allowed

// max / sum over the two lane halves
__device__ __forceinline__ float half_max(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16-byte chunk c of a row in LDS: moved so that the rows that lanes 0..15 read
// together (tokens 0-3, 16-19, 4-7, 20-23 of K; channels 0-15 of V) fall into
// different banks.
template <int CHUNKS>
__device__ __forceinline__ int k_chunk(int row, int c)
{
    if constexpr (CHUNKS % 16 == 0)
        return row * CHUNKS + (c ^ ((row & 3) | ((row >> 2) & 4) | ((row << 1) & 8)));
    else
        return row * CHUNKS + (c ^ (((row >> 1) & 1) | ((row >> 3) & 2) | (row & 4)));
}
__device__ __forceinline__ int v_chunk(int row, int c) { return row * 8 + (c ^ ((row >> 1) & 7)); }

// Waves a SIMD that the registers are held to.
constexpr int tile_occupancy(int dc, int) { return dc == 1 ? 3 : dc == 2 ? 2 : 1; }

template <int DC, int WAVES, int FMT>
__global__ void __launch_bounds__(WAVES * 64, tile_occupancy(DC, WAVES)) kv8_tile_kernel(Kv8Attn a)
{
    constexpr int D = DC * 64, DT = D / 32, KS = D / 16, CH = D / 8;
    constexpr int THREADS = WAVES * 64, PIECES = STEP * D / 16;        // of 16 codes, of K and of V, a step
    constexpr int NP = (PIECES + THREADS - 1) / THREADS;               // that a thread stages
    static_assert(PIECES % THREADS == 0 || PIECES < THREADS, "pieces of a step");
    __shared__ u32x4 lk[2][STEP * CH], lv[2][D * 8];
    __shared__ float ls[2][4][4];   // of 16 tokens: score scale, log2 and reciprocal of the V scale, V scale > 0
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, h = lane >> 5;
    const int head = blockIdx.x, b = blockIdx.z;
    const int split = blockIdx.y % a.splits, tile = a.row_tiles - 1 - blockIdx.y / a.splits;   // longest first
    const int c0 = a.cu[b], q = a.cu[b + 1] - c0;
    const int rows = min(q, a.max_q) * a.group, row0 = tile * (32 * WAVES);
    if (q <= 0 || row0 >= rows || c0 < 0 || (int64_t)c0 + q > a.tokens)
        return;
    const int len = max(min(a.lens[b], (int)min((int64_t)a.width * a.bs, (int64_t)min(a.max_kv, 0x7fff0000))), 0);
    const int n_pos = a.lens[b];   // positions go by the sequence's own length

    // what the workgroup's rows see, and this wave's
    const auto see = [&](int r) { return span_of(min(r, rows - 1) / a.group, q, n_pos, a.causal, a.window); };
    const int lo_all = see(row0).lo, hi_all = min(see(row0 + 32 * WAVES - 1).hi, len);
    const int wrow = row0 + 32 * wave;
    const Span w_first = see(wrow), w_last = see(wrow + 31);
    const int w_lo = w_first.lo, w_hi = wrow < rows ? min(w_last.hi, len) : 0;   // any row of the wave sees
    const int in_lo = w_last.lo, in_hi = min(w_first.hi, len);                   // every row sees
    const int row = min(wrow + n, rows - 1);
    Span span = see(row);
    span.hi = min(span.hi, len);

    bf16x8 qf[KS];
    {
        const uint16_t *p = a.Q + (int64_t)(c0 + row / a.group) * a.ldq + (head * a.group + row % a.group) * D + 8 * h;
#pragma unroll
        for (int k = 0; k < KS; ++k)
            qf[k] = *(const bf16x8 *)(p + 16 * k);
    }

    const int step_lo = lo_all / STEP, step_hi = (hi_all + STEP - 1) / STEP;
    const int s0 = step_lo + split * a.split_steps, s1 = min(s0 + a.split_steps, step_hi);
    const int bshift = __builtin_ctz(a.bs);
    const int32_t *table = a.table + b * a.ldt;
    const int64_t unit_bytes = (int64_t)a.bs * D;

    // ---- staging: this thread's pieces of a step (16 codes each): K piece i is
    // piece i * THREADS + t of [token][D / 16], V piece i of [channel][token / 16]
    u32x4 rk[NP], rv[NP];
    float r_sk = 0.0f, r_sv = 0.0f, held = 1.0f;
    const auto block_at = [&](int tok) {
        int id = -1;
        if (tok < hi_all && tok + 16 > lo_all)
            id = table[tok >> bshift];
        return (unsigned)id < (unsigned)a.blocks ? id : -1;
    };
    // the blocks of the step to come, a step before its codes: a table entry's
    // trip from memory is not waited for
    int kid[NP], vid = -1, vid_now = -1;   // V: the thread's pieces share their 16 tokens
    const auto blocks = [&](int s) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            kid[i] = block_at((s * STEP + (i * THREADS + (int)threadIdx.x) % PIECES / (D / 16)) & ~15);
        vid = block_at(s * STEP + ((int)threadIdx.x & 3) * 16);
    };
    const auto fetch = [&](int s) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = (i * THREADS + threadIdx.x) % PIECES;
            const int tok = s * STEP + p / (D / 16), d = p % (D / 16) * 16;
            rk[i] = *(const u32x4 *)(a.ck + ((int64_t)max(kid[i], 0) * a.kv_heads + head) * unit_bytes +
                                     (int64_t)(tok & (a.bs - 1)) * D + d);
        }
        vid_now = vid;
        const int64_t u = (int64_t)max(vid, 0) * a.kv_heads + head;
        const int vtok = s * STEP + ((int)threadIdx.x & 3) * 16;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int d = (i * THREADS + (int)threadIdx.x) % PIECES >> 2;
            rv[i] = *(const u32x4 *)(a.cv + u * unit_bytes + (int64_t)d * a.bs + (vtok & (a.bs - 1)));
        }
        r_sk = a.sk[u];
        r_sv = a.sv[u];
    };
    const auto put = [&](int s, int buf) {
        if (PIECES < THREADS && threadIdx.x >= PIECES)
            return;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = i * THREADS + threadIdx.x;
            const int tok = p / (D / 16), c = p % (D / 16) * 2;
            const u32x2 w0 = codes4_bf16<FMT>(rk[i][0]), w1 = codes4_bf16<FMT>(rk[i][1]);
            const u32x2 w2 = codes4_bf16<FMT>(rk[i][2]), w3 = codes4_bf16<FMT>(rk[i][3]);
            lk[buf][k_chunk<CH>(tok, c)] = u32x4{w0[0], w0[1], w1[0], w1[1]};
            lk[buf][k_chunk<CH>(tok, c + 1)] = u32x4{w2[0], w2[1], w3[0], w3[1]};
        }
        // (a scale of a block that is not there may be anything)
        r_sk = vid_now >= 0 ? score_scale(r_sk, r_sv, a.scale2) : 0.0f;
        r_sv = vid_now >= 0 ? r_sv : 0.0f;
        // V codes that no row sees (0 * NaN), or whose scale is zero, are cleared
        const int vtok = s * STEP + (threadIdx.x & 3) * 16;   // the same for every piece of the thread
        if (!(r_sv > 0.0f) || vtok < lo_all || vtok + 16 > hi_all) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unsigned keep = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r_sv > 0.0f && vtok + 4 * k + e >= lo_all && vtok + 4 * k + e < hi_all)
                        keep |= 0xffu << (8 * e);
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    rv[i][k] &= keep;
            }
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = i * THREADS + threadIdx.x;
            const int d = p >> 2, c = (p & 3) * 2;
            const u32x2 w0 = codes4_f16<FMT>(rv[i][0]), w1 = codes4_f16<FMT>(rv[i][1]);
            const u32x2 w2 = codes4_f16<FMT>(rv[i][2]), w3 = codes4_f16<FMT>(rv[i][3]);
            lv[buf][v_chunk(d, c)] = u32x4{w0[0], w0[1], w1[0], w1[1]};
            lv[buf][v_chunk(d, c + 1)] = u32x4{w2[0], w2[1], w3[0], w3[1]};
        }
        const VScale v = v_scale(r_sv, held);
        if (threadIdx.x < 4) {
            ls[buf][threadIdx.x][0] = r_sk;
            ls[buf][threadIdx.x][1] = v.log2;
            ls[buf][threadIdx.x][2] = v.inv;
            ls[buf][threadIdx.x][3] = vid_now >= 0 ? 1.0f : 0.0f;
        }
    };

    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[d][i] = 0.0f;
    float l = 0.0f, zero = 0.0f;   // sum of weights; the exponent of weight 1
    bool seen = false;             // the row has seen a key: zero is its reference

    if (s0 < s1) {
        blocks(s0);
        fetch(s0);
        blocks(s0 + 1);
        put(s0, 0);
    }
    __syncthreads();
    const int krow = ((n >> 2) & 1) * 16 + (n >> 3) * 4 + (n & 3);   // the token in product row n
    for (int s = s0; s < s1; ++s) {
        const int buf = (s - s0) & 1, base = s * STEP;
        if (s + 1 < s1) {
            fetch(s + 1);
            blocks(s + 2);
        }
        if (base < w_hi && base + STEP > w_lo) {
            f32x16 sc[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sc[t][i] = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const bf16x8 kf = __builtin_bit_cast(bf16x8, lk[buf][k_chunk<CH>(32 * t + krow, 2 * k + h)]);
                    sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[k], sc[t], 0, 0, 0);
                }
            }
            float y[32], inv[2];
            bool there = true;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f32x4 sm = *(const f32x4 *)ls[buf][2 * t + h];
                const float c = sm[1] - zero;
                inv[t] = sm[2];
                there = there && sm[3] > 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    y[16 * t + i] = fmaf(sc[t][i], sm[0], c);
            }
            if (!(base >= in_lo && base + STEP <= in_hi && __all(there))) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const bool live = ls[buf][2 * t + h][3] > 0.0f;
                    const int tok = base + 32 * t + 16 * h;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!live || tok + i < span.lo || tok + i >= span.hi)
                            y[16 * t + i] = NEG_INF;
                }
            }
            float top = y[0];
#pragma unroll
            for (int i = 1; i < 32; ++i)
                top = fmaxf(top, y[i]);
            top = half_max(top);
            const bool move = seen ? top > LIMIT : top > NEG_INF;
            if (__any(move)) {
                const float by = move ? top - TOP : 0.0f;
                const float fade = seen ? __builtin_amdgcn_exp2f(-by) : 1.0f;
                seen = seen || move;
                zero += by;
                l *= fade;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    y[i] -= by;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[d][i] *= fade;
            }
            f16x8 pf[4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    y[16 * t + i] = __builtin_amdgcn_exp2f(y[16 * t + i]);
                    sum += y[16 * t + i];
                }
                l = fmaf(sum * SUM_UNIT, inv[t], l);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    u32x4 w;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = pack_f16(y[16 * t + 8 * u + 2 * i], y[16 * t + 8 * u + 2 * i + 1]);
                    pf[2 * t + u] = __builtin_bit_cast(f16x8, w);
                }
            }
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int tu = 0; tu < 4; ++tu) {
                    const f16x8 vf = __builtin_bit_cast(f16x8, lv[buf][v_chunk(32 * d + n, 4 * (tu >> 1) + 2 * h + (tu & 1))]);
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[tu], o[d], 0, 0, 0);
                }
        }
        if (s + 1 < s1)
            put(s + 1, buf ^ 1);
        __syncthreads();
    }

    l = half_sum(l);
    if (wrow + n >= rows)
        return;
    const int64_t tok = c0 + row / a.group;
    const int hq = head * a.group + row % a.group;
    if (a.splits == 1) {
        const RowSum f = row_sum(l);
        const float inv = 1.0f / f.sum;
        uint16_t *out = a.O + tok * a.ldo + hq * D + 4 * h;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[d][i] = o[d][i] * f.pre * inv;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(u32x2 *)(out + 32 * d + 8 * i) =
                    u32x2{pack_bf16(o[d][4 * i], o[d][4 * i + 1]), pack_bf16(o[d][4 * i + 2], o[d][4 * i + 3])};
        }
    } else {
        const int64_t at = (tok * a.kv_heads * a.group + hq) * a.splits + split;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(f32x4 *)(a.part + at * D + 32 * d + 8 * i + 4 * h) =
                    f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        if (h == 0) {
            a.stat[2 * at] = seen ? zero : NEG_INF;
            a.stat[2 * at + 1] = l;
        }
    }
}

template <int DC, int WAVES>
hipError_t launch_waves(const Kv8Attn &a, hipStream_t s)
{
    const dim3 grid((unsigned)a.kv_heads, (unsigned)(a.row_tiles * a.splits), (unsigned)a.batch);
    if (a.fmt == KV8_E4M3)
        hipLaunchKernelGGL((kv8_tile_kernel<DC, WAVES, KV8_E4M3>), grid, dim3(WAVES * 64), 0, s, a);
    else
        hipLaunchKernelGGL((kv8_tile_kernel<DC, WAVES, KV8_I8>), grid, dim3(WAVES * 64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

int kv8_tile_occupancy(int dc, int waves)
{
    // eight waves, a step's codes shared by 256 rows: D = 128 (4096 tokens over
    // 8192 480 us against 494 with four; four of up to 1000 over 1500 95 against
    // 90; 512 over 2048 and 6 of up to 300 alike).  D = 64 four (five prompts of up
    // to 1777 tokens 72 against 102 with eight, four of up to 1000 55 against 70,
    // 4096 over 8192 alike), of which three workgroups are resident
    return waves == 4 || (waves == 8 && dc == 2) ? tile_occupancy(dc, waves) : 0;
}

hipError_t launch_kv8_tile(const Kv8Attn &a, hipStream_t s)
{
    switch (a.dim) {
    case 64: return launch_waves<1, 4>(a, s);
    case 128: return a.waves == 8 ? launch_waves<2, 8>(a, s) : launch_waves<2, 4>(a, s);
    case 192: return launch_waves<3, 4>(a, s);
    default: return launch_waves<4, 4>(a, s);
    }
}

}  // namespace qgemm
