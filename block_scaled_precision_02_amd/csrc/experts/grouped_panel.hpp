// grouped_panel.hpp -- grouped products of a few tens of rows an expert: bound
// by streaming the experts' weights, as in grouped_stream.hpp, with enough rows
// that A has to be shared.
//
// A workgroup of four waves takes MB blocks of 16 rows by 128 columns; each
// wave has 32 of the columns (two 16x16 products wide) and all the rows.  B
// goes from memory straight into the registers of the one wave that uses it,
// three stages ahead: registers hold several times what LDS does, and what is
// in flight is what a stream needs.  A's rows, which all four waves use, are
// fetched into LDS four stages deep (qgemm_dma.hpp's fetch and pair layout).
// A stage is 128 bytes of every row; one barrier a stage.
//
//  * K map and steps are those of qgemm_skinny.hpp: lane group g (lane / 16)
//    takes byte chunk g of each 64-byte piece, and for e4m3 its 128-byte step
//    is the whole stage.  Sums run over the steps in their order.
//  * Scales of A (MX, blockscale): the bytes that a round of four stages takes
//    of each row are fetched into LDS a round ahead; of B: the same bytes into
//    the registers of the lanes that use them.
//  * Waits: loads return in order.  A wave waits for its share of stage t's
//    fetch by the count of loads it has issued since (see AFTER), then meets
//    the others at the barrier, after which stage t - 1's slot is free.
//  * Stages past K are zeros (descriptors' range), their scale words zero.
//
// One MI355X: 16 tokens, 8 of 128 experts of 4096x7168, e2m1, 64 to 77 of which
// have rows, 175 to 213 us, 5.4 to 5.7 TB/s of weights; 64 experts of 4096x7168
// with 16 rows each, INT8 321 us, 5.9 TB/s.  With 32 or 128 rows a panel: 2 to 4% and
// 5 to 15% slower.
#pragma once
#include "../qgemm_dma.hpp"
#include "../qgemm_skinny.hpp"

namespace qgemm {

constexpr int PANEL_BN = 128, PANEL_THREADS = 256;

template <int PATH, int MB, bool BIAS, int BROWS>
__global__ void __launch_bounds__(PANEL_THREADS, 2) qgemm_panel_kernel(const GroupedParams p)
{
    using T = SkinnyTraits<PATH>;
    using Acc = typename T::Acc;
    constexpr bool MX = PATH == PATH_MX8 || PATH == PATH_MX4;
    constexpr bool BS = PATH == PATH_F8B;
    constexpr bool INK = MX || BS;
    constexpr int NW = PANEL_THREADS / 64, BM = 16 * MB, NB = 2;
    constexpr int NST = 4;                                   // stages in LDS, and B's ring
    constexpr int STAGE = BM * 128;                          // bytes of A a stage
    constexpr int NA = BM / 8 / NW > 0 ? BM / 8 / NW : 1;    // A fetches a wave and stage (8 rows each)
    static_assert(BM % 32 == 0, "every wave fetches rows of A");
    constexpr int NBL = 2 * NB;                              // B loads a wave and stage
    constexpr int SCB = INK ? (PATH == PATH_MX4 ? 32 : 16) : 0;   // scale bytes of a row and round
    constexpr int NSA = INK ? 1 : 0;                         // A scale fetches a wave and round
    constexpr int NSB = MX ? NB * SCB / 16 : BS ? 1 : 0;     // B scale loads a wave and round
    constexpr int ROWS_PER_SF = 1024 / (SCB ? SCB : 16);     // rows that one scale fetch covers
    constexpr int NSF = (BM + ROWS_PER_SF - 1) / ROWS_PER_SF;   // scale fetches that cover the rows
    static_assert(NSF <= NW, "one scale fetch a wave");
    constexpr int SCL_OFF = NST * STAGE, SCL_BUF = NSF * 1024;
    constexpr int SA_OFF = SCL_OFF + (INK ? 2 * SCL_BUF : 0);
    __shared__ __attribute__((aligned(1024))) uint8_t lds[SA_OFF + (INK ? 0 : BM * 4)];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;

    GroupedTile tile;
    if (!grouped_tile<BM>(p, tile))
        return;
    const int n0 = tile.tn * PANEL_BN + 32 * wave;           // this wave's first column
    const int rows_b = min(32, p.N - n0);                    // below 1: none
    const int32_t *const order = p.order ? p.order + tile.row0 : nullptr;
    const int64_t base = order ? 0 : tile.row0;
    const int src_rows = order ? (int)p.a_rows : tile.rows;
    auto src = [&](int r) -> unsigned {
        if (r >= tile.rows)
            return ~0u;
        return order ? (unsigned)order[r] / (unsigned)p.top_k : (unsigned)r;
    };

    // B: rows n0 + 16 b + r16
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B + (int64_t)tile.expert * p.b_expert + (int64_t)n0 * p.ldb,
                                                rows_b > 0 ? (uint32_t)((rows_b - 1) * p.ldb + p.kbytes) : 0u);
    unsigned b_row[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        b_row[b] = 16 * b + r16 < rows_b ? (unsigned)((16 * b + r16) * p.ldb) + 16 * g : OOB;
    // A: fetch j of this wave covers rows 8 (NA wave + j) .. +7
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + base * p.lda, (uint32_t)((src_rows - 1) * p.lda + p.kbytes));
    unsigned a_row[NA];
    const int a_col = 16 * ((lane & 7) ^ (lane >> 4));       // the chunk's byte in the stage, in even groups of 8 rows
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        const int r = 8 * (NA * wave + j) + (lane >> 3);
        const unsigned s = src(r);
        // slot lane % 8 of row r holds chunk (lane & 7) ^ ((r >> 1) & 7): bit 2
        // flips in odd groups
        const int col = a_col ^ (((NA * wave + j) & 1) << 6);
        a_row[j] = s < (unsigned)src_rows ? (unsigned)(s * p.lda) + col : OOB;
    }
    // scales
    __amdgpu_buffer_rsrc_t rsa, rsb;
    unsigned sa_off = OOB, sb_off[NB] = {OOB, OOB};
    if constexpr (INK) {
        rsa = make_rsrc(p.mx_sa + base * p.kblocks, (uint32_t)(src_rows * p.kblocks));
        const int srows = (p.N + BROWS - 1) / BROWS;
        const int sb0 = n0 / BROWS, nsb = rows_b > 0 ? (n0 + rows_b - 1) / BROWS - sb0 + 1 : 0;
        rsb = make_rsrc(p.mx_sb + ((int64_t)tile.expert * srows + sb0) * p.kblocks, (uint32_t)(nsb * p.kblocks));
        constexpr int LPR = SCB / 16;                        // lanes a row
        const int r = ROWS_PER_SF * (wave % NSF) + lane / LPR;
        const unsigned s = r < BM ? src(r) : ~0u;
        sa_off = s < (unsigned)src_rows ? (unsigned)(s * p.kblocks) + 16 * (lane % LPR) : OOB;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            sb_off[b] = BS ? 0u : 16 * b + r16 < rows_b ? (unsigned)((16 * b + r16) * p.kblocks) : OOB;
    }
    // rows' own scales (int8, e4m3 a row)
    if constexpr (!INK) {
        if (tid < BM) {
            const unsigned s = src(tid);
            *(float *)&lds[SA_OFF + 4 * tid] = s < (unsigned)src_rows ? p.scale_a[base + s] : 0.0f;
        }
    }

    const int nst = (p.kbytes + 127) / 128;
    u32x4 fb[NST][NB][2];
    constexpr int UQ = MX ? SCB / 16 : 1;                    // 16-byte words of a B row's round
    u32x4 sb_nxt[INK ? NB : 1][UQ], sb_use[INK ? NB : 1][UQ];
    Acc acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            acc[i][b] = Acc{};

    auto fetch_a = [&](int t, auto slotc) {
        constexpr int SLOT = decltype(slotc)::value;
#pragma unroll
        for (int j = 0; j < NA; ++j) {
            // a chunk at or past K reads zeros (a row's last stage may be half)
            const int col = a_col ^ (((NA * wave + j) & 1) << 6);
            const unsigned o = 128 * t + col < p.kbytes ? a_row[j] + (unsigned)(128 * t) : OOB;
            dma16(ra, o, &lds[SLOT * STAGE + 1024 * (NA * wave + j)]);
        }
    };
    auto load_b = [&](int t, auto slotc) {
        constexpr int SLOT = decltype(slotc)::value;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int k = 128 * t + 64 * c;
                fb[SLOT][b][c] = ld16(rb, k + 16 * g < p.kbytes ? b_row[b] + (unsigned)k : OOB);
            }
    };
    // round u of the scales (stages 4u .. 4u+3)
    auto fetch_scales = [&](int u) {
        if constexpr (INK) {
            dma16(rsa, sa_off + (unsigned)(SCB * u), &lds[SCL_OFF + (u & 1) * SCL_BUF + 1024 * (wave % NSF)]);
#pragma unroll
            for (int b = 0; b < (BS ? 1 : NB); ++b)
#pragma unroll
                for (int w = 0; w < UQ; ++w)
                    sb_nxt[b][w] = ld16(rsb, sb_off[b] + (unsigned)(SCB * u + 16 * w));
        }
    };
    // (words past K/32 are the next row's: zero)
    auto use_scales = [&](int u) {
        if constexpr (INK) {
#pragma unroll
            for (int b = 0; b < (BS ? 1 : NB); ++b)
#pragma unroll
                for (int w = 0; w < UQ; ++w)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sb_use[b][w][j] = SCB * u + 16 * w + 4 * j < p.kblocks ? sb_nxt[b][w][j] : 0;
        }
    };

    auto multiply = [&](int t, auto slotc) {
        constexpr int J = decltype(slotc)::value;            // t % 4
        const uint8_t *ta = &lds[J * STAGE];
        const uint8_t *sc = &lds[SCL_OFF + ((t >> 2) & 1) * SCL_BUF];
        unsigned wb[NB][2] = {};
        float fsb = 0.0f;
        if constexpr (PATH == PATH_MX8) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                wb[b][0] = sb_use[b][0][J] >> (8 * g);
        } else if constexpr (PATH == PATH_MX4) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    wb[b][c] = sb_use[b][J >> 1][2 * (J & 1) + c] >> (8 * g);
        } else if constexpr (BS) {
            const unsigned w = sb_use[0][0][J];
            fsb = __builtin_bit_cast(float, w);
        }
        // scale words of A past K: zero (masked, not branched over: the compiler
        // would move the products of all four stages behind the last branch)
        const unsigned live = t < nst ? ~0u : 0u, live1 = 256 * t + 128 < p.K ? ~0u : 0u;
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int row = 16 * i + r16;
            const i32x4 a0 = *(const i32x4 *)(ta + plds_off(row, g));
            const i32x4 a1 = *(const i32x4 *)(ta + plds_off(row, 4 + g));
            if constexpr (PATH == PATH_I8) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    acc[i][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, fb[J][b][0]), a0,
                                                                      acc[i][b], 0, 0, 0);
                    acc[i][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, fb[J][b][1]), a1,
                                                                      acc[i][b], 0, 0, 0);
                }
            } else if constexpr (PATH == PATH_MX4) {
                const u32x2 v = *(const u32x2 *)(sc + 32 * row + 8 * J);
                const unsigned w0 = v[0], w1 = v[1];
                const unsigned s0 = (w0 & live) >> (8 * g), s1 = (w1 & live1) >> (8 * g);
                const i32x8 x0 = {a0[0], a0[1], a0[2], a0[3], 0, 0, 0, 0};
                const i32x8 x1 = {a1[0], a1[1], a1[2], a1[3], 0, 0, 0, 0};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const i32x4 y0 = __builtin_bit_cast(i32x4, fb[J][b][0]), y1 = __builtin_bit_cast(i32x4, fb[J][b][1]);
                    const i32x8 b0 = {y0[0], y0[1], y0[2], y0[3], 0, 0, 0, 0};
                    const i32x8 b1 = {y1[0], y1[1], y1[2], y1[3], 0, 0, 0, 0};
                    acc[i][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b0, x0, acc[i][b], 4, 4, 0,
                                                                                 (int)wb[b][0], 0, (int)s0);
                    acc[i][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b1, x1, acc[i][b], 4, 4, 0,
                                                                                 (int)wb[b][1], 0, (int)s1);
                }
            } else {
                const i32x8 x = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
                unsigned s = 0;
                if constexpr (INK) {
                    const unsigned w = *(const unsigned *)(sc + 16 * row + 4 * J);
                    s = (w & live) >> (MX ? 8 * g : 0);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const i32x4 y0 = __builtin_bit_cast(i32x4, fb[J][b][0]), y1 = __builtin_bit_cast(i32x4, fb[J][b][1]);
                    const i32x8 y = {y0[0], y0[1], y0[2], y0[3], y1[0], y1[1], y1[2], y1[3]};
                    if constexpr (MX) {
                        acc[i][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y, x, acc[i][b], 0, 0, 0,
                                                                                     (int)wb[b][0], 0, (int)s);
                    } else if constexpr (BS) {
                        const f32x4 part =
                            __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y, x, f32x4{}, 0, 0, 0, 0, 0, 0);
                        const float w = __builtin_bit_cast(float, s) * fsb;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[i][b][r] = __builtin_fmaf(part[r], w, acc[i][b][r]);
                    } else {
                        acc[i][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y, x, acc[i][b], 0, 0, 0, 0, 0, 0);
                    }
                }
            }
        }
    };

    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    // (issue order is what the waits count)
    fetch_scales(0);
    __builtin_amdgcn_sched_barrier(0);
    fetch_a(0, I0());
    __builtin_amdgcn_sched_barrier(0);
    load_b(0, I0());
    __builtin_amdgcn_sched_barrier(0);
    fetch_a(1, I1());
    __builtin_amdgcn_sched_barrier(0);
    load_b(1, I1());
    __builtin_amdgcn_sched_barrier(0);
    fetch_a(2, I2());
    __builtin_amdgcn_sched_barrier(0);
    load_b(2, I2());
    __builtin_amdgcn_sched_barrier(0);
    for (int t0 = 0; t0 < nst; t0 += NST) {
        static_for<0, NST>([&](auto jc) {
            constexpr int J = decltype(jc)::value;
            const int t = t0 + J;
            // Loads issued after stage t's fetch of A: its B, stages t+1 and
            // t+2, and the next round's scales where they went out since (at a
            // round's first stage, before its own fetches).
            constexpr int AFTER = NBL + 2 * (NA + NBL) + (J == 1 || J == 2 ? NSA + NSB : 0);
            twin_sync();
            wait_vmcnt<AFTER>();
            lds_barrier();
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (J == 0) {
                use_scales(t >> 2);
                fetch_scales((t >> 2) + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            fetch_a(t + 3, std::integral_constant<int, (J + 3) % NST>());
            __builtin_amdgcn_sched_barrier(0);
            load_b(t + 3, std::integral_constant<int, (J + 3) % NST>());
            __builtin_amdgcn_sched_barrier(0);
            multiply(t, jc);
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    wait_vmcnt<0>();   // nothing may still be landing in LDS when the workgroup ends

    // The epilogue of the main kernels: lane has row 16 i + r16, columns 4 g .. +3
    // of each of its 16.
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int nloc = 16 * b + 4 * g;
        unsigned sbw[4] = {0, 0, 0, 0}, bbw[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (nloc + r < rows_b) {
                const int64_t at = (int64_t)tile.expert * p.N + n0 + nloc + r;
                if constexpr (!INK)
                    sbw[r] = __builtin_bit_cast(unsigned, p.scale_b[at]);
                if constexpr (BIAS)
                    bbw[r] = (unsigned)p.bias[at] << 16;
            }
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int mloc = 16 * i + r16;
            if (mloc >= tile.rows)
                continue;
            float f[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x = (float)acc[i][b][r];
                if constexpr (!INK) {
                    x = x * *(const float *)&lds[SA_OFF + 4 * mloc];
                    x = x * __builtin_bit_cast(float, sbw[r]);
                }
                if constexpr (BIAS)
                    x = x + __builtin_bit_cast(float, bbw[r]);
                f[r] = x;
            }
            uint16_t *out = (uint16_t *)p.C + (int64_t)(tile.row0 + mloc) * p.ldc + n0 + nloc;
            const u32x2 v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
            if (nloc + 4 <= rows_b) {
                *(u32x2 *)out = v;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (nloc + r < rows_b)
                        out[r] = (uint16_t)(v[r >> 1] >> (16 * (r & 1)));
            }
        }
    }
}

}  // namespace qgemm
