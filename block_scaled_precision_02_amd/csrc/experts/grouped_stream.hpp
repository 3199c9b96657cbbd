// grouped_stream.hpp -- grouped products of few rows an expert: bound by
// streaming the weights of the experts that have any.
//
// A wave takes a tile of 16 rows (TM blocks of them) by 16 columns over the
// whole of K by itself: no LDS, no barrier, no wave waits for another.  Its
// fragments, B's and A's (a handful of rows, from L2), are loaded D steps ahead
// into a ring of registers, and the ring runs on from one tile into the wave's
// next, so that loads are in flight all the time.  The grid is what is resident
// at once; each wave walks an even share of the tiles.
//
// Fragment and scale maps, steps and the order of the sums are those of
// qgemm_skinny.hpp: there eight waves each sum every eighth step of K and the
// eight sums are added in their order; here one wave keeps the eight sums.  Its
// results are the same, bit for bit, so that either may be chosen.  (One MI355X: 3
// tokens, 8 of 64 experts of 2112x7168, e4m3 MX 67 us, 128x128 tiles 87; one token of
// 2048x7168, INT8 23 us, 39.)
#pragma once
#include "../qgemm_skinny.hpp"

namespace qgemm {

// A wave's place in the tiles: those of each expert in turn, all row tiles of
// one column tile next to one another (they read the same weights).
struct StreamTile {
    int expert, row0, rows, tn;
};

template <int PATH> struct StreamTraits;
// steps in flight: 8 KB of B a wave
template <> struct StreamTraits<PATH_I8> { static constexpr int D = 8, WAVES = 2; };
template <> struct StreamTraits<PATH_MX4> { static constexpr int D = 8, WAVES = 2; };
template <> struct StreamTraits<PATH_F8> { static constexpr int D = 4, WAVES = 2; };
template <> struct StreamTraits<PATH_MX8> { static constexpr int D = 4, WAVES = 2; };
template <> struct StreamTraits<PATH_F8B> { static constexpr int D = 4, WAVES = 2; };

constexpr int STREAM_THREADS = 256;

// The product that made v stays in front of the next branch: the compiler moved
// it behind, where it kept all its operands.
template <class V>
__device__ __forceinline__ void keep_here(V &v)
{
    asm volatile("" : "+v"(v));
}

template <int PATH, int TM, bool BIAS, int BROWS>
__global__ void __launch_bounds__(STREAM_THREADS, StreamTraits<PATH>::WAVES) qgemm_stream_kernel(const GroupedParams p)
{
    using T = SkinnyTraits<PATH>;
    using Frag = typename T::Frag;
    using Acc = typename T::Acc;
    constexpr bool MX = PATH == PATH_MX8 || PATH == PATH_MX4;
    constexpr bool BS = PATH == PATH_F8B;
    constexpr bool INK = MX || BS;
    constexpr int BM = 16 * TM;
    constexpr int D = StreamTraits<PATH>::D, NS = SK_WAVES;     // ring; sums
    static_assert(NS % D == 0, "a turn of the sums is whole turns of the ring");
    const int lane = threadIdx.x & 63;
    const int r16 = lane & 15, g = lane >> 4;
    const int wid = (int)blockIdx.x * (STREAM_THREADS / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = (int)gridDim.x * (STREAM_THREADS / 64);

    // Row tiles of the experts, counted as in grouped_tile.
    auto bound = [&](int e) { return min(max(p.offsets[e], 0), p.M); };
    auto tiles_of = [&](int lo, int hi) { return hi > lo ? (hi - lo + BM - 1) / BM : 0; };
    int first, count;              // this wave's tiles
    int expert, in_expert;         // of the first of them: its expert, its place there
    {
        const int share = (p.experts + 63) >> 6;
        const int e0 = min(lane * share, p.experts), e1 = min(e0 + share, p.experts);
        int n = 0, lo = bound(e0);
        for (int e = e0; e < e1; ++e) {
            const int hi = bound(e + 1);
            n += tiles_of(lo, hi);
            lo = hi;
        }
        int scan = n;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(scan, off);
            scan += lane >= off ? v : 0;
        }
        const int64_t total = (int64_t)__builtin_amdgcn_readlane(scan, 63) * p.tiles_n;
        first = (int)(total * wid / waves);
        count = (int)(total * (wid + 1) / waves) - first;
        if (count <= 0)
            return;
        const int owner = __builtin_ctzll(__ballot((int64_t)scan * p.tiles_n > first));
        int left = first -
                   (__builtin_amdgcn_readlane(scan, owner) - __builtin_amdgcn_readlane(n, owner)) * p.tiles_n;
        int e = owner * share;
        int a = bound(e), b = bound(e + 1);
        while (left >= tiles_of(a, b) * p.tiles_n && e + 1 < p.experts) {
            left -= tiles_of(a, b) * p.tiles_n;
            ++e;
            a = b;
            b = bound(e + 1);
        }
        expert = e;
        in_expert = left;
    }

    const int ksteps = (p.kbytes + T::KSTEP - 1) / T::KSTEP;
    const int turns = (ksteps + NS - 1) / NS;                   // of NS steps a tile

    // What a tile's loads need.  Descriptors of A and its scales cover the
    // tokens, or the tile's own rows.
    int e_lo = bound(expert), e_hi = bound(expert + 1);
    StreamTile cur;                                             // the tile being loaded
    __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
    unsigned b_row, sb_row = OOB, a_row[TM], sa_row[TM], src[TM];
    auto enter = [&]() {
        const int mt = max(tiles_of(e_lo, e_hi), 1);
        cur.expert = expert;
        cur.tn = in_expert / mt;
        cur.row0 = e_lo + (in_expert - cur.tn * mt) * BM;
        cur.rows = min(BM, e_hi - cur.row0);
        const int n0 = cur.tn * 16, rows_b = min(16, p.N - n0);
        rb = make_rsrc(p.B + (int64_t)expert * p.b_expert + (int64_t)n0 * p.ldb,
                       (uint32_t)((rows_b - 1) * p.ldb + p.kbytes));
        b_row = r16 < rows_b ? (unsigned)(r16 * p.ldb) : OOB;
        if constexpr (INK) {
            const int srows = (p.N + BROWS - 1) / BROWS;
            const int sb0 = n0 / BROWS, nsb = (n0 + rows_b - 1) / BROWS - sb0 + 1;
            rsb = make_rsrc(p.mx_sb + ((int64_t)expert * srows + sb0) * p.kblocks, (uint32_t)(nsb * p.kblocks));
            sb_row = r16 < rows_b ? (unsigned)(((n0 + r16) / BROWS - sb0) * p.kblocks) : OOB;
        }
        const int64_t base = p.order ? 0 : cur.row0;
        const int src_rows = p.order ? (int)p.a_rows : max(cur.rows, 1);
        ra = make_rsrc(p.A + base * p.lda, (uint32_t)((src_rows - 1) * p.lda + p.kbytes));
        if constexpr (INK)
            rsa = make_rsrc(p.mx_sa + base * p.kblocks, (uint32_t)(src_rows * p.kblocks));
        else
            rsa = make_rsrc(p.scale_a + base, (uint32_t)(src_rows * 4));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = 16 * i + r16;
            src[i] = ~0u;
            if (r < cur.rows)
                src[i] = p.order ? (unsigned)p.order[cur.row0 + r] / (unsigned)p.top_k : (unsigned)r;
            a_row[i] = src[i] < (unsigned)src_rows ? (unsigned)(src[i] * p.lda) : OOB;
            sa_row[i] = src[i] < (unsigned)src_rows ? (unsigned)(src[i] * (INK ? p.kblocks : 4)) : OOB;
        }
    };
    // the tile after: false at the end of this wave's
    auto next = [&]() {
        ++in_expert;
        while (in_expert >= tiles_of(e_lo, e_hi) * p.tiles_n) {
            if (expert + 1 >= p.experts)
                return;
            in_expert = 0;
            ++expert;
            e_lo = e_hi;
            e_hi = bound(expert + 1);
        }
    };

    Frag fa[D][TM], fb[D];
    // block scales: those of step s (BS); MX: the 16 bytes of a row that four
    // steps take (a quad), as loaded and as in use
    constexpr int NQD = D / 4;
    unsigned ssa[BS ? D : 1][TM], ssb[BS ? D : 1];
    u32x4 qa[MX ? NQD : 1][TM], qb[MX ? NQD : 1], ua[TM], ub;
    Acc acc[NS][TM];

    // Step s of the entered tile into ring slot SLOT (zeros past K).
    auto load = [&](auto slotc, int s) {
        constexpr int SLOT = decltype(slotc)::value;
#pragma unroll
        for (int c = 0; c < T::NCH; ++c) {
            const int kc = s * T::KSTEP + 64 * c + 16 * g;
            const bool kin = kc < p.kbytes;
            const u32x4 vb = ld16(rb, kin ? b_row + (unsigned)kc : OOB);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                fb[SLOT][4 * c + q] = (int)vb[q];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const u32x4 va = ld16(ra, kin ? a_row[i] + (unsigned)kc : OOB);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    fa[SLOT][i][4 * c + q] = (int)va[q];
            }
        }
        if constexpr (BS) {
            const bool bin = s < ksteps;
            ssb[SLOT] = __builtin_amdgcn_raw_buffer_load_b32(rsb, bin ? (unsigned)(4 * s) : OOB, 0, 0);
#pragma unroll
            for (int i = 0; i < TM; ++i)
                ssa[SLOT][i] = __builtin_amdgcn_raw_buffer_load_b32(rsa, bin ? sa_row[i] + (unsigned)(4 * s) : OOB, 0, 0);
        }
    };
    auto load_quad = [&](auto qc, int s) {
        constexpr int Q = decltype(qc)::value;
        if constexpr (MX) {
            qb[Q] = ld16(rsb, sb_row + (unsigned)(4 * s));
#pragma unroll
            for (int i = 0; i < TM; ++i)
                qa[Q][i] = ld16(rsa, sa_row[i] + (unsigned)(4 * s));
        }
    };
    // (words past K/32 are the next row's)
    auto use_quad = [&](auto qc, int s) {
        constexpr int Q = decltype(qc)::value;
        if constexpr (MX) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = s + j < ksteps;
                ub[j] = in ? qb[Q][j] : 0;
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    ua[i][j] = in ? qa[Q][i][j] : 0;
            }
        }
    };
    auto mma = [&](auto slotc, auto sumc) {
        constexpr int SLOT = decltype(slotc)::value;
        constexpr int SUM = decltype(sumc)::value;
        unsigned wb = 0;
        if constexpr (MX)
            wb = ub[SUM & 3] >> (8 * g);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            Acc &c = acc[SUM][i];
            if constexpr (PATH == PATH_I8) {
                c = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[SLOT], fa[SLOT][i], c, 0, 0, 0);
            } else if constexpr (PATH == PATH_F8) {
                c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[SLOT], fa[SLOT][i], c, 0, 0, 0, 0, 0, 0);
            } else if constexpr (PATH == PATH_MX8) {
                c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[SLOT], fa[SLOT][i], c, 0, 0, 0, (int)wb, 0,
                                                                     (int)(ua[i][SUM & 3] >> (8 * g)));
            } else if constexpr (PATH == PATH_F8B) {
                const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[SLOT], fa[SLOT][i], f32x4{}, 0, 0,
                                                                                   0, 0, 0, 0);
                const float w = __builtin_bit_cast(float, ssa[SLOT][i]) * __builtin_bit_cast(float, ssb[SLOT]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    c[r] = __builtin_fmaf(part[r], w, c[r]);
            } else {
                const i32x4 b4 = fb[SLOT], a4 = fa[SLOT][i];
                const i32x8 b8 = {b4[0], b4[1], b4[2], b4[3], 0, 0, 0, 0};
                const i32x8 a8 = {a4[0], a4[1], a4[2], a4[3], 0, 0, 0, 0};
                c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b8, a8, c, 4, 4, 0, (int)wb, 0,
                                                                     (int)(ua[i][SUM & 3] >> (8 * g)));
            }
        }
    };

    // (a quad's scales go out before its operands: loads return in order)
    enter();
    static_for<0, D>([&](auto sc) {
        constexpr int S = decltype(sc)::value;
        if constexpr (S % 4 == 0)
            load_quad(std::integral_constant<int, S / 4>(), S);
        load(sc, S);
    });
    for (int t = 0; t < count; ++t) {
        const StreamTile tile = cur;
        // (the row scales are the entered tile's: taken before the next one is)
        float sa[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            sa[i] = 1.0f;
            if constexpr (!INK)
                sa[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsa, sa_row[i], 0, 0));
        }
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < TM; ++i)
                acc[s][i] = Acc{};
        for (int turn = 0; turn < turns; ++turn) {
            static_for<0, NS / D>([&](auto hc) {
                constexpr int H = decltype(hc)::value;
                // the loads of this pass over the ring are for step NS * turn + D * (H + 1) on:
                // past the tile's last turn they are the next tile's first
                int ahead = NS * turn + D * (H + 1);
                if (H == NS / D - 1 && turn == turns - 1) {
                    ahead = 0;
                    if (t + 1 < count) {
                        next();
                        enter();
                    }
                }
                static_for<0, D>([&](auto sc) {
                    constexpr int S = decltype(sc)::value;
                    if constexpr (S % 4 == 0) {
                        use_quad(std::integral_constant<int, S / 4>(), NS * turn + D * H + S);
                        load_quad(std::integral_constant<int, S / 4>(), ahead + S);
                    }
                    mma(sc, std::integral_constant<int, D * H + S>());
                    load(sc, ahead + S);
                });
                static_for<0, D>([&](auto sc) {
#pragma unroll
                    for (int i = 0; i < TM; ++i)
                        keep_here(acc[D * H + decltype(sc)::value][i]);
                });
            });
        }

        // the eight sums in their order, then the epilogue of the main kernels
        const int n0 = tile.tn * 16, rows_b = min(16, p.N - n0), nloc = 4 * g;
        const bool full_n = nloc + 4 <= rows_b;
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
        for (int i = 0; i < TM; ++i) {
            Acc sum = acc[0][i];
#pragma unroll
            for (int s = 1; s < NS; ++s)
                sum += acc[s][i];
            const int mloc = 16 * i + r16;
            if (mloc >= tile.rows)
                continue;
            float f[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x = (float)sum[r];
                if constexpr (!INK) {
                    x = x * sa[i];
                    x = x * __builtin_bit_cast(float, sbw[r]);
                }
                if constexpr (BIAS)
                    x = x + __builtin_bit_cast(float, bbw[r]);
                f[r] = x;
            }
            uint16_t *out = (uint16_t *)p.C + (int64_t)(tile.row0 + mloc) * p.ldc + n0 + nloc;
            const u32x2 v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
            if (full_n) {
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
