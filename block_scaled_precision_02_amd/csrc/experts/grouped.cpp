// grouped.cpp -- grouped products: the tile for a call and its parameters.
#include <algorithm>
#include <cstring>

#include "grouped.hpp"

namespace qgemm {

namespace {

// The tile by what the host knows: the rows an expert has on average (how they
// are spread is known on the device alone) and the most experts that can have
// any.  One MI355X, us, experts chosen at random, some more often:
//  * Above 96 rows an expert the 256-row tiles, bound by the matrix cores (64
//    experts of 4096x4096: at 122 rows i8 288 and 337 on 128x128, at 66 rows 267
//    and 270; e2m1 178 and 187, 161 and 152).  Blockscale, whose 256x128 tile has
//    one wave a SIMD, from 2048 rows (8 of 4096x4096, 4096 rows: 714 and 749; 64
//    of 4096x2048, 375 rows: 364 and 354).
//  * Above 16 the 128x128 tile (64 of 4096x4096, 32 rows: i8 241, panel 247; e2m1
//    139 and 148).
//  * Up to 16 rows the weights' bytes are all that counts, and a chip full of
//    loads: the panel where it has two workgroups a CU (64 tokens, 8 of 256
//    experts of 2048x7168: blockscale 418, 128x128 451, stream 572; 16 tokens, 8 of
//    128 of 4096x7168: e4m3 MX 363, 409 and 350).
//  * Fewer workgroups: the stream, whose waves each take 16 columns (3 tokens, 8
//    of 64 of 2112x7168: e4m3 MX 67, panel 82, 128x128 87; one token, 2048x7168: i8
//    23, 35 and 39) while an expert's rows are one tile of it mostly; else the
//    128x128 tile (10 tokens, 4 of 8 of 4096x4096: 35 for all three).
//  * So few columns that a wave over K would be the whole time: the small-M
//    kernel, eight waves over K (one token, 8 of 64 of 512x7168: i8 10.5, stream
//    20, 128x128 24; 1024x7168: 19, 20 and 25).
int pick_tile(int path, const GroupedArgs &a)
{
    const int64_t each = (a.rows + a.experts - 1) / a.experts;
    if (each > (path == PATH_F8B ? 2048 : 96))
        return path == PATH_F8B ? F8B256_TILE : DMA8_TILE;
    if (each > 16)
        return DMA128_TILE;
    const int64_t panels = std::min<int64_t>(a.rows, a.experts) * ((a.N + PANEL_BN - 1) / PANEL_BN);
    if (panels <= 64)
        return SKINNY16_TILE;
    if (panels >= 512)
        return PANEL64_TILE;
    return each <= 4 ? STREAM16_TILE : DMA128_TILE;
}

int edge_m(int tile) { return tile == STREAM16_TILE ? 16 : tile == PANEL64_TILE ? 64 : tile_edge_m(tile); }
int edge_n(int tile) { return tile == STREAM16_TILE ? 16 : tile == PANEL64_TILE ? PANEL_BN : tile_edge_n(tile); }

// The most row tiles there can be: one partly filled for each expert with rows.
int64_t most_tiles_m(int tile, const GroupedArgs &a)
{
    return a.rows / edge_m(tile) + std::min<int64_t>(a.rows, a.experts);
}

int64_t tiles_n(int tile, const GroupedArgs &a) { return ((int64_t)a.N + edge_n(tile) - 1) / edge_n(tile); }

}  // namespace

bool grouped_fits(int path, const GroupedArgs &a)
{
    const int tile = pick_tile(path, a);
    // fewer than 2^32 threads a launch
    return most_tiles_m(tile, a) * tiles_n(tile, a) < ((int64_t)1 << 32) / tile_threads(tile);
}

hipError_t launch_grouped(int path, const GroupedArgs &a, hipStream_t s)
{
    const int tile = pick_tile(path, a);
    GroupedParams p;
    memset(&p, 0, sizeof p);
    p.A = a.A;
    p.B = a.B;
    p.lda = a.lda;
    p.ldb = a.ldb;
    p.b_expert = a.b_expert;
    if (path == PATH_I8 || path == PATH_F8) {
        p.scale_a = (const float *)a.SA;
        p.scale_b = (const float *)a.SB;
    } else {
        p.mx_sa = (const uint8_t *)a.SA;
        p.mx_sb = (const uint8_t *)a.SB;
    }
    p.bias = a.bias;
    p.C = a.C;
    p.ldc = a.ldc;
    p.M = (int)a.rows;
    p.N = a.N;
    p.K = a.K;
    p.kbytes = path == PATH_MX4 ? a.K / 2 : a.K;
    p.ksteps = (p.kbytes + KSTEP_BYTES - 1) / KSTEP_BYTES;
    p.kblocks = a.K / 32;
    p.tiles_m = (int)most_tiles_m(tile, a);
    p.tiles_n = (int)tiles_n(tile, a);
    p.group_m = is_skinny_tile(tile) ? 1 : 8;
    p.c_cached = 1;
    p.offsets = a.offsets;
    p.order = a.order;
    p.a_rows = a.a_rows;
    p.top_k = a.top_k;
    p.experts = a.experts;
    switch (path) {
    case PATH_I8: return launch_grouped_i8(tile, a.bias != nullptr, p, s);
    case PATH_F8: return launch_grouped_f8(tile, a.bias != nullptr, p, s);
    case PATH_F8B: return launch_grouped_f8b(tile, a.bias != nullptr, p, s);
    case PATH_MX8: return launch_grouped_mx8(tile, a.bias != nullptr, p, s);
    default: return launch_grouped_mx4(tile, a.bias != nullptr, p, s);
    }
}

}  // namespace qgemm
