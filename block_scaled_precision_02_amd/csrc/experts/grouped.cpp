// grouped.cpp -- grouped products: the tile for a call and its parameters.
#include <algorithm>
#include <cstring>

#include "grouped.hpp"

namespace qgemm {

namespace {

// The tile by what the host knows: the rows an expert has room for on average
// (how many there are, fewer than that where slots belong to other ranks'
// experts, and how they are spread, is known on the device alone: 64 experts of
// 4096x4096, 8192 slots on 4 ranks, i8 219 us, by the live rows' tile 208; 16 of
// 2048x7168, 128 slots on 8 ranks, 36 and 53) and the most experts that can have
// any.  One MI355X, us; "of random experts": some chosen more often than others,
// else every expert has the rows named:
//  * Above 96 rows an expert the 256-row tiles, bound by the matrix cores (32
//    experts of 4096x4096, 190 rows: i8 156 and 191 on 128x256, e2m1 91 and 120;
//    100 rows: 148 and 141, 73 and 71).  Blockscale, whose 256x128 tile has one
//    wave a SIMD, from 448 rows (375 rows: 319 and 300, 512 rows: 369 and 387).
//  * Above 16 the 128x256 tile, bound by its loads (64 of 7168x2048, 64 rows:
//    blockscale 204, 128x128 224, panel 217; i8 199, 222 and 231), where its tiles
//    fill the CUs they are spread over: it takes a CU for itself (8 of 4096x4096,
//    128 tiles: i8 30, 128x128 23; 24, 384 tiles: 113 and 98; 16, 256 tiles: 44 and
//    48).  Else 128x128, two a CU.
//  * Up to 16 rows the weights' bytes are all that counts, and a chip full of
//    loads: the panel where it has two workgroups a CU (64 of 4096x7168, 16 rows:
//    i8 321, 128x256 339, 128x128 348; 64 tokens, 8 of 256 random experts of
//    2048x7168: blockscale 418, stream 572).
//  * Fewer workgroups: the stream, whose waves each take 16 columns (3 tokens, 8
//    of 64 of 2112x7168: e4m3 MX 67, panel 82, 128x128 87; one token, 2048x7168: i8
//    23, 35 and 39) while an expert's rows are one tile of it mostly; else the
//    128x128 tile (10 tokens, 4 of 8 of 4096x4096: 35 for all three).
//  * So few columns that a wave over K would be the whole time: the small-M
//    kernel, eight waves over K (one token, 8 of 64 of 512x7168: i8 10.5, stream
//    20, 128x128 24; 1024x7168: 19, 20 and 25).
int pick_tile(int path, const GroupedArgs &a)
{
    const int64_t each = (a.rows + a.experts - 1) / a.experts, with_rows = std::min<int64_t>(a.rows, a.experts);
    if (each > (path == PATH_F8B ? 448 : 96))
        return path == PATH_F8B ? F8B256_TILE : DMA8_TILE;
    if (each > 16) {
        const int64_t wide = with_rows * ((each + 127) / 128) * ((a.N + 255) / 256), rounds = (wide + 255) / 256;
        return wide >= 768 || 8 * wide >= 7 * 256 * rounds ? WIDE128_TILE : DMA128_TILE;
    }
    const int64_t panels = with_rows * ((a.N + PANEL_BN - 1) / PANEL_BN);
    if (panels <= 64)
        return SKINNY16_TILE;
    if (panels >= 512)
        return PANEL64_TILE;
    return each <= 4 ? STREAM16_TILE : DMA128_TILE;
}

int edge_m(int tile)
{
    return tile == STREAM16_TILE ? 16 : tile == PANEL64_TILE ? 64 : tile == WIDE128_TILE ? 128 : tile_edge_m(tile);
}

int edge_n(int tile)
{
    return tile == STREAM16_TILE ? 16 : tile == PANEL64_TILE ? PANEL_BN : tile == WIDE128_TILE ? 256 : tile_edge_n(tile);
}

int threads(int tile) { return tile == WIDE128_TILE ? 512 : tile_threads(tile); }

// The most row tiles there can be: one partly filled for each expert with rows.
int64_t most_tiles_m(int tile, const GroupedArgs &a)
{
    return a.rows / edge_m(tile) + std::min<int64_t>(a.rows, a.experts);
}

int64_t tiles_n(int tile, const GroupedArgs &a) { return ((int64_t)a.N + edge_n(tile) - 1) / edge_n(tile); }

}  // namespace

int grouped_tile_id(int path, const GroupedArgs &a) { return pick_tile(path, a); }

bool grouped_fits(int path, const GroupedArgs &a)
{
    const int tile = pick_tile(path, a);
    // fewer than 2^32 threads a launch
    return most_tiles_m(tile, a) * tiles_n(tile, a) < ((int64_t)1 << 32) / threads(tile);
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
    // Tiles in the order of experts and columns (an expert's weights go by once,
    // its rows stay in L2) up to 256 rows an expert, in groups of eight row tiles
    // above; one MI355X, us, groups of one and of eight: 64 experts of 4096x4096 i8,
    // 16 rows 195 and 217, 66 rows 259 and 273, 188 rows 347 and 358; of 2048x8192, 32
    // rows 221 and 263 (eight experts' rows at one stride of 8 KB share memory
    // channels); 32 of 4096x7168, 1024 rows 1005 and 975.
    p.group_m = (a.rows + a.experts - 1) / a.experts <= 256 ? 1 : 8;
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
