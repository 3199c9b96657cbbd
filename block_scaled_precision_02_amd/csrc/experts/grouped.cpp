// grouped.cpp -- grouped products: the tile for a call and its parameters.
#include <algorithm>
#include <cstring>

#include "grouped.hpp"

namespace qgemm {

namespace {

// The tile by the rows an expert has on average (how they are spread is known
// on the device alone).
int pick_tile(int path, const GroupedArgs &a)
{
    const int64_t each = (a.rows + a.experts - 1) / a.experts;
    if (each <= 16)
        return SKINNY16_TILE;
    if (each <= 160)
        return DMA128_TILE;
    return path == PATH_F8B ? F8B256_TILE : DMA8_TILE;
}

// The most row tiles there can be: one partly filled for each expert with rows.
int64_t most_tiles_m(int tile, const GroupedArgs &a)
{
    return a.rows / tile_edge_m(tile) + std::min<int64_t>(a.rows, a.experts);
}

int64_t tiles_n(int tile, const GroupedArgs &a) { return ((int64_t)a.N + tile_edge_n(tile) - 1) / tile_edge_n(tile); }

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
