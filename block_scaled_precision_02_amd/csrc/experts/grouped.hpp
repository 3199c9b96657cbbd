// grouped.hpp -- grouped products: the host's choice of tile and the launch of
// one path's kernels.
#pragma once
#include <algorithm>

#include "../qgemm_launch.hpp"
#include "experts.hpp"
#include "grouped_panel.hpp"
#include "grouped_stream.hpp"

namespace qgemm {

// Tiles of grouped products beside those of the host table (qgemm_launch.hpp):
//  16 -> 16 rows by 16 columns, a wave over the whole of K (grouped_stream.hpp)
//  17 -> 64 rows by 128 columns, B straight into registers (grouped_panel.hpp)
//  18 -> 128 rows by 256 columns, eight waves, fetched into LDS (qgemm_dma.hpp): an
//        expert's rows are read half as often from L2 as by 128 columns
constexpr int STREAM16_TILE = 16, PANEL64_TILE = 17, WIDE128_TILE = 18;

// Per-path entry points, one translation unit each.
hipError_t launch_grouped_i8(int tile, bool bias, const GroupedParams &p, hipStream_t s);
hipError_t launch_grouped_f8(int tile, bool bias, const GroupedParams &p, hipStream_t s);
hipError_t launch_grouped_f8b(int tile, bool bias, const GroupedParams &p, hipStream_t s);
hipError_t launch_grouped_mx8(int tile, bool bias, const GroupedParams &p, hipStream_t s);
hipError_t launch_grouped_mx4(int tile, bool bias, const GroupedParams &p, hipStream_t s);

template <int PATH, bool BIAS>
hipError_t launch_grouped_tile(int tile, const GroupedParams &p, hipStream_t s)
{
    constexpr int BROWS = PATH == PATH_F8B ? 128 : 1;
    if (tile == STREAM16_TILE) {
        // what is resident at once, by the registers
        static const int per_cu = [] {
            int n = 0;
            if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, qgemm_stream_kernel<PATH, 1, BIAS, BROWS>,
                                                             STREAM_THREADS, 0) != hipSuccess || n < 1)
                n = 2;
            return n;
        }();
        const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, waves = STREAM_THREADS / 64;
        const unsigned blocks = (unsigned)std::min<int64_t>(256 * per_cu, (tiles + waves - 1) / waves);
        hipLaunchKernelGGL((qgemm_stream_kernel<PATH, 1, BIAS, BROWS>), dim3(blocks), dim3(STREAM_THREADS), 0, s, p);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((int64_t)p.tiles_m * p.tiles_n)), block(tile_threads(tile));
    switch (tile) {
    case PANEL64_TILE:
        hipLaunchKernelGGL((qgemm_panel_kernel<PATH, 4, BIAS, BROWS>), grid, dim3(PANEL_THREADS), 0, s, p);
        break;
    case WIDE128_TILE:
        hipLaunchKernelGGL((qgemm_dma_kernel<PATH, 4, 2, 2, BIAS, BROWS, OUT_BF16, false, true>), grid, dim3(512), 0, s, p);
        break;
    case SKINNY16_TILE:
        hipLaunchKernelGGL((qgemm_skinny_kernel<PATH, 1, skinny_depth<PATH, 1>(), BIAS, BROWS, true>), grid, block, 0, s,
                           p);
        break;
    case DMA128_TILE:
        hipLaunchKernelGGL((qgemm_dma_kernel<PATH, 2, 2, 2, BIAS, BROWS, OUT_BF16, false, true>), grid, block, 0, s, p);
        break;
    case DMA8_TILE:
        if constexpr (PATH != PATH_F8B) {
            hipLaunchKernelGGL((qgemm_dma_kernel<PATH, 4, 4, 2, BIAS, BROWS, OUT_BF16, false, true>), grid, block, 0, s,
                               p);
            break;
        }
        return hipErrorInvalidValue;
    case F8B256_TILE:
        if constexpr (PATH == PATH_F8B) {
            hipLaunchKernelGGL((qgemm_dma_kernel<PATH, 2, 4, 2, BIAS, BROWS, OUT_BF16, false, true>), grid, block, 0, s,
                               p);
            break;
        }
        return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace qgemm
