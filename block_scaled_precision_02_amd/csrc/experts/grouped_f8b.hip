// Grouped products, e4m3 with fp32 scales per 128 K elements.
#include "grouped.hpp"

namespace qgemm {
hipError_t launch_grouped_f8b(int tile, bool bias, const GroupedParams &p, hipStream_t s)
{
    return bias ? launch_grouped_tile<PATH_F8B, true>(tile, p, s) : launch_grouped_tile<PATH_F8B, false>(tile, p, s);
}
}  // namespace qgemm
