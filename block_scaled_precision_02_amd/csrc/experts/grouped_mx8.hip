// Grouped products, MX, e4m3 elements.
#include "grouped.hpp"

namespace qgemm {
hipError_t launch_grouped_mx8(int tile, bool bias, const GroupedParams &p, hipStream_t s)
{
    return bias ? launch_grouped_tile<PATH_MX8, true>(tile, p, s) : launch_grouped_tile<PATH_MX8, false>(tile, p, s);
}
}  // namespace qgemm
