// Grouped products, MX, e2m1 elements.
#include "grouped.hpp"

namespace qgemm {
hipError_t launch_grouped_mx4(int tile, bool bias, const GroupedParams &p, hipStream_t s)
{
    return bias ? launch_grouped_tile<PATH_MX4, true>(tile, p, s) : launch_grouped_tile<PATH_MX4, false>(tile, p, s);
}
}  // namespace qgemm
