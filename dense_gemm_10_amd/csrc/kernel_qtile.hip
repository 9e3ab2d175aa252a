// Instantiations of the products with 4-bit weights (qstream.hpp): many rows.
#include "qstream.hpp"

namespace dg {

hipError_t launch_qweight_tile(const QweightArgs &a, uint32_t programs, hipStream_t s)
{
    return launch_shape<4, 2, 8, 1, 2, 64>(a, programs, s);
}

// Group sizes that are multiples of 128 only: with more scales in a panel
// the eight wavefronts' sums do not fit into registers.
hipError_t launch_qweight_wide_tile(const QweightArgs &a, uint32_t programs, hipStream_t s)
{
    return launch_scaled<4, 4, 4, 8, 1, 1, 64>(a, programs, s);
}

} // namespace dg
