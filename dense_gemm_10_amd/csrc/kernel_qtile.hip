// Instantiations of the products with 4-bit weights (qstream.hpp): many rows.
#include "qstream.hpp"

namespace dg {

hipError_t launch_qweight_tile(const QweightArgs &a, uint32_t programs, hipStream_t s)
{
    return launch_shape<4, 2, 8, 1, 2, 64>(a, programs, s);
}

} // namespace dg
