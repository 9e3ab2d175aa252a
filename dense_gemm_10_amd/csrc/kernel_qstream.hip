// Instantiations of the products with 4-bit weights (qstream.hpp): few rows.
#include "qstream.hpp"

namespace dg {

hipError_t launch_qweight_rows(int32_t variant, const QweightArgs &a, uint32_t programs,
                               hipStream_t s)
{
    switch (variant) {
    case 0: return launch_shape<1, 1, 1, 8, 2, 16>(a, programs, s);
    case 1: return launch_shape<1, 1, 2, 4, 2, 16>(a, programs, s);
    case 2: return launch_shape<1, 1, 4, 2, 2, 16>(a, programs, s);
    case 3: return launch_shape<2, 1, 2, 4, 2, 32>(a, programs, s);
    case 4: return launch_shape<2, 1, 4, 2, 2, 32>(a, programs, s);
    case 5: return launch_shape<2, 2, 4, 2, 1, 32>(a, programs, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace dg
