// Stand-ins for the launchers of the routed-token and 8-bit kernels, linked
// into the host-code sanitizer build of the library
// (tests/test_tokens_sanitizers.py) in place of the kernels.  Nothing in that
// test launches a kernel; each stand-in reports a launch error if it is ever
// reached.
#include "scaled.hpp"
#include "tokens.hpp"

namespace dg {

hipError_t launch_dispatch_sort(const DispatchArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_dispatch_few(const DispatchArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_spread(const SpreadArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_combine(const CombineArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_combine_grad(const CombineArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_quantize(const QuantizeArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_scaled_stream(int32_t, const ScaledArgs &, uint32_t, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_scaled_few(int32_t, const ScaledArgs &, uint32_t, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_scaled_tile(int32_t, const ScaledArgs &, uint32_t, hipStream_t) { return hipErrorInvalidValue; }

} // namespace dg
