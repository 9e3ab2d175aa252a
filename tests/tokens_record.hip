// Stand-ins for the launchers of the routed-token kernels that keep what they
// are given, for tests of the host side on the CPU (tests/test_tokens_launches.py).
#include "tokens.hpp"

namespace dg {

static CombineArgs last;

hipError_t launch_dispatch_sort(const DispatchArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_dispatch_few(const DispatchArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_spread(const SpreadArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize(const QuantizeArgs &, hipStream_t) { return hipSuccess; }

hipError_t launch_combine(const CombineArgs &a, hipStream_t)
{
    last = a;
    return hipSuccess;
}

hipError_t launch_combine_grad(const CombineArgs &a, hipStream_t)
{
    last = a;
    return hipSuccess;
}

} // namespace dg

// y (dy), z, weights; tokens, top_k, rows, columns of the last combine launch
extern "C" void last_combine(int64_t *out)
{
    const dg::CombineArgs &a = dg::last;
    const int64_t v[] = {(int64_t)a.y, (int64_t)a.z, (int64_t)a.w, a.tokens, a.top_k, a.limit, a.width};
    for (int i = 0; i < 7; ++i)
        out[i] = v[i];
}
