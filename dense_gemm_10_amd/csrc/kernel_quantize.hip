// 8-bit codes and scales of rows (codes.hpp): one workgroup per token; a row of
// up to 8 CHUNKS x 256 elements stays in registers, so x is read once.
//
// Measured (MI355X, bf16, kernel times): 8232 x 4096 22.9 us, 102 MB moved, 4.4
// TB/s; 2048 x 4096 8.9 us, 2.9 TB/s.  In a graph 512 rows of 4096 take 4.5 us,
// 1024 5.8, 2048 9.0, 4096 14.7, 8232 24.2: some 3 us of launch, load, barrier
// and store in turn before the last figure's rate is reached.
#include "codes.hpp"

namespace dg {

namespace {

constexpr int QT = 256;

__device__ __forceinline__ void store_codes(int8_t *p, uint2 c, int n)
{
    if (n >= 8) {
        __builtin_memcpy(p, &c, 8);
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            p[e] = (int8_t)((e < 4 ? c.x : c.y) >> (8 * (e % 4)));
}

// CHUNKS > 0: the row is held, 8 elements per thread and chunk; 0: any
// length, read twice.
template <int T, int CHUNKS>
__global__ __launch_bounds__(QT) void quantize_kernel(QuantizeArgs a)
{
    constexpr int ES = elem_bytes<T>(), NC = CHUNKS > 0 ? CHUNKS : 1;
    __shared__ uint32_t tops[2][QT / 64];
    const int tid = threadIdx.x;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x, turn ^= 1) {
        const char *row = a.x + t * a.ldx;
        Raw8<T> held[NC];
        uint32_t m = 0;
        auto left = [&](int64_t c) {               // elements of the piece at c
            const int64_t n = a.width - c;
            return n < 0 ? 0 : n > 8 ? 8 : (int)n;
        };
        if constexpr (CHUNKS > 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = (int64_t)(i * QT + tid) * 8;
                held[i] = load_raw8<T>(row + c * ES, left(c));
            }
#pragma unroll
            for (int i = 0; i < NC; ++i)
                m = max(m, raw_abs_max<T>(held[i]));
        } else {
            for (int64_t c = (int64_t)tid * 8; c < a.width; c += QT * 8)
                m = max(m, raw_abs_max<T>(load_raw8<T>(row + c * ES, left(c))));
        }
        m = wave_max(m);
        if ((tid & 63) == 0)
            tops[turn][tid >> 6] = m;
        __syncthreads();                            // the next token uses the other half
#pragma unroll
        for (int w = 0; w < QT / 64; ++w)
            m = max(m, tops[turn][w]);
        const RowScale s = row_scale<T>(m);
        const int32_t copies = a.place ? a.top_k : 1;
        auto put = [&](int64_t c, uint2 q) {
            for (int32_t j = 0; j < copies; ++j) {
                int64_t p = t;
                if (a.place) {
                    p = a.place[t * a.top_k + j];
                    if (p < 0 || p >= a.limit)
                        continue;
                }
                store_codes(a.q + p * a.ldq + c, q, left(c));
            }
        };
        if constexpr (CHUNKS > 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = (int64_t)(i * QT + tid) * 8;
                if (c < a.width)
                    put(c, codes<T>(held[i], s));
            }
        } else {
            for (int64_t c = (int64_t)tid * 8; c < a.width; c += QT * 8)
                put(c, codes<T>(load_raw8<T>(row + c * ES, left(c)), s));
        }
        for (int32_t j = tid; j < copies; j += QT) {
            const int64_t p = a.place ? a.place[t * a.top_k + j] : t;
            if (!a.place || (p >= 0 && p < a.limit))
                a.scales[p] = s.scale;
        }
    }
}

template <int T>
void quantize_choice(const QuantizeArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)(a.tokens < (1 << 20) ? a.tokens : 1 << 20)), block(QT);
    if (a.width <= QT * 8)
        hipLaunchKernelGGL((quantize_kernel<T, 1>), grid, block, 0, s, a);
    else if (a.width <= 2 * QT * 8)
        hipLaunchKernelGGL((quantize_kernel<T, 2>), grid, block, 0, s, a);
    else if (a.width <= 4 * QT * 8)
        hipLaunchKernelGGL((quantize_kernel<T, 4>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((quantize_kernel<T, 0>), grid, block, 0, s, a);
}

} // namespace

hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t s)
{
    if (a.x_type == DT_F32)
        quantize_choice<DT_F32>(a, s);
    else if (a.x_type == DT_F16)
        quantize_choice<DT_F16>(a, s);
    else
        quantize_choice<DT_BF16>(a, s);
    return hipGetLastError();
}

} // namespace dg
