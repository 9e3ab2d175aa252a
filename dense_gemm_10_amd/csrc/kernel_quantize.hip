// 8-bit codes and scales of rows.
//
// One workgroup per token: the row's largest absolute value by an integer
// maximum of the bits below the sign (a NaN is the largest, an infinity the
// next, so neither is lost), then the codes.  A row of up to 8 CHUNKS x
// 256 elements stays in registers, so x is read once.
//
// The code is the nearest integer to 127 x / max, ties to even, from the
// exact quotient: with both scaled by a power of two so that max is in
// [1, 2), x * (127 / max) in fp32 is off by less than 127 * 3 * 2^-24 <
// 3e-5, so the nearest integer is right unless the rest comes within 1e-4 of
// a half; then the sign of 127 x - (q +- 1/2) max decides, exact in fp64.
#include "grouped.hpp"
#include "tokens.hpp"

namespace dg {

namespace {

constexpr int QT = 256;

template <int T>
__device__ __forceinline__ uint32_t raw_abs_max(const Raw8<T> &r)      // fp32: bits; else 16 bits
{
    uint32_t m = 0;
    if constexpr (T == DT_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, r.w[i] & 0x7fffffffu);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = max(m, r.w[i] & 0x7fffu);
            m = max(m, (r.w[i] >> 16) & 0x7fffu);
        }
    }
    return m;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v)               // v below 2^31
{
    return (uint32_t)__builtin_amdgcn_readlane(wave_scan_max((int32_t)v), 63);
}

struct RowScale {
    float top, inv;      // of the row scaled by 2^shift: in [1, 2), and 127 / top
    int shift;
    bool zero;           // every code is 0
};

// The code of x from the exact quotient.
__device__ __forceinline__ float exact_code(float xs, float q, float top)
{
    const double r2 = 2.0 * (127.0 * (double)xs - (double)q * (double)top);   // exact
    const double t = (double)top;
    const bool odd = ((int)q & 1) != 0;
    if (r2 > t || (r2 == t && odd))
        return q + 1.0f;
    if (r2 < -t || (r2 == -t && odd))
        return q - 1.0f;
    return q;
}

// Eight codes, packed.
template <int T>
__device__ __forceinline__ uint2 codes(const Raw8<T> &r, const RowScale &s)
{
    float q[8], worst = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = __builtin_amdgcn_ldexpf(raw_value<T>(r, e), s.shift) * s.inv;
        q[e] = __builtin_rintf(v);
        worst = fmaxf(worst, fabsf(v - q[e]));
    }
    if (worst > 0.4999f) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            q[e] = exact_code(__builtin_amdgcn_ldexpf(raw_value<T>(r, e), s.shift), q[e], s.top);
    }
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        b[e] = s.zero ? 0u : (uint32_t)(int32_t)q[e] & 255u;
    return make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
}

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
        const float top = T == DT_F32 ? __uint_as_float(m)
                                      : half_to_f32<T == DT_F32 ? DT_BF16 : T>((uint16_t)m);
        const bool finite = top < __builtin_inff();            // false for NaN
        RowScale s;
        s.zero = !finite || top == 0.0f;
        s.shift = s.zero ? 0 : 1 - __builtin_amdgcn_frexp_expf(top);
        s.top = s.zero ? 1.0f : __builtin_amdgcn_ldexpf(top, s.shift);
        s.inv = 127.0f / s.top;
        const float scale = finite ? (float)((double)top / 127.0) : __builtin_nanf("");
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
                a.scales[p] = scale;
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
