// 8-bit codes of rows: the row's largest absolute value by an integer maximum
// of the bits below the sign (a NaN is the largest, an infinity the next, so
// neither is lost), then the codes.
//
// The code is the nearest integer to 127 x / max, ties to even, from the
// exact quotient: with both scaled by a power of two so that max is in
// [1, 2), x * (127 / max) in fp32 is off by less than 127 * 3 * 2^-24 <
// 3e-5, so the nearest integer is right unless the rest comes within 1e-4 of
// a half; then the sign of 127 x - (q +- 1/2) max decides, exact in fp64.
#pragma once
#include "tokens.hpp"

namespace dg {

namespace {

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
    float scale;         // largest absolute value / 127
    int shift;
    bool zero;           // every code is 0
};

template <int T>
__device__ __forceinline__ RowScale row_scale(uint32_t bits)
{
    const float top = T == DT_F32 ? __uint_as_float(bits)
                                  : half_to_f32<T == DT_F32 ? DT_BF16 : T>((uint16_t)bits);
    const bool finite = top < __builtin_inff();                // false for NaN
    RowScale s;
    s.zero = !finite || top == 0.0f;
    s.shift = s.zero ? 0 : 1 - __builtin_amdgcn_frexp_expf(top);
    s.top = s.zero ? 1.0f : __builtin_amdgcn_ldexpf(top, s.shift);
    s.inv = 127.0f / s.top;
    s.scale = finite ? (float)((double)top / 127.0) : __builtin_nanf("");
    return s;
}

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

} // namespace

} // namespace dg
