// Tokens sorted by group and back, and 8-bit codes of rows: the kernels'
// arguments and launchers (kernel_dispatch.hip, kernel_combine.hip,
// kernel_quantize.hip; host side in tokens_api.cpp).
#pragma once
#include "grouped.hpp"

namespace dg {

constexpr int64_t kMaxDispatchGroups = 8192;   // counters of a workgroup fit its LDS

struct DispatchArgs {
    const void *index;
    const char *x;             // null: maps only
    int32_t *offsets, *order, *place;
    char *rows;
    int64_t ld_index;          // elements
    int64_t ldx, ldr;          // bytes
    int64_t width;             // bytes of a row
    int32_t slots, top_k, groups;
    int32_t index_bits;
    int32_t elem;              // bytes of an element
};

struct SpreadArgs {
    const char *x;
    char *rows;
    const int32_t *place;
    int64_t ldx, ldr, width;   // bytes
    int64_t tokens;
    int32_t top_k, limit;      // rows in [0, limit)
    int32_t elem;
};

struct CombineArgs {
    const char *z;
    char *y;                   // dy in the gradient, read only
    const int32_t *place;
    const void *w;             // null: ones
    char *dz;
    void *dw;
    int64_t ldz, lddz, ldy;    // bytes
    int64_t ldw;               // elements
    int64_t tokens, width;     // width in elements
    int32_t top_k, limit;
    int32_t z_type, y_type, w_type;
    float beta;
};

struct QuantizeArgs {
    const char *x;
    const int32_t *place;      // null: row t
    int8_t *q;
    float *scales;
    int64_t ldx, ldq;          // bytes
    int64_t tokens, width;
    int32_t top_k, limit;
    int32_t x_type;
};

// Launchers; each returns hipSuccess or the launch error.
hipError_t launch_dispatch_sort(const DispatchArgs &a, hipStream_t s);
// maps and rows in one launch; slots <= kDispatchFewSlots
hipError_t launch_dispatch_few(const DispatchArgs &a, hipStream_t s);
hipError_t launch_spread(const SpreadArgs &a, hipStream_t s);
hipError_t launch_combine(const CombineArgs &a, hipStream_t s);
hipError_t launch_combine_grad(const CombineArgs &a, hipStream_t s);
hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t s);

// 4096 slots, 2 a token, 4096 bf16: 14.8 us against 7.3 + 9.8; 6000 slots 19.8
// against 7.6 + 7.2
constexpr int32_t kDispatchFewSlots = 4096;

// ---- eight elements of a row -------------------------------------------------
// Rows start on any element, so 16 bytes go by loads and stores that need no
// alignment (gfx950 takes them at any address).
struct Raw16 { uint32_t w[4]; };

__device__ __forceinline__ Raw16 load_raw16(const char *p)
{
    Raw16 r;
    __builtin_memcpy(&r, p, 16);
    return r;
}

// Outputs are written non-temporal: they are read, if at all, by another
// kernel, from beyond the L2s (combine with gradients, 4095 tokens, 8 rows
// each, 1000 fp16: 54.6 us with plain stores, 41.5 so; 8192 tokens, 2 rows, 4096
// bf16: 107 and 101, and their dispatch with its gradient 96 and 89).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void store_raw16(char *p, const Raw16 &r)
{
    const u32x4_any v = {r.w[0], r.w[1], r.w[2], r.w[3]};
    __builtin_nontemporal_store(v, (u32x4_any *)p);
}

template <int T> constexpr int elem_bytes() { return T == DT_F32 ? 4 : 2; }

// Eight elements as they lie in memory.
template <int T> struct Raw8 { uint32_t w[T == DT_F32 ? 8 : 4]; };

// Elements [0, n) of the eight at p; zeros behind them.  LAST: what is read
// will not be read again soon, and is loaded non-temporal.
template <int T, bool LAST = false>
__device__ __forceinline__ Raw8<T> load_raw8(const char *p, int n)
{
    Raw8<T> r;
    if (n >= 8) {
        if constexpr (LAST) {
#pragma unroll
            for (int i = 0; i < (int)sizeof r / 16; ++i) {
                const u32x4_any v = __builtin_nontemporal_load((const u32x4_any *)(p + 16 * i));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r.w[4 * i + e] = v[e];
            }
        } else {
            __builtin_memcpy(&r, p, sizeof r);
        }
        return r;
    }
    r = Raw8<T>{};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e >= n)
            continue;
        if constexpr (T == DT_F32)
            r.w[e] = ((const uint32_t *)p)[e];
        else
            r.w[e / 2] |= (uint32_t)((const uint16_t *)p)[e] << (16 * (e % 2));
    }
    return r;
}

template <int T>
__device__ __forceinline__ float raw_value(const Raw8<T> &r, int e)
{
    if constexpr (T == DT_F32)
        return __uint_as_float(r.w[e]);
    else
        return half_to_f32<T>((uint16_t)(r.w[e / 2] >> (16 * (e % 2))));
}

// Elements [0, n) of v, each rounded once.
template <int T>
__device__ __forceinline__ void store_8(char *p, const float (&v)[8], int n)
{
    Raw8<T> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (T == DT_F32)
            r.w[e] = __float_as_uint(v[e]);
        else if (e % 2 == 0)
            r.w[e / 2] = (uint32_t)f32_to_half<T>(v[e]) | (uint32_t)f32_to_half<T>(v[e + 1]) << 16;
    }
    if (n >= 8) {
        store_raw16(p, Raw16{{r.w[0], r.w[1], r.w[2], r.w[3]}});
        if constexpr (T == DT_F32)
            store_raw16(p + 16, Raw16{{r.w[4], r.w[5], r.w[6], r.w[7]}});
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e >= n)
            continue;
        if constexpr (T == DT_F32)
            ((uint32_t *)p)[e] = r.w[e];
        else
            ((uint16_t *)p)[e] = (uint16_t)(r.w[e / 2] >> (16 * (e % 2)));
    }
}

} // namespace dg
