// Products in 8-bit integers with scales for rows and columns: the kernels'
// arguments and launchers (host side in scaled_api.cpp).
#pragma once
#include "grouped.hpp"

namespace dg {

struct ScaledArgs {
    // of group 0; A and B int8, lda, ldb and sb in bytes; M is set per group
    GemmArgs g;
    const float *scale_a;      // null: ones (and where alpha is 0)
    const void *scale_b;       // null: ones
    const int32_t *offsets;    // null: one group of all rows
    int32_t groups, rows;
    int32_t scale_type;        // of scale_b
    int64_t stride_s, stride_bias;   // elements
    uint32_t tiles_n;
    // few rows whose codes the product makes itself: their type and leading
    // dimension in bytes
    const char *x;
    int64_t ldx;
    int32_t x_type;
};

// What a workgroup holds in registers while it makes the codes of few rows
// (make_codes): 16 elements per thread of each row.  That all rows together
// have no more is a choice (few_rows in scaled_api.cpp has the times).
constexpr int kFewRows = 4;
constexpr int64_t kFewElements = 8192;      // of all of them

// Tile of program `pid` of one matrix of `rows` rows: as find_group_tile of
// one group, without the lookup.
template <int BM, int G = 4>
__device__ __forceinline__ GroupTile matrix_tile(int32_t rows, uint32_t tiles_n, uint32_t pid)
{
    const uint32_t own = ((uint32_t)rows + (BM - 1)) / BM, P = own * tiles_n;
    GroupTile t{-1, 0, 0, 0, 0};
    if (pid >= P)
        return t;
    const uint32_t x = pid % kNumXcd, q = P / kNumXcd, r = P % kNumXcd;
    const uint32_t L = x * q + (x < r ? x : r) + pid / kNumXcd;
    const uint32_t band = L / (G * tiles_n), o = L - band * (G * tiles_n);
    const uint32_t left = own - band * G, h = left < G ? left : G;
    t.group = 0;
    t.rows = rows;
    t.col_tile = o / h;
    t.row_tile = band * G + (o - t.col_tile * h);
    return t;
}

template <int BM, int G = 4>
__device__ __forceinline__ GroupTile scaled_tile(const ScaledArgs &a)
{
    return a.offsets ? find_group_tile<BM, G>(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x)
                     : matrix_tile<BM, G>(a.rows, a.tiles_n, blockIdx.x);
}

// The argument block of one group's product, bytes as above.
__device__ __forceinline__ GemmArgs scaled_args(const ScaledArgs &a, int32_t e, int32_t start, int32_t len)
{
    GemmArgs g = a.g;
    g.M = len;
    g.A = (const char *)g.A + (int64_t)start * g.lda;
    g.B = (const char *)g.B + e * g.sb;
    g.C = (char *)g.C + (int64_t)start * g.ldc * (g.c_type == DT_F32 ? 4 : 2);
    if (g.bias)
        g.bias = (const char *)g.bias + e * a.stride_bias * (g.bias_type == DT_F32 ? 4 : 2);
    g.sa = g.sb = g.sc = 0;
    return g;
}

__device__ __forceinline__ const float *row_scales(const ScaledArgs &a, int32_t start)
{
    return a.scale_a ? a.scale_a + start : nullptr;
}
__device__ __forceinline__ const void *col_scales(const ScaledArgs &a, int32_t e)
{
    return a.scale_b ? (const char *)a.scale_b + e * a.stride_s * (a.scale_type == DT_F32 ? 4 : 2) : nullptr;
}

// 16 bytes of a row from any address (gfx950 loads them so).
struct Bytes16 { uint32_t w[4]; };

__device__ __forceinline__ Bytes16 load_bytes16(const int8_t *p)
{
    Bytes16 r;
    __builtin_memcpy(&r, p, 16);
    return r;
}

// Bytes k .. k + 15 of a row of K, zero from K on, and nothing read past K.
// Where K cuts them, the row's last 16 bytes are loaded and moved down.
__device__ __forceinline__ Bytes16 load_masked16(const int8_t *row, int64_t k, int64_t K)
{
    if (k + 16 <= K)
        return load_bytes16(row + k);
    if (k >= K)
        return Bytes16{};
    if (K < 16) {
        Bytes16 r{};
#pragma unroll
        for (int i = 0; i < 15; ++i)               // k is 0 then
            if (i < K)
                r.w[i / 4] |= (uint32_t)(uint8_t)row[i] << (8 * (i % 4));
        return r;
    }
    const Bytes16 end = load_bytes16(row + K - 16);
    const int by = 8 * (16 - (int)(K - k));        // bits to go: 8 .. 120
    uint64_t lo = end.w[0] | (uint64_t)end.w[1] << 32, hi = end.w[2] | (uint64_t)end.w[3] << 32;
    lo = by >= 64 ? hi >> (by - 64) : lo >> by | hi << (64 - by);
    hi = by >= 64 ? 0 : hi >> by;
    return Bytes16{{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)}};
}

// Launchers; each returns hipSuccess or the launch error.
hipError_t launch_scaled_stream(int32_t variant, const ScaledArgs &a, uint32_t programs, hipStream_t s);
// of x, up to kFewRows rows and kFewElements
hipError_t launch_scaled_few(int32_t variant, const ScaledArgs &a, uint32_t programs, hipStream_t s);
hipError_t launch_scaled_tile(int32_t variant, const ScaledArgs &a, uint32_t programs, hipStream_t s);

} // namespace dg
