// C ABI of the products over groups of rows and of the products with 4-bit
// weights: host-side validation (no HIP calls), choice of the kernel and
// launch.  Nothing is known of the groups' lengths here: the grid covers an
// upper bound of the tiles, and the choice goes by the mean length.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/densegemm.h"
#include "checks.hpp"
#include "grouped.hpp"

using namespace dg;

namespace {

constexpr int64_t kMaxGroups = 65536;
constexpr int64_t kMaxRows = INT32_MAX;
constexpr int kCus = 256;                // MI355X compute units

bool dtype_ok(int32_t t) { return t == DG_F32 || t == DG_BF16 || t == DG_F16; }
bool act_ok(int32_t a) { return a >= DG_ACT_NONE && a <= DG_ACT_GELU_TANH; }

// Bytes of `count` matrices of `rows` rows of `len` elements, `ld` apart,
// `stride` from one matrix to the next.
bool bytes_of(int64_t count, int64_t stride, int64_t rows, int64_t len, int64_t ld, int64_t es,
              int64_t *bytes)
{
    int64_t span, total;
    return matrix_span(DG_ROW_MAJOR, rows, len, ld, &span) &&
           batch_span(span, count, stride, &total) && mul_ok(total, es, bytes);
}

// Row tiles of a launch over groups of unknown lengths.
int64_t row_tiles(int64_t rows, int64_t groups, int64_t bm)
{
    return rows / bm + (groups < rows ? groups : rows);
}

// A grid of `a` x `b` workgroups of `threads` threads, if a launch can have
// it: below 2^32 threads, with the 128 workgroups that launch_grouped_mixed
// adds.  The kernels' 32-bit tile numbers are then far from their end.
bool grid_ok(int64_t a, int64_t b, int32_t threads, uint32_t *programs)
{
    int64_t p;
    if (!mul_ok(a, b, &p) || p > (int64_t)UINT32_MAX / threads - 128)
        return false;
    *programs = (uint32_t)p;
    return true;
}

// `chosen`, or where its grid is more than a launch can have the first of
// `table` (tiles in ascending order) with larger tiles and a grid that is
// not.  fits(k): k takes the problem and its grid can be launched; it sets
// the plan's programs.
template <typename K, size_t N, typename Fits>
const K *fitting_kernel(const K *chosen, const K *const (&table)[N], Fits &&fits)
{
    if (fits(*chosen))
        return chosen;
    for (const K *k : table)
        if (k->bm * k->bn > chosen->bm * chosen->bn && fits(*k))
            return k;
    return nullptr;
}

// ---- grouped products -------------------------------------------------------

struct Spans {
    int64_t a, b, c, bias, offsets;      // bytes
};

bool reads_ab(const dg_grouped_desc *d)
{
    return d->alpha != 0.0f && d->rows > 0 && (d->ragged == DG_RAGGED_K || d->K > 0);
}

bool is_noop(const dg_grouped_desc *d)
{
    return d->groups == 0 || d->N == 0 ||
           (d->ragged == DG_RAGGED_M ? d->rows == 0 : d->M == 0);
}

dg_status validate(const dg_grouped_desc *d, Spans *s)
{
    if (!d || d->struct_size != sizeof(dg_grouped_desc))
        return DG_ERROR_INVALID_VALUE;
    if (d->ragged != DG_RAGGED_M && d->ragged != DG_RAGGED_K)
        return DG_ERROR_INVALID_VALUE;
    const bool rk = d->ragged == DG_RAGGED_K;
    if (!dtype_ok(d->a_type) || !dtype_ok(d->b_type) || !dtype_ok(d->c_type) ||
        (d->b_order != DG_ROW_MAJOR && d->b_order != DG_COL_MAJOR) || !act_ok(d->act))
        return DG_ERROR_INVALID_VALUE;
    if (d->groups < 0 || d->rows < 0 || d->N < 0 || (rk ? d->M : d->K) < 0)
        return DG_ERROR_INVALID_VALUE;
    if (d->bias && !dtype_ok(d->bias_type))
        return DG_ERROR_INVALID_VALUE;
    const int64_t a_len = rk ? d->M : d->K;
    const int64_t b_len = rk || d->b_order == DG_ROW_MAJOR ? d->N : d->K;
    if (d->lda < 1 || d->ldb < 1 || d->ldc < 1 || d->lda < a_len || d->ldb < b_len ||
        d->ldc < d->N)
        return DG_ERROR_INVALID_VALUE;
    if ((rk ? d->stride_c : d->stride_b) < 0 || (d->bias && d->stride_bias < 0))
        return DG_ERROR_INVALID_VALUE;
    if (d->a_type != d->b_type || (d->a_type == DG_F32 && d->c_type != DG_F32))
        return DG_ERROR_NOT_SUPPORTED;
    if (d->groups > kMaxGroups || d->rows > kMaxRows)
        return DG_ERROR_NOT_SUPPORTED;
    if (rk && (d->b_order != DG_ROW_MAJOR || d->bias || d->act != DG_ACT_NONE))
        return DG_ERROR_NOT_SUPPORTED;
    const int64_t es = elem_size(d->a_type), cs = elem_size(d->c_type);
    s->offsets = (d->groups + 1) * 4;
    s->bias = 0;
    bool ok;
    if (rk) {
        ok = bytes_of(1, 0, d->rows, d->M, d->lda, es, &s->a) &&
             bytes_of(1, 0, d->rows, d->N, d->ldb, es, &s->b) &&
             bytes_of(d->groups, d->stride_c, d->M, d->N, d->ldc, cs, &s->c);
        int64_t one;
        if (ok && d->groups > 1 && d->M > 0 && d->N > 0 &&
            (!matrix_span(DG_ROW_MAJOR, d->M, d->N, d->ldc, &one) || d->stride_c < one))
            return DG_ERROR_INVALID_VALUE;       // C matrices overlap
    } else {
        const bool row = d->b_order == DG_ROW_MAJOR;
        ok = bytes_of(1, 0, d->rows, d->K, d->lda, es, &s->a) &&
             bytes_of(d->groups, d->stride_b, row ? d->K : d->N, row ? d->N : d->K, d->ldb, es,
                      &s->b) &&
             bytes_of(1, 0, d->rows, d->N, d->ldc, cs, &s->c);
        if (d->bias)
            ok = ok && bytes_of(d->groups, d->stride_bias, 1, d->N, d->N > 0 ? d->N : 1,
                                elem_size(d->bias_type), &s->bias);
    }
    return ok ? DG_SUCCESS : DG_ERROR_INVALID_VALUE;
}

using GroupedLaunch = hipError_t (*)(const GroupedArgs &, uint32_t, hipStream_t);

// A kernel of the grouped products: its tile, the threads of a workgroup (at
// most) and its launchers (null: not for this kind).
struct GroupedKernel {
    const char *name;
    int32_t bm, bn, threads;
    GroupedLaunch ragged_m, ragged_k;
};

hipError_t generic_m(const GroupedArgs &a, uint32_t p, hipStream_t s)
{
    return launch_grouped_generic(a, false, p, s);
}
hipError_t generic_k(const GroupedArgs &a, uint32_t p, hipStream_t s)
{
    return launch_grouped_generic(a, true, p, s);
}
template <int V>
hipError_t stream_m(const GroupedArgs &a, uint32_t p, hipStream_t s)
{
    return launch_grouped_stream(V, a, p, s);
}

hipError_t tile256_m(const GroupedArgs &a, uint32_t p, hipStream_t s)
{
    return a.g.ab_type == DT_F16 ? launch_grouped16_m256_f16(a, p, s)
                                 : launch_grouped16_m256_bf16(a, p, s);
}

const GroupedKernel kGeneric = {"generic", kGroupedGenericTile, kGroupedGenericTile, 256,
                                generic_m, generic_k};
const GroupedKernel kTile256 = {"mfma16_256x256", 256, 256, 256, tile256_m,
                                launch_grouped16_k256};
const GroupedKernel kTile128 = {"mfma16_128x128", 128, 128, 256, launch_grouped16_m128,
                                launch_grouped16_k128};
const GroupedKernel kTileF32 = {"mfma_f32_128x128", 128, 128, 256, launch_grouped_f32_m,
                                launch_grouped_f32_k};
const GroupedKernel kStream16x32 = {"stream_16x32", 16, 32, 512, stream_m<0>, nullptr};
const GroupedKernel kStream16x64 = {"stream_16x64", 16, 64, 512, stream_m<1>, nullptr};
const GroupedKernel kStream32x64 = {"stream_32x64", 32, 64, 512, stream_m<2>, nullptr};
const GroupedKernel *const kGrouped16[] = {&kStream16x32, &kStream16x64, &kStream32x64, &kTile128,
                                           &kTile256};
const GroupedKernel *const kGroupedF32[] = {&kStream16x32, &kStream16x64, &kStream32x64, &kTileF32};

// The kernel of `table` that DG_FORCE_GROUPED names (benchmarking and
// tests), or NULL.
template <typename K, size_t N>
const K *forced_kernel(const K *const (&table)[N])
{
    const char *want = getenv("DG_FORCE_GROUPED");
    for (const K *k : table)
        if (want && !strcmp(want, k->name))
            return k;
    return nullptr;
}

struct GroupedPlan {
    const GroupedKernel *kernel;
    uint32_t programs;
};

// The matrix-core kernels read whole 16-byte pieces of rows; the 16-bit
// tiles address a tile with 32-bit byte offsets.
bool mfma_ok(const dg_grouped_desc *d, const void *A, const void *B)
{
    const int64_t n = d->a_type == DG_F32 ? 4 : 8;
    return aligned_to(A, 16) && aligned_to(B, 16) && d->lda % n == 0 && d->ldb % n == 0 &&
           d->lda < (1 << 22) && d->ldb < (1 << 22) &&
           (d->ragged == DG_RAGGED_K || d->groups <= 1 || d->stride_b % n == 0);
}

// The kernel for a problem.  Group lengths are unknown; the mean stands for
// them, and half the groups are taken to end in one more tile.
//
// Ragged rows, by the mean rows of a group (us, MI355X, bf16; ranges span
// cards, orders of B, and weights in and out of the Infinity Cache):
//   up to 8 rows, the 16-row streaming kernels: 64 groups, 512 rows, 2048 x
//     2048: 98-101 against 98-118 on the 128 x 128 tile; 64 rows, 2048 x
//     1024: 28-36 against 33-52.  32 columns per workgroup where 64 would
//     make fewer than 512 workgroups (8 groups, 8 rows, 1024 x 1024: 3.6-5.5
//     against 5.0-7.3);
//   up to 16, the 32-row one: 1024 rows on those 64 groups 105-106 against
//     112-120 on 16 rows (and 102-115 on the tile), 4 groups, 64 rows, 4096 x
//     4096 25-34 against 32-43 and 29-51 on the tile;
//   fp32 keeps the 32-row one below 1024 tiles of 128 x 128 (1000 rows, 5
//     groups, 512 x 260: 9.2 against 62, and 8.8 and 10.5 on 16 rows x 32 and
//     64; 4096 rows, 16 groups, 2048 x 2048: 327-390 against 393-407, and
//     482 and 342 on 16 rows) and takes the tile above (8192 rows, 2048 x
//     4096: 1151-1166, on another card 1280, against 1228-1440);
//   above, 16 bits, a tile: 256 x 256 (with half-height tiles, see
//     grouped16.hpp) for groups of 128 rows and more, K from 768 and at
//     least 128 tiles, else 128 x 128 (8192 rows, 16 groups, 4096 x 4096:
//     305-316 against 390-418; 2000 rows, 16 groups, 4096 x 2048: 75-78
//     against 101-103; but 1000 rows, 4 groups, 4096 x 1024, 28 tiles: 61-74
//     against 33-51, and 6000 rows, 48 groups, 512 x 1024: 27-32 against
//     22-27).
// Ragged K: the 128 x 128 tile, whose other workgroups on a CU cover one's
// epilogue (16 groups of 2048 x 2048, 8192 rows: 99-102 against 100-112; 32
// of 512 x 1024: 22-24 against 24-29), unless the groups are long and 256 x
// 256 tiles fill the chip twice, so that long and short groups even out
// (16384 rows, 8 groups, 4096 x 4096: 484-505 against 521-585, 2048 x 2048:
// 136-167 against 142-185; but 8192 rows, 1024 x 2048, 256 tiles: 52-58
// against 45-52), or once with one group (4096 rows, 4096 x 4096: 112-120
// against 123-133).
const GroupedKernel *choose(const dg_grouped_desc *d, const void *A, const void *B)
{
    if (!mfma_ok(d, A, B))
        return &kGeneric;
    const bool rk = d->ragged == DG_RAGGED_K, f32 = d->a_type == DG_F32;
    if (const GroupedKernel *k = f32 ? forced_kernel(kGroupedF32) : forced_kernel(kGrouped16))
        if (rk ? k->ragged_k : k->ragged_m)
            return k;
    if (f32 && rk)
        return &kTileF32;
    const double mean = (double)d->rows / (double)d->groups;
    const double n256 = (double)ceil_div(d->N, 256);
    if (rk) {
        const double tiles = (double)d->groups * (double)ceil_div(d->M, 256) * n256;
        return mean >= 768 && tiles >= (d->groups > 1 ? 480 : 240) ? &kTile256 : &kTile128;
    }
    if (mean <= 8)
        return row_tiles(d->rows, d->groups, 16) * ceil_div(d->N, 64) < 512 ? &kStream16x32
                                                                            : &kStream16x64;
    if (mean <= 16)
        return &kStream32x64;
    if (f32)
        return row_tiles(d->rows, d->groups, 128) * ceil_div(d->N, 128) < 4 * kCus ? &kStream32x64
                                                                                   : &kTileF32;
    const double tiles = ((double)d->rows / 256 + 0.5 * (double)d->groups) * n256;
    return mean >= 128 && d->K >= 768 && tiles >= 128 ? &kTile256 : &kTile128;
}

dg_status make_plan(const dg_grouped_desc *d, const void *A, const void *B, GroupedPlan *p)
{
    const bool rk = d->ragged == DG_RAGGED_K;
    auto fits = [&](const GroupedKernel &k) {
        const int64_t tn = ceil_div(d->N, k.bn);
        const int64_t tm = rk ? ceil_div(d->M, k.bm) : row_tiles(d->rows, d->groups, k.bm);
        int64_t t;
        return (rk ? k.ragged_k : k.ragged_m) && mul_ok(tm, tn, &t) && t <= INT32_MAX &&
               grid_ok(t, rk ? d->groups : 1, k.threads, &p->programs);
    };
    const GroupedKernel *first = choose(d, A, B);
    if (first == &kGeneric)
        p->kernel = fits(kGeneric) ? &kGeneric : nullptr;
    else if (d->a_type == DG_F32)
        p->kernel = fitting_kernel(first, kGroupedF32, fits);
    else
        p->kernel = fitting_kernel(first, kGrouped16, fits);
    return p->kernel ? DG_SUCCESS : DG_ERROR_NOT_SUPPORTED;
}

// ---- 4-bit weights ----------------------------------------------------------

struct QSpans {
    int64_t a, q, scales, zeros, c, bias, offsets;
};

bool is_noop(const dg_qweight_desc *d) { return d->groups == 0 || d->N == 0 || d->M == 0; }
bool reads_ab(const dg_qweight_desc *d) { return d->alpha != 0.0f && d->K > 0; }

dg_status validate(const dg_qweight_desc *d, QSpans *s)
{
    if (!d || d->struct_size != sizeof(dg_qweight_desc))
        return DG_ERROR_INVALID_VALUE;
    if (!dtype_ok(d->a_type) || !dtype_ok(d->c_type) || !dtype_ok(d->scale_type) ||
        (d->bias && !dtype_ok(d->bias_type)) || !act_ok(d->act))
        return DG_ERROR_INVALID_VALUE;
    if (d->groups < 0 || d->M < 0 || d->N < 0 || d->K < 0 || d->group_size < 1)
        return DG_ERROR_INVALID_VALUE;
    const int64_t qlen = d->K / 2 + d->K % 2;
    const int64_t slen = d->K / d->group_size + (d->K % d->group_size != 0);
    if (d->lda < 1 || d->ldc < 1 || d->ldq < 1 || d->lds < 1 || d->lda < d->K || d->ldc < d->N ||
        d->ldq < qlen || d->lds < slen)
        return DG_ERROR_INVALID_VALUE;
    if (d->stride_q < 0 || d->stride_s < 0 || (d->bias && d->stride_bias < 0))
        return DG_ERROR_INVALID_VALUE;
    if (d->a_type == DG_F32 || d->group_size % 32 != 0)
        return DG_ERROR_NOT_SUPPORTED;
    if (d->groups > kMaxGroups || d->M > kMaxRows)
        return DG_ERROR_NOT_SUPPORTED;
    s->offsets = (d->groups + 1) * 4;
    s->bias = 0;
    const bool ok =
        bytes_of(1, 0, d->M, d->K, d->lda, 2, &s->a) &&
        bytes_of(d->groups, d->stride_q, d->N, qlen, d->ldq, 1, &s->q) &&
        bytes_of(d->groups, d->stride_s, d->N, slen, d->lds, elem_size(d->scale_type),
                 &s->scales) &&
        bytes_of(d->groups, d->stride_s, d->N, slen, d->lds, 1, &s->zeros) &&
        bytes_of(1, 0, d->M, d->N, d->ldc, elem_size(d->c_type), &s->c) &&
        (!d->bias || bytes_of(d->groups, d->stride_bias, 1, d->N, d->N > 0 ? d->N : 1,
                              elem_size(d->bias_type), &s->bias));
    return ok ? DG_SUCCESS : DG_ERROR_INVALID_VALUE;
}

using QweightLaunch = hipError_t (*)(const QweightArgs &, uint32_t, hipStream_t);

struct QweightKernel {
    const char *name;
    int32_t bm, bn;
    QweightLaunch launch;
};

template <int V>
hipError_t qrows(const QweightArgs &a, uint32_t p, hipStream_t s)
{
    return launch_qweight_rows(V, a, p, s);
}
const QweightKernel kQGeneric = {"generic", kGroupedGenericTile, kGroupedGenericTile,
                                 launch_qweight_generic};
const QweightKernel kQ16x16 = {"qstream_16x16", 16, 16, qrows<0>};
const QweightKernel kQ16x32 = {"qstream_16x32", 16, 32, qrows<1>};
const QweightKernel kQ16x64 = {"qstream_16x64", 16, 64, qrows<2>};
const QweightKernel kQ32x32 = {"qstream_32x32", 32, 32, qrows<3>};
const QweightKernel kQ32x64 = {"qstream_32x64", 32, 64, qrows<4>};
const QweightKernel kQ32x128 = {"qstream_32x128", 32, 128, qrows<5>};
const QweightKernel kQ64x256 = {"qtile_64x256", 64, 256, launch_qweight_tile};
// group sizes that are multiples of 128 only
const QweightKernel kQ64x512 = {"qtile_64x512", 64, 512, launch_qweight_wide_tile};
const QweightKernel *const kQweight[] = {&kQ16x16, &kQ16x32,  &kQ16x64,  &kQ32x32,
                                         &kQ32x64, &kQ32x128, &kQ64x256, &kQ64x512};
constexpr int32_t kQweightThreads = 512;   // of the matrix-core kernels

struct QweightPlan {
    const QweightKernel *kernel;
    uint32_t programs;
};

// The matrix-core kernels read A and Q in whole 16-byte pieces and K in
// whole steps of 32, and address a tile (up to 64 rows, 512 columns) with
// 32-bit byte offsets.
bool qstream_ok(const dg_qweight_desc *d, const void *A, const void *Q)
{
    return aligned_to(A, 16) && aligned_to(Q, 16) && d->lda % 8 == 0 && d->ldq % 16 == 0 &&
           (d->groups <= 1 || d->stride_q % 16 == 0) && d->K % 32 == 0 && d->lda < (1 << 24) &&
           d->ldq < (1 << 23) && d->lds < (1 << 21);
}

// One group's rows, with or without offsets, make at most ceil(M / bm) tiles.
int64_t row_tiles(const dg_qweight_desc *d, const QweightKernel &k)
{
    return d->groups > 1 ? row_tiles(d->M, d->groups, k.bm) : ceil_div(d->M, k.bm);
}

// Times a tile's place on the chip is taken: one workgroup per CU.
int64_t chip_passes(int64_t row_tiles, int64_t n, int64_t bn)
{
    const int64_t per_pass = 256, cols = ceil_div(n, bn);
    if (row_tiles > INT64_MAX / cols)
        return INT64_MAX / 8;       // not reached for a grid that can be launched
    return ceil_div(row_tiles * cols, per_pass);
}

// From 256 rows a group, if 64 x 256 tiles fill the chip, the tile (us, 4096
// x 4096, bf16, group size 128): 1024 rows 49 against 63 on 32 x 128, 2048
// rows 97 against 124; 256 rows of 16384 x 4096 49 against 63 (of 14336 x
// 4096, 224 tiles, which the rule leaves to 32 x 128, 48 against 60); where
// they do not, it loses (256 rows of 4096 x 4096: 46 against 21).  A pass of
// 64 x 512 tiles over the chip takes 79-86 us where one of 64 x 256 takes
// 46-49 (four column blocks per wavefront read a row of A once, but hold 256
// registers), so they are taken where they need less than 3/5 of the passes:
// 2048 rows 86 against 97, of 8192 x 8192 329 against 365; 1024 rows 81
// against 49.
// Else 32 rows where a group has more than 16, and the widest workgroup
// (each reads A once) that still makes 512 of them for up to 4 rows, 256
// for more, where A's traffic counts:
//   1 row,   4096 x 4096: 5.4 on 16 columns, 6.9 on 32, 10.4 on 64;
//            16384 x 4096: 12.5, 10.2, 11.8;  8192 x 8192: 10.5, 12.6, 19.1
//   16 rows, 4096 x 4096: 6.1-7.2, 7.8-9.2, 11.1-11.8;  16384 x 4096:
//     15.9-18.6, 11.6-14.0, 12.0-13.3
//   64 rows, 16384 x 4096: 30 on 16 x 64, 30 on 32 x 32, 25 on 32 x 64, 21 on
//     32 x 128
//   512 rows, 4096 x 4096: 55 on 32 x 32, 45 on 32 x 64, 33 on 32 x 128 (two
//     column blocks per wavefront halve its reads of A from LDS)
const QweightKernel *choose(const dg_qweight_desc *d, const void *A, const void *Q)
{
    if (!qstream_ok(d, A, Q))
        return &kQGeneric;
    const bool wide = d->group_size % 128 == 0;
    if (const QweightKernel *k = forced_kernel(kQweight))
        if (k != &kQ64x512 || wide)
            return k;
    const int64_t rows = d->M / d->groups;
    const int64_t want = rows <= 4 ? 512 : 256;
    for (const QweightKernel *k : {&kQ64x256, &kQ32x128, &kQ32x64, &kQ32x32, &kQ16x64, &kQ16x32}) {
        const bool rows_fit = k->bm == 64 ? rows >= 256 : k->bm == 32 ? rows > 16 : k->bm == 16;
        if (!rows_fit || ceil_div(d->N, k->bn) < ceil_div(want, row_tiles(d, *k)))
            continue;
        const int64_t rt = row_tiles(d, *k);
        const bool fewer = 5 * chip_passes(rt, d->N, 512) < 3 * chip_passes(rt, d->N, 256);
        return k == &kQ64x256 && wide && fewer ? &kQ64x512 : k;
    }
    return &kQ16x16;
}

dg_status make_plan(const dg_qweight_desc *d, const void *A, const void *Q, QweightPlan *p)
{
    auto fits = [&](const QweightKernel &k) {
        return (&k != &kQ64x512 || d->group_size % 128 == 0) &&
               grid_ok(row_tiles(d, k), ceil_div(d->N, k.bn),
                       &k == &kQGeneric ? 256 : kQweightThreads, &p->programs);
    };
    const QweightKernel *first = choose(d, A, Q);
    if (first == &kQGeneric)
        p->kernel = fits(kQGeneric) ? &kQGeneric : nullptr;
    else
        p->kernel = fitting_kernel(first, kQweight, fits);
    return p->kernel ? DG_SUCCESS : DG_ERROR_NOT_SUPPORTED;
}

} // namespace

extern "C" {

dg_status dg_gemm_grouped(const dg_grouped_desc *d, const void *A, const void *B, void *C,
                          const int32_t *offsets, void *stream)
{
    Spans sp;
    dg_status st = validate(d, &sp);
    if (st != DG_SUCCESS)
        return st;
    if (is_noop(d))
        return DG_SUCCESS;
    if (!C || !offsets || (reads_ab(d) && (!A || !B)))
        return DG_ERROR_INVALID_VALUE;
    if (!aligned_to(A, elem_size(d->a_type)) || !aligned_to(B, elem_size(d->b_type)) ||
        !aligned_to(C, elem_size(d->c_type)) || !aligned_to(offsets, 4) ||
        (d->bias && !aligned_to(d->bias, elem_size(d->bias_type))))
        return DG_ERROR_INVALID_VALUE;
    if ((reads_ab(d) && (ranges_overlap(C, sp.c, A, sp.a) || ranges_overlap(C, sp.c, B, sp.b))) ||
        ranges_overlap(C, sp.c, d->bias, sp.bias) || ranges_overlap(C, sp.c, offsets, sp.offsets))
        return DG_ERROR_INVALID_VALUE;
    GroupedPlan p;
    st = make_plan(d, A, B, &p);
    if (st != DG_SUCCESS)
        return st;
    const bool rk = d->ragged == DG_RAGGED_K;
    GroupedArgs a;
    memset(&a, 0, sizeof a);
    a.g.A = A;
    a.g.B = B;
    a.g.C = C;
    a.g.bias = d->bias;
    a.g.M = rk ? d->M : 0;
    a.g.N = d->N;
    a.g.K = rk ? 0 : d->K;
    a.g.lda = d->lda;
    a.g.ldb = d->ldb;
    a.g.ldc = d->ldc;
    a.g.sb = rk ? 0 : d->stride_b;
    a.g.sc = rk ? d->stride_c : 0;
    a.g.alpha = d->alpha;
    a.g.beta = d->beta;
    a.g.a_col = rk;
    a.g.b_col = d->b_order == DG_COL_MAJOR;
    a.g.c_type = d->c_type;
    a.g.bias_type = d->bias_type;
    a.g.act = d->act;
    a.g.ab_type = d->a_type;
    a.offsets = offsets;
    a.groups = (int32_t)d->groups;
    a.rows = (int32_t)d->rows;
    a.stride_bias = d->stride_bias;
    a.tiles_n = (uint32_t)ceil_div(d->N, p.kernel->bn);
    a.tiles = rk ? (uint32_t)(ceil_div(d->M, p.kernel->bm) * a.tiles_n) : 0;
    const hipError_t err =
        (rk ? p.kernel->ragged_k : p.kernel->ragged_m)(a, p.programs, (hipStream_t)stream);
    return err == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_gemm_grouped_describe(const dg_grouped_desc *d, char *buf, size_t len)
{
    if (!buf || len == 0)
        return DG_ERROR_INVALID_VALUE;
    Spans sp;
    dg_status st = validate(d, &sp);
    if (st != DG_SUCCESS)
        return st;
    if (is_noop(d)) {
        snprintf(buf, len, "noop");
        return DG_SUCCESS;
    }
    GroupedPlan p;
    st = make_plan(d, nullptr, nullptr, &p);
    if (st == DG_SUCCESS)
        snprintf(buf, len, "kernel=%s bm=%d bn=%d programs=%u", p.kernel->name, p.kernel->bm,
                 p.kernel->bn, p.programs);
    return st;
}

dg_status dg_gemm_qweight(const dg_qweight_desc *d, const void *A, const void *Q,
                          const void *scales, const void *zeros, void *C, const int32_t *offsets,
                          void *stream)
{
    QSpans sp;
    dg_status st = validate(d, &sp);
    if (st != DG_SUCCESS)
        return st;
    if (!offsets && d->groups > 1)
        return DG_ERROR_INVALID_VALUE;
    if (is_noop(d))
        return DG_SUCCESS;
    if (!C || (reads_ab(d) && (!A || !Q || !scales)))
        return DG_ERROR_INVALID_VALUE;
    if (!aligned_to(A, 2) || !aligned_to(scales, elem_size(d->scale_type)) ||
        !aligned_to(C, elem_size(d->c_type)) || !aligned_to(offsets, 4) ||
        (d->bias && !aligned_to(d->bias, elem_size(d->bias_type))))
        return DG_ERROR_INVALID_VALUE;
    if ((reads_ab(d) &&
         (ranges_overlap(C, sp.c, A, sp.a) || ranges_overlap(C, sp.c, Q, sp.q) ||
          ranges_overlap(C, sp.c, scales, sp.scales) || ranges_overlap(C, sp.c, zeros, sp.zeros))) ||
        ranges_overlap(C, sp.c, d->bias, sp.bias) || ranges_overlap(C, sp.c, offsets, sp.offsets))
        return DG_ERROR_INVALID_VALUE;
    QweightPlan p;
    st = make_plan(d, A, Q, &p);
    if (st != DG_SUCCESS)
        return st;
    QweightArgs a;
    memset(&a, 0, sizeof a);
    a.A = A;
    a.Q = (const uint8_t *)Q;
    a.scales = scales;
    a.zeros = (const uint8_t *)zeros;
    a.C = C;
    a.bias = d->bias;
    a.offsets = offsets;
    a.groups = (int32_t)d->groups;
    a.rows = (int32_t)d->M;
    a.N = d->N;
    a.K = d->K;
    a.group_size = d->group_size;
    a.lda = d->lda;
    a.ldc = d->ldc;
    a.ldq = d->ldq;
    a.lds = d->lds;
    a.stride_q = d->stride_q;
    a.stride_s = d->stride_s;
    a.stride_bias = d->stride_bias;
    a.alpha = d->alpha;
    a.beta = d->beta;
    a.a_type = d->a_type;
    a.c_type = d->c_type;
    a.scale_type = d->scale_type;
    a.bias_type = d->bias_type;
    a.act = d->act;
    a.tiles_n = (uint32_t)ceil_div(d->N, p.kernel->bn);
    const hipError_t err = p.kernel->launch(a, p.programs, (hipStream_t)stream);
    return err == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_gemm_qweight_describe(const dg_qweight_desc *d, char *buf, size_t len)
{
    if (!buf || len == 0)
        return DG_ERROR_INVALID_VALUE;
    QSpans sp;
    dg_status st = validate(d, &sp);
    if (st != DG_SUCCESS)
        return st;
    if (is_noop(d)) {
        snprintf(buf, len, "noop");
        return DG_SUCCESS;
    }
    QweightPlan p;
    st = make_plan(d, nullptr, nullptr, &p);
    if (st == DG_SUCCESS)
        snprintf(buf, len, "kernel=%s bm=%d bn=%d programs=%u", p.kernel->name, p.kernel->bm,
                 p.kernel->bn, p.programs);
    return st;
}

} // extern "C"
