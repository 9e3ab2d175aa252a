// C ABI of the products in 8-bit integers: host-side validation (no HIP
// calls), choice of the kernel and launch.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/densegemm.h"
#include "checks.hpp"
#include "scaled.hpp"
#include "tokens.hpp"

using namespace dg;

namespace {

constexpr int64_t kMaxGroups = 65536;
constexpr int64_t kMaxK = 131071;        // 2^14 each: below 2^31

bool float_type(int32_t t) { return t == DG_F32 || t == DG_BF16 || t == DG_F16; }

int64_t a_bytes(const dg_scaled_desc *d) { return d->a_type == DG_I8 ? 1 : elem_size(d->a_type); }

// Bytes of `count` matrices of `rows` rows of `len` elements, `ld` apart,
// `stride` from one matrix to the next.
bool bytes_of(int64_t count, int64_t stride, int64_t rows, int64_t len, int64_t ld, int64_t es,
              int64_t *bytes)
{
    int64_t span, total;
    return matrix_span(DG_ROW_MAJOR, rows, len, ld, &span) &&
           batch_span(span, count, stride, &total) && mul_ok(total, es, bytes);
}

struct Spans {
    int64_t a, sa, b, sb, c, bias, offsets;      // bytes
    int64_t codes, workspace;                    // of a float A
};

bool is_noop(const dg_scaled_desc *d) { return d->groups == 0 || d->N == 0 || d->M == 0; }
bool reads_ab(const dg_scaled_desc *d) { return d->alpha != 0.0f && d->K > 0; }

// Few float rows, whose codes every workgroup of the product makes itself: no
// workspace and no second launch.  A 1 x 4096 x 4096 call takes the host 7.0 us
// instead of 11.8.  On the GPU, in a graph, us against those of two launches,
// rows x columns x K, up to the limits: 1 x 4096 x 4096 8.2 and 9.6, 1 x 4096 x
// 8192 11.9 and 14.7, 1 x 16384 x 8192 29.7 and 31.7, 2 x 4096 x 4096 9.1 and
// 9.5, 2 x 16384 x 4096 18.5 and 18.3; but 4 x 4096 x 2048 8.9 and 7.5, 4 x 16384
// x 2048 14.7 and 12.7: of more than two rows only the shorter call wins.  Beyond
// 8192 elements of one row a thread would hold more than 16; of all rows
// together two launches win (4 x 16384 x 8192 35.8 against 31.8), and so they do
// in a layer of experts (64 rows, 64 groups, 2048 x 2048 44.8 us a call against
// 35.6).
bool few_rows(const dg_scaled_desc *d)
{
    return d->a_type != DG_I8 && d->groups == 1 && d->M <= DG_SCALED_FEW_ROWS && d->M * d->K <= DG_SCALED_FEW_ELEMENTS;
}
static_assert(DG_SCALED_FEW_ROWS == kFewRows && DG_SCALED_FEW_ELEMENTS == kFewElements, "as the kernel has it");

// Leading dimension of the codes made of a float A: rows on 16 bytes.
int64_t codes_ld(const dg_scaled_desc *d) { return d->K > 0 ? ceil_div(d->K, 16) * 16 : 16; }

dg_status validate(const dg_scaled_desc *d, Spans *s)
{
    if (!d || d->struct_size != sizeof(dg_scaled_desc))
        return DG_ERROR_INVALID_VALUE;
    if ((!float_type(d->a_type) && d->a_type != DG_I8) || !float_type(d->c_type) ||
        !float_type(d->scale_type) || (d->bias && !float_type(d->bias_type)) ||
        d->act < DG_ACT_NONE || d->act > DG_ACT_GELU_TANH)
        return DG_ERROR_INVALID_VALUE;
    if (d->groups < 0 || d->M < 0 || d->N < 0 || d->K < 0 || d->lda < 1 || d->ldb < 1 || d->ldc < 1 ||
        d->lda < d->K || d->ldb < d->K || d->ldc < d->N || d->stride_b < 0 || d->stride_s < 0 ||
        (d->bias && d->stride_bias < 0))
        return DG_ERROR_INVALID_VALUE;
    if (d->groups > kMaxGroups || d->M > INT32_MAX || d->K > kMaxK)
        return DG_ERROR_NOT_SUPPORTED;
    s->offsets = (d->groups + 1) * 4;
    s->bias = 0;
    s->sa = d->M * 4;
    const int64_t n_ld = d->N > 0 ? d->N : 1;
    const bool ok =
        bytes_of(1, 0, d->M, d->K, d->lda, a_bytes(d), &s->a) &&
        bytes_of(d->groups, d->stride_b, d->N, d->K, d->ldb, 1, &s->b) &&
        bytes_of(d->groups, d->stride_s, 1, d->N, n_ld, elem_size(d->scale_type), &s->sb) &&
        bytes_of(1, 0, d->M, d->N, d->ldc, elem_size(d->c_type), &s->c) &&
        (!d->bias || bytes_of(d->groups, d->stride_bias, 1, d->N, n_ld, elem_size(d->bias_type), &s->bias));
    const bool made = d->a_type != DG_I8 && !few_rows(d);
    s->codes = made ? d->M * codes_ld(d) : 0;                        // below 2^31 * 2^18
    s->workspace = made ? s->codes + s->sa : 0;
    return ok ? DG_SUCCESS : DG_ERROR_INVALID_VALUE;
}

using ScaledLaunch = hipError_t (*)(const ScaledArgs &, uint32_t, hipStream_t);

struct ScaledKernel {
    const char *name;
    int32_t bm, bn, threads;
    bool any_alignment;
    ScaledLaunch launch;
    ScaledLaunch few;          // of few float rows, whose codes it makes itself
};

template <int V>
hipError_t stream_kernel(const ScaledArgs &a, uint32_t p, hipStream_t s) { return launch_scaled_stream(V, a, p, s); }
template <int V>
hipError_t tile_kernel(const ScaledArgs &a, uint32_t p, hipStream_t s) { return launch_scaled_tile(V, a, p, s); }

template <int V>
hipError_t few_kernel(const ScaledArgs &a, uint32_t p, hipStream_t s) { return launch_scaled_few(V, a, p, s); }

const ScaledKernel kS16x16 = {"i8_stream_16x16", 16, 16, 512, true, stream_kernel<0>, few_kernel<0>};
const ScaledKernel kS16x32 = {"i8_stream_16x32", 16, 32, 512, true, stream_kernel<1>, few_kernel<1>};
const ScaledKernel kS16x32short = {"i8_stream_16x32_short", 16, 32, 256, true, stream_kernel<2>, nullptr};
const ScaledKernel kS16x64 = {"i8_stream_16x64", 16, 64, 512, true, stream_kernel<3>, few_kernel<2>};
const ScaledKernel kS32x32 = {"i8_stream_32x32", 32, 32, 512, true, stream_kernel<4>, nullptr};
const ScaledKernel kAny64 = {"i8_any_64x128", 64, 128, 512, true, tile_kernel<0>, nullptr};
const ScaledKernel kAny128 = {"i8_any_128x128", 128, 128, 512, true, tile_kernel<1>, nullptr};
const ScaledKernel kT64 = {"i8_tile_64x128", 64, 128, 512, false, tile_kernel<2>, nullptr};
const ScaledKernel kT128deep = {"i8_tile_128x128_deep", 128, 128, 512, false, tile_kernel<3>, nullptr};
const ScaledKernel kT128 = {"i8_tile_128x128", 128, 128, 512, false, tile_kernel<4>, nullptr};
const ScaledKernel kT256 = {"i8_tile_256x256", 256, 256, 512, false, tile_kernel<5>, nullptr};
const ScaledKernel *const kKernels[] = {&kS16x16, &kS16x32short, &kS16x32, &kS16x64, &kS32x32,
                                        &kAny64, &kT64, &kAny128, &kT128deep, &kT128, &kT256};

struct ScaledPlan {
    const ScaledKernel *kernel;
    uint32_t programs;
};

int64_t row_tiles(const dg_scaled_desc *d, int64_t bm)
{
    return d->groups > 1 ? d->M / bm + (d->groups < d->M ? d->groups : d->M) : ceil_div(d->M, bm);
}

// The tiles read whole 16-byte pieces and pairs of k, and address a tile
// with 32-bit byte offsets.
bool tile_ok(const dg_scaled_desc *d, const void *A, const void *B)
{
    const bool own = d->a_type != DG_I8;          // codes of the workspace
    return (own || (aligned_to(A, 16) && d->lda % 16 == 0 && d->lda < (1 << 23))) && aligned_to(B, 16) &&
           d->ldb % 16 == 0 && d->ldb < (1 << 23) && (d->groups <= 1 || d->stride_b % 16 == 0) && d->K % 2 == 0;
}

// Tiles of bm x bn that a launch has to do, about: group lengths are unknown,
// and half the groups are taken to end in one more tile.
double expected_tiles(const dg_scaled_desc *d, int64_t bm, int64_t bn)
{
    const double rt = d->groups > 1 ? (double)d->M / (double)bm + 0.5 * (double)d->groups
                                    : (double)ceil_div(d->M, bm);
    return rt * (double)ceil_div(d->N, bn);
}

// The kernel for a problem, by the mean rows of a group (us, MI355X, int8 in,
// bf16 out, B from memory; M x N x K):
//   up to 16 (8 with groups), the 16-row streaming kernels.  16 columns where
//     32 would make fewer than 160 workgroups (1 x 4096 x 4096 6.1 against
//     7.7, and 11.2 on 64; 1 x 6000 x 4096 8.4 against 7.7); four wavefronts
//     instead of eight on 32 for K up to 2048 (64 rows, 64 groups, 2048 x
//     2048 25.2 against 28; 2048 x 1024 16.8 against 18.5; but 16 x 8192 x 8192
//     16.3 against 15.8), 64 columns from 256 workgroups of them with one
//     matrix and longer K (13 x 16384 x 8192 26.4 against 28.1, and 31.6 on
//     16);
//   one matrix, up to 32 rows: 16 x 32 while that is one workgroup per
//     compute unit (32 x 4096 x 4096 9.3 against 11.3 on 32 x 32);
//   then 32 x 32 while that is: 64 x 4096 x 4096 11.5 against 12.9 on 64 x 128;
//     64 x 8192 x 4096 19.5 against 15.9; with groups up to 16 rows, unless
//     128 x 128 tiles fill the chip twice (100 rows, 8 groups, 4096 x 4096 33
//     against 36; 1024 rows, 64 groups, 2048 x 2048 80 against 57.6, and 74 on
//     16 x 64);
//   rings of four stages with one workgroup per compute unit up to 256 tiles,
//     of 64 x 128 (256 x 4096 x 4096 13.5 against 17.6 on 128 x 128; 512 x 2048 x
//     8192 21.3 and 29; 300 rows, 16 groups, 1024 x 2048 11.8 and 13.9; 1024 x
//     4096 x 4096, 512 of them, 26.9 and 21.5), then of 128 x 128 (27.0 with two
//     stages, 29.3 on 256 x 256);
//   128 x 128 with two stages and two workgroups (2000 rows, 16 groups, 4096 x
//     2048 46.2 against 47.4 with four and 51.7);
//   256 x 256, cut in halves where that saves a wave, from half a chip of
//     them, with groups of 256 rows from a whole chip (2048 x 4096 x 4096 34.6
//     against 36.2 on 128 x 128; 4096 x 4096 x 4096 57 against 70; 8192 rows,
//     16 groups, 4096 x 4096 157 against 181, with bias and erf GELU 177 and
//     198; of 8192 rows, 8 groups, 1024 x 4096, 144 of them, the lengths decide:
//     61 against 59 with some, 48 against 55 with others).
// Off the 16-byte grid, or with odd K: the same streaming kernels, then tiles
// filled through registers, of 64 x 128 up to one per compute unit (64 x 4097 x
// 1001 11.8 against 15.1 on 128 x 128, and 17 on 32 x 64 streamed; 300 x 4096 x
// 4096 24.7 and 32.6), then of 128 x 128 (700 x 4097 x 1001 16.1 against 17.5;
// 2048 x 4096 x 4096 61 against 88).
const ScaledKernel *choose(const dg_scaled_desc *d, bool tile)
{
    if (few_rows(d) && reads_ab(d)) {
        const char *want = getenv("DG_FORCE_GROUPED");
        for (const ScaledKernel *k : {&kS16x16, &kS16x32, &kS16x64})
            if (want && !strcmp(want, k->name))
                return k;
        return d->N >= 256 * 64 && d->K > 2048 ? &kS16x64 : ceil_div(d->N, 32) < 160 ? &kS16x16 : &kS16x32;
    }
    if (const char *want = getenv("DG_FORCE_GROUPED"))         // benchmarking and tests
        for (const ScaledKernel *k : kKernels)
            if (!strcmp(want, k->name) && (k->any_alignment || tile))
                return k;
    const bool groups = d->groups > 1;
    const double mean = (double)d->M / (double)d->groups;
    if (mean <= (groups ? 8 : 16)) {
        const int64_t rt = row_tiles(d, 16);
        if (!groups && d->N >= 256 * 64 && d->K > 2048)
            return &kS16x64;
        return rt * ceil_div(d->N, 32) < 160 ? &kS16x16 : d->K > 2048 ? &kS16x32 : &kS16x32short;
    }
    if (!groups && mean <= 32 && expected_tiles(d, 16, 32) <= 256)
        return d->K > 2048 ? &kS16x32 : &kS16x32short;
    const double t64 = expected_tiles(d, 64, 128), t128 = expected_tiles(d, 128, 128), t256 = expected_tiles(d, 256, 256);
    if (groups ? mean <= 16 && t128 <= 512 : expected_tiles(d, 32, 32) <= 256)
        return &kS32x32;
    if (!tile)
        return t64 <= 256 ? &kAny64 : &kAny128;
    if (t64 <= 256)
        return &kT64;
    if (groups ? mean >= 256 && t256 >= 256 : t256 >= 128)
        return &kT256;
    return t128 <= 256 ? &kT128deep : &kT128;
}

dg_status make_plan(const dg_scaled_desc *d, const void *A, const void *B, ScaledPlan *p)
{
    const bool tile = tile_ok(d, A, B);
    auto fits = [&](const ScaledKernel &k) {
        int64_t n;
        if ((!k.any_alignment && !tile) || (few_rows(d) && reads_ab(d) && !k.few) || !mul_ok(row_tiles(d, k.bm), ceil_div(d->N, k.bn), &n) ||
            n > (int64_t)UINT32_MAX / k.threads - 128)      // launch_mixed adds 128
            return false;
        p->programs = (uint32_t)n;
        return true;
    };
    p->kernel = choose(d, tile);
    if (fits(*p->kernel))
        return DG_SUCCESS;
    for (const ScaledKernel *k : kKernels)         // the next larger tile that a launch can have
        if (k->bm * k->bn > p->kernel->bm * p->kernel->bn && fits(*k)) {
            p->kernel = k;
            return DG_SUCCESS;
        }
    return DG_ERROR_NOT_SUPPORTED;
}

} // namespace

extern "C" {

dg_status dg_gemm_scaled_workspace_size(const dg_scaled_desc *d, size_t *bytes)
{
    Spans sp;
    const dg_status st = bytes ? validate(d, &sp) : DG_ERROR_INVALID_VALUE;
    if (st == DG_SUCCESS)
        *bytes = is_noop(d) || !reads_ab(d) ? 0 : (size_t)sp.workspace;
    return st;
}

dg_status dg_gemm_scaled(const dg_scaled_desc *d, const void *A, const float *scale_a, const int8_t *B,
                         const void *scale_b, void *C, const int32_t *offsets, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    Spans sp;
    dg_status st = validate(d, &sp);
    if (st != DG_SUCCESS)
        return st;
    const bool reads = reads_ab(d), few = few_rows(d) && reads, make = d->a_type != DG_I8 && reads && !few;
    if ((!offsets && d->groups > 1) || (d->a_type != DG_I8 && scale_a))
        return DG_ERROR_INVALID_VALUE;
    if (is_noop(d))
        return DG_SUCCESS;
    if (!C || (reads && (!A || !B)))
        return DG_ERROR_INVALID_VALUE;
    if (!aligned_to(A, a_bytes(d)) || !aligned_to(scale_a, 4) || !aligned_to(scale_b, elem_size(d->scale_type)) ||
        !aligned_to(C, elem_size(d->c_type)) || !aligned_to(offsets, 4) || !aligned_to(workspace, 16) ||
        (d->bias && !aligned_to(d->bias, elem_size(d->bias_type))))
        return DG_ERROR_INVALID_VALUE;
    if (make && (!workspace || workspace_bytes < (size_t)sp.workspace))
        return DG_ERROR_INSUFFICIENT_WORKSPACE;
    const struct { const void *p; int64_t n; } others[] = {
        {A, reads ? sp.a : 0}, {B, reads ? sp.b : 0}, {scale_a, d->alpha != 0.0f ? sp.sa : 0},
        {scale_b, d->alpha != 0.0f ? sp.sb : 0}, {d->bias, sp.bias}, {offsets, sp.offsets}};
    for (const auto &o : others)
        if (ranges_overlap(C, sp.c, o.p, o.n) || (make && ranges_overlap(workspace, sp.workspace, o.p, o.n)))
            return DG_ERROR_INVALID_VALUE;
    if (make && ranges_overlap(workspace, sp.workspace, C, sp.c))
        return DG_ERROR_INVALID_VALUE;
    ScaledPlan p;
    st = make_plan(d, A, B, &p);
    if (st != DG_SUCCESS)
        return st;

    ScaledArgs a;
    memset(&a, 0, sizeof a);
    a.g.A = make ? workspace : A;
    a.g.B = B;
    a.g.C = C;
    a.g.bias = d->bias;
    a.g.N = d->N;
    a.g.K = reads ? d->K : 0;
    a.g.lda = make ? codes_ld(d) : d->lda;
    a.g.ldb = d->ldb;
    a.g.ldc = d->ldc;
    a.g.sb = d->stride_b;
    a.g.alpha = d->alpha;
    a.g.beta = d->beta;
    a.g.c_type = d->c_type;
    a.g.bias_type = d->bias_type;
    a.g.act = d->act;
    a.g.ab_type = DT_I8;
    if (d->alpha != 0.0f) {
        a.scale_a = make ? (const float *)((char *)workspace + sp.codes) : scale_a;
        a.scale_b = scale_b;
    }
    a.offsets = offsets;
    a.groups = (int32_t)d->groups;
    a.rows = (int32_t)d->M;
    a.scale_type = d->scale_type;
    a.stride_s = d->stride_s;
    a.stride_bias = d->stride_bias;
    a.tiles_n = (uint32_t)ceil_div(d->N, p.kernel->bn);
    if (make) {
        QuantizeArgs q;
        memset(&q, 0, sizeof q);
        q.x = (const char *)A;
        q.q = (int8_t *)workspace;
        q.scales = (float *)((char *)workspace + sp.codes);
        q.ldx = d->lda * a_bytes(d);
        q.ldq = codes_ld(d);
        q.tokens = d->M;
        q.width = d->K;
        q.x_type = d->a_type;
        if (launch_quantize(q, (hipStream_t)stream) != hipSuccess)
            return DG_ERROR_LAUNCH;
    }
    if (few) {
        a.x = (const char *)A;
        a.ldx = d->lda * a_bytes(d);
        a.x_type = d->a_type;
    }
    const hipError_t err = (few ? p.kernel->few : p.kernel->launch)(a, p.programs, (hipStream_t)stream);
    return err == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_gemm_scaled_describe(const dg_scaled_desc *d, char *buf, size_t len)
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
    ScaledPlan p;
    st = make_plan(d, nullptr, nullptr, &p);
    if (st == DG_SUCCESS)
        snprintf(buf, len, "kernel=%s bm=%d bn=%d programs=%u", p.kernel->name, p.kernel->bm, p.kernel->bn,
                 p.programs);
    return st;
}

} // extern "C"
