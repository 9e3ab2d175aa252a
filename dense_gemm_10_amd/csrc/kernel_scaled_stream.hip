// 8-bit products with few rows per group, and of operands of any alignment.
//
// As in stream.hpp, a workgroup owns 16 FM rows x 16 FN columns and its KW
// wavefronts take the steps of 128 k in turn; A and B go from memory into
// MFMA operand registers, 16 bytes of a row per lane, by loads that need no
// alignment.  K's last part is masked in A, whose zeros make B's bytes there
// count for nothing.  The wavefronts' integer sums meet in LDS, are added,
// and take scales and epilogue once.
//
// Measured (MI355X, kernel times, operands the same from call to call): 13 rows
// of 16384 x 8192 22.2 us, 135 MB read, 6.1 TB/s; 64 rows on 64 experts of 2048 x
// 2048 25.2 us, 164 MB read, 6.5 TB/s; one bf16 row through 4096 x 4096, its codes
// included, 6.4 us, 17 MB, 2.7 TB/s.
#include "codes.hpp"
#include "scaled.hpp"
#include "stream.hpp"

namespace dg {

namespace {

__device__ __forceinline__ i32x4_t load_piece(const int8_t *p)
{
    return __builtin_bit_cast(i32x4_t, load_bytes16(p));
}

__device__ __forceinline__ i32x4_t load_piece_masked(const int8_t *row, int64_t k, int64_t K)
{
    return __builtin_bit_cast(i32x4_t, load_masked16(row, k, K));
}

// Codes of up to kFewRows rows of x, in LDS: row r at r * ld, zeros from K to
// the next multiple of 128, and the rows' scales.  Every workgroup makes them
// for itself; x comes from the L2s.
template <int T, int NT>
__device__ __forceinline__ void make_codes(const char *x, int64_t ldx, int rows, int64_t K, int8_t *codes_s,
                                           int ld, float *scales_s)
{
    constexpr int ES = elem_bytes<T>(), NW = NT / 64;
    constexpr int CH = (int)(kFewElements / 8) / NT;       // pieces of eight of a thread and row
    static_assert(CH * NT * 8 == kFewElements, "whole pieces");
    __shared__ uint32_t tops[kFewRows][NW];
    const int tid = threadIdx.x;
    Raw8<T> held[kFewRows][CH];
    auto left = [&](int i) {
        const int64_t n = K - (int64_t)(i * NT + tid) * 8;
        return n < 0 ? 0 : n > 8 ? 8 : (int)n;
    };
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
        if (r < rows)
#pragma unroll
            for (int i = 0; i < CH; ++i)
                held[r][i] = load_raw8<T>(x + r * ldx + (int64_t)(i * NT + tid) * 8 * ES, left(i));
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
        if (r >= rows)
            continue;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            m = max(m, raw_abs_max<T>(held[r][i]));
        m = wave_max(m);
        if ((tid & 63) == 0)
            tops[r][tid >> 6] = m;
    }
    lds_barrier();
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
        if (r >= rows)
            continue;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            m = max(m, tops[r][w]);
        const RowScale s = row_scale<T>(m);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int at = (i * NT + tid) * 8;
            if (at < ld)                                   // zeros of x make zero codes
                *(uint2 *)(codes_s + r * ld + at) = codes<T>(held[r][i], s);
        }
        if (tid == 0)
            scales_s[r] = s.scale;
    }
    lds_barrier();
}

// T: DT_I8, or the type of few rows, one tile high, whose codes the workgroup
// makes (FM 1).
template <int T, int FM, int FN, int KW, int D>
__global__ __launch_bounds__(64 * KW) void scaled_stream_kernel(ScaledArgs a)
{
    constexpr bool OWN = T != DT_I8;
    constexpr int SK = 128, NT = 64 * KW, TILE = 16 * FM * 16 * FN, LD = 16 * FN + 4;
    static_assert(!OWN || FM == 1, "few rows");
    extern __shared__ __attribute__((aligned(16))) int32_t sums[];
    __shared__ float made_scales[OWN ? kFewRows : 1];
    // codes behind the sums
    const int code_ld = OWN ? ((int)a.g.K + SK - 1) / SK * SK : 0;
    int8_t *made = (int8_t *)(sums + KW * 16 * FM * LD);
    const GroupTile t = scaled_tile<16 * FM, 16>(a);
    if (t.group < 0)
        return;
    const GemmArgs g = scaled_args(a, t.group, t.start, t.rows);
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)t.row_tile * (16 * FM), n0 = (int64_t)t.col_tile * (16 * FN);
    const int rows = (int)(g.M - m0 < 16 * FM ? g.M - m0 : 16 * FM);
    const int cols = (int)(g.N - n0 < 16 * FN ? g.N - n0 : 16 * FN);

    const int8_t *ap[FM], *bp[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = 16 * i + c < rows ? 16 * i + c : rows - 1;
        ap[i] = OWN ? made + r * code_ld : (const int8_t *)g.A + (m0 + r) * g.lda;
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
        bp[j] = (const int8_t *)g.B + (n0 + (16 * j + c < cols ? 16 * j + c : cols - 1)) * g.ldb;

    struct Step {
        i32x4_t a[2][OWN ? 1 : FM], b[2][FN];
        int64_t k;
    };
    auto load = [&](Step &s, int64_t k) {
        s.k = k;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                s.b[h][j] = load_piece(bp[j] + k + 64 * h + 16 * kg);
            if constexpr (!OWN) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    s.a[h][i] = load_piece(ap[i] + k + 64 * h + 16 * kg);
            }
        }
    };
    i32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = i32x4_t{0, 0, 0, 0};
    auto multiply = [&](const Step &s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4_t x[FM];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                x[i] = OWN ? *(const i32x4_t *)(ap[i] + s.k + 64 * h + 16 * kg) : s.a[h][OWN ? 0 : i];
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    acc[i][j] = mfma_16x16x64(x[i], s.b[h][j], acc[i][j]);
        }
    };

    if (OWN || g.alpha != 0.0f) {          // uniform: OWN's barriers are below
        // A ring of D steps in registers, whose loads are under way while the
        // step before is multiplied.  Loads past the last whole step repeat it
        // and are not used: with none left out, the compiler can count them.
        // D = 2 only where few wavefronts fit a compute unit anyway: more
        // registers cost wavefronts (13 rows, 16384 x 8192, 16 x 64: 30 us
        // with two, 28.3 with one).
        // Workgroups begin at different steps, so that those running at one
        // time do not all read the same few k of rows a power of two apart
        // (13 rows, 16384 x 8192: 28.3 us without, 26.4 with; 64 rows, 4
        // groups, 4096 x 4096 18.9 and 17.2).
        const int32_t full = (int32_t)(g.K / SK);
        const int32_t turn = full > 0 ? (int32_t)(t.col_tile * 5 % (uint32_t)full) : 0;
        int32_t s = wave;
        Step ring[D];
        auto fetch = [&](Step &r, int32_t at) {
            at = (at < full ? at : full - 1) + turn;
            load(r, (int64_t)(at < full ? at : at - full) * SK);
        };
        if (s < full) {
#pragma unroll
            for (int i = 0; i < D; ++i)
                fetch(ring[i], s + i * KW);
        }
        if constexpr (OWN)
            make_codes<T, NT>(a.x + t.start * a.ldx, a.ldx, rows, g.K, made, code_ld, made_scales);
        if (s < full) {
            for (; s + D * KW < full; s += D * KW) {
#pragma unroll
                for (int i = 0; i < D; ++i) {
                    multiply(ring[i]);
                    fetch(ring[i], s + (D + i) * KW);
                }
            }
#pragma unroll
            for (int i = 0; i < D; ++i)
                if (s + i * KW < full)
                    multiply(ring[i]);
        }
        // at most one step is left, the turn of wavefront full mod KW
        const int64_t k0 = (int64_t)full * SK;
        if (k0 < g.K && wave == full % KW) {
            Step last;
            last.k = k0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = k0 + 64 * h + 16 * kg;
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    last.b[h][j] = load_piece_masked(bp[j], k, g.K);
                if constexpr (!OWN) {
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        last.a[h][i] = load_piece_masked(ap[i], k, g.K);
                }
            }
            multiply(last);
        }
    }

    int32_t *mine = sums + wave * (16 * FM * LD);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                mine[(16 * i + 4 * kg + v) * LD + 16 * j + c] = acc[i][j][v];
    lds_barrier();
    const float *sa = OWN ? made_scales : row_scales(a, t.start);
    const void *sb = col_scales(a, t.group);
    for (int o = tid; o < TILE; o += NT) {
        const int r = o / (16 * FN), col = o % (16 * FN);
        if (r >= rows || col >= cols)
            continue;
        int32_t sum = 0;
#pragma unroll
        for (int w = 0; w < KW; ++w)
            sum += sums[w * (16 * FM * LD) + r * LD + col];
        const float v =
            (float)sum * (sa ? sa[m0 + r] : 1.0f) * (sb ? load_as_f32(sb, a.scale_type, n0 + col) : 1.0f);
        store_c(g, 0, m0 + r, n0 + col, epilogue_value(g, 0, m0 + r, n0 + col, v));
    }
}

template <int FM, int FN, int KW, int D>
hipError_t launch(const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    constexpr size_t lds = (size_t)KW * 16 * FM * (16 * FN + 4) * 4;
    hipLaunchKernelGGL((scaled_stream_kernel<DT_I8, FM, FN, KW, D>), dim3(programs), dim3(64 * KW), lds, s, a);
    return hipGetLastError();
}

template <int FN, int D>
hipError_t launch_own(const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    const size_t lds = (size_t)8 * 16 * (16 * FN + 4) * 4 + (size_t)a.rows * ((a.g.K + 127) / 128 * 128);
    if (a.x_type == DT_F32)
        hipLaunchKernelGGL((scaled_stream_kernel<DT_F32, 1, FN, 8, D>), dim3(programs), dim3(512), lds, s, a);
    else if (a.x_type == DT_F16)
        hipLaunchKernelGGL((scaled_stream_kernel<DT_F16, 1, FN, 8, D>), dim3(programs), dim3(512), lds, s, a);
    else
        hipLaunchKernelGGL((scaled_stream_kernel<DT_BF16, 1, FN, 8, D>), dim3(programs), dim3(512), lds, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_scaled_few(int32_t variant, const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    switch (variant) {
    case 0: return launch_own<1, 2>(a, programs, s);
    case 1: return launch_own<2, 1>(a, programs, s);
    case 2: return launch_own<4, 1>(a, programs, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_scaled_stream(int32_t variant, const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    switch (variant) {
    case 0: return launch<1, 1, 8, 2>(a, programs, s);
    case 1: return launch<1, 2, 8, 1>(a, programs, s);
    case 2: return launch<1, 2, 4, 2>(a, programs, s);
    case 3: return launch<1, 4, 8, 1>(a, programs, s);
    case 4: return launch<2, 2, 8, 1>(a, programs, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace dg
