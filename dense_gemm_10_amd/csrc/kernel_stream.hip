// Grouped products with few rows per group (stream.hpp): 16-bit or fp32
// weights in either order.
//
// K-contiguous B[e] (BT false): lane l's operand of a 16 x 16 x 32 MFMA is
// 16 bytes of column l mod 16, k = 8 (l / 16) .. + 7: one load each.
// N-contiguous B[e] (BT true): lane 16 g + c loads columns FN c .. FN c +
// FN - 1 of the eight rows k = 8 g .. 8 g + 7 and pairs the rows in
// registers, two k of one column per register: FN operands, operand j
// holding columns FN c + j.  Either way a step is 64 k: 128 bytes of a
// column, or FN * 32 bytes of each row.
//
// fp32 has the same pieces of half as many k: lane 16 g + c holds k = 4 g ..
// 4 g + 3 of 16, and element t of every lane's piece makes MFMA t (16 x 16 x
// 4), whose four k are 4 g + t.
#include "stream.hpp"

namespace dg {

namespace {


// 16-bit halves of two words: (lo(a), lo(b)) and (hi(a), hi(b)).
__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// FN consecutive elements of ES bytes as words.
template <int FN, int ES> struct Run { uint32_t w[FN * ES / 4]; };

template <int FN, int ES>
__device__ __forceinline__ Run<FN, ES> load_run(const char *p)
{
    Run<FN, ES> r;
    __builtin_memcpy(&r, __builtin_assume_aligned(p, ES * FN), ES * FN);
    return r;
}

__device__ __forceinline__ uint32_t word(uint4 v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// acc += one piece of A against one piece of B.
template <int T>
__device__ __forceinline__ f32x4_t mfma_piece(uint4 a, uint4 b, f32x4_t acc)
{
    if constexpr (T == DT_F32) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(word(a, t)),
                                                       __uint_as_float(word(b, t)), acc, 0, 0, 0);
        return acc;
    } else {
        using frag_t = typename frag_of<T>::type;
        return mfma_16x16x32(__builtin_bit_cast(frag_t, a), __builtin_bit_cast(frag_t, b), acc);
    }
}

template <int T, bool BT, int FM, int FN, int KW>
__global__ __launch_bounds__(64 * KW) void grouped_stream_kernel(GroupedArgs a)
{
    constexpr int ES = T == DT_F32 ? 4 : 2;      // bytes of an element
    constexpr int VK = 16 / ES;                  // k of a 16-byte piece
    constexpr int HK = 4 * VK, SK = 2 * HK;      // k of half a step, and of a step
    static_assert(!BT || FN == 2 || FN == 4, "runs of 4 to 16 bytes");
    extern __shared__ uint4 lds[];
    const GroupTile t =
        find_group_tile<16 * FM, 16>(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x);
    if (t.group < 0)
        return;
    const GemmArgs g = group_args<false>(a, t.group, t.start, t.rows);
    const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m0 = (int64_t)t.row_tile * (16 * FM), n0 = (int64_t)t.col_tile * (16 * FN);
    const int rows = (int)(g.M - m0 < 16 * FM ? g.M - m0 : 16 * FM);
    const int cols = (int)(g.N - n0 < 16 * FN ? g.N - n0 : 16 * FN);

    // this lane's sources at k = 0 (rows of A, columns of a K-contiguous B),
    // and at its first k of a step (rows of an N-contiguous B)
    const char *ap[FM], *bp[BT ? 1 : FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = 16 * i + c < rows ? 16 * i + c : rows - 1;
        ap[i] = (const char *)g.A + (m0 + r) * g.lda * ES;
    }
    if constexpr (BT) {
        // the last run that starts inside the row; where N cuts it, it
        // reaches into the row's padding, or past the matrix on the last
        // row, which the masked step below therefore takes
        const int run = FN * c < cols ? FN * c : (cols - 1) / FN * FN;
        bp[0] = (const char *)g.B + (VK * kg * g.ldb + n0 + run) * ES;
    } else {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = 16 * j + c < cols ? 16 * j + c : cols - 1;
            bp[j] = (const char *)g.B + (n0 + n) * g.ldb * ES;
        }
    }

    struct Step {
        uint4 a[2][FM];
        uint4 b[BT ? 1 : 2][BT ? 1 : FN];
        Run<BT ? FN : 2, ES> run[BT ? 2 : 1][VK];
    };
    auto load = [&](Step &s, int64_t k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t kl = k + HK * h + VK * kg;     // this lane's first k
            if constexpr (BT) {
#pragma unroll
                for (int r = 0; r < VK; ++r)
                    s.run[h][r] = load_run<FN, ES>(bp[0] + (k + HK * h + r) * g.ldb * ES);
            } else {
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    s.b[h][j] = *(const uint4 *)(bp[j] + kl * ES);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
                s.a[h][i] = *(const uint4 *)(ap[i] + kl * ES);
        }
    };
    // the step at k with k >= K read as zero (and no load past a row's end)
    auto load_masked = [&](Step &s, int64_t k) {
        for (int h = 0; h < 2; ++h) {
            const int64_t kl = k + HK * h + VK * kg;
#pragma unroll
            for (int i = 0; i < FM; ++i)
                s.a[h][i] = piece16<T, VK>(ap[i], kl, 1, g.K, true);
            if constexpr (BT) {
#pragma unroll
                for (int r = 0; r < VK; ++r) {
                    uint32_t w[FN * ES / 4] = {};
                    const char *p = (const char *)g.B + ((kl + r) * g.ldb + n0 + FN * c) * ES;
#pragma unroll
                    for (int e = 0; e < FN; ++e) {
                        if (kl + r < g.K && FN * c + e < cols) {
                            if (ES == 4)
                                w[e] = ((const uint32_t *)p)[e];
                            else
                                w[e / 2] |= (uint32_t)((const uint16_t *)p)[e] << (16 * (e % 2));
                        }
                    }
                    __builtin_memcpy(&s.run[h][r], w, sizeof w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    s.b[h][j] = piece16<T, VK>(bp[j], kl, 1, g.K, true);
            }
        }
    };

    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Step &s) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                uint4 b;
                if constexpr (BT) {
                    uint32_t w[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        if constexpr (ES == 4) {
                            w[p] = s.run[h][p].w[j];
                        } else {
                            const uint32_t x = s.run[h][2 * p].w[j / 2];
                            const uint32_t y = s.run[h][2 * p + 1].w[j / 2];
                            w[p] = j % 2 ? pair_hi(x, y) : pair_lo(x, y);
                        }
                    }
                    b = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    b = s.b[h][j];
                }
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    acc[i][j] = mfma_piece<T>(s.a[h][i], b, acc[i][j]);
            }
    };

    if (g.alpha != 0.0f) {
        const bool cut = BT && cols % FN != 0;
        const int64_t full = (g.K - (cut && g.K > 0 ? 1 : 0)) / SK;
        int64_t s = wave;
        if (s < full) {
            Step now, next;
            load(now, s * SK);
            for (; s + KW < full; s += KW) {
                load(next, (s + KW) * SK);
                multiply(now);
                now = next;
            }
            multiply(now);
            s += KW;
        }
        // at most one step is left, and one wavefront's turn
        if (s * SK < g.K) {
            Step last;
            load_masked(last, s * SK);
            multiply(last);
        }
    }
    stream_store<FM, FN, KW, BT>(g, m0, n0, rows, cols, acc, (float *)lds);
}

template <int T, int FM, int FN, int KW>
hipError_t launch(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    constexpr size_t lds = stream_lds_bytes<FM, FN, KW>();
    if (a.g.b_col)
        hipLaunchKernelGGL((grouped_stream_kernel<T, false, FM, FN, KW>), dim3(programs),
                           dim3(64 * KW), lds, s, a);
    else
        hipLaunchKernelGGL((grouped_stream_kernel<T, true, FM, FN, KW>), dim3(programs),
                           dim3(64 * KW), lds, s, a);
    return hipGetLastError();
}

// 16-bit operands on <FM, FN, KW>, fp32 ones on 8 wavefronts: an fp32 MFMA
// is eight times slower, so its K is split further.
template <int FM, int FN, int KW>
hipError_t launch_typed(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    if (a.g.ab_type == DT_F32)
        return launch<DT_F32, FM, FN, 8>(a, programs, s);
    return a.g.ab_type == DT_F16 ? launch<DT_F16, FM, FN, KW>(a, programs, s)
                                 : launch<DT_BF16, FM, FN, KW>(a, programs, s);
}

} // namespace

hipError_t launch_grouped_stream(int32_t variant, const GroupedArgs &a, uint32_t programs,
                                 hipStream_t s)
{
    switch (variant) {
    case 0: return launch_typed<1, 2, 8>(a, programs, s);
    case 1: return launch_typed<1, 4, 8>(a, programs, s);
    case 2: return launch_typed<2, 4, 4>(a, programs, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace dg
