// Plain LDS-tiled kernels of the grouped products and of the products with
// 4-bit weights: every type, leading dimension and alignment.  They serve
// the operands the matrix-core kernels do not take (rows that do not start
// on 16 bytes, K not a whole number of steps).
//
// The tile is the generic dense kernel's: 64 x 64 outputs, K in steps of
// 16, 256 threads with 4 x 4 outputs each, fp32 products and sums, loads
// masked on the group's rows, N and K.  Bound by the vector FMA and LDS
// rate (about 10 TFLOP/s).
#include "grouped.hpp"

namespace dg {

namespace {

constexpr int GT = kGroupedGenericTile, GK = 16, GTHREADS = 256;

// acc += the product over [0, K) of a(row, k) and b(col, k), rows and
// columns of the tile at (m0, n0).  a_k / b_k: consecutive threads walk k
// (the operand is K-contiguous).
template <typename LA, typename LB>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], int64_t K, bool a_k, bool b_k,
                                             LA &&a, LB &&b)
{
    __shared__ float As[GK][GT + 1];
    __shared__ float Bs[GK][GT + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    for (int64_t k0 = 0; k0 < K; k0 += GK) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int idx = tid + GTHREADS * e;
            const int am = a_k ? idx / GK : idx % GT, ak = a_k ? idx % GK : idx / GT;
            const int bn = b_k ? idx / GK : idx % GT, bk = b_k ? idx % GK : idx / GT;
            As[ak][am] = k0 + ak < K ? a(am, k0 + ak) : 0.0f;
            Bs[bk][bn] = k0 + bk < K ? b(bn, k0 + bk) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < GK; ++k) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = As[k][ty + 16 * i];
                y[i] = Bs[k][tx + 16 * i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
        }
        __syncthreads();
    }
}

__device__ __forceinline__ void store_tile(const GemmArgs &g, int64_t m0, int64_t n0,
                                           const float (&acc)[4][4])
{
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < g.M && n < g.N)
                store_c(g, 0, m, n, epilogue_value(g, 0, m, n, acc[i][j]));
        }
}

template <int T, bool RAGGED_K>
__global__ __launch_bounds__(GTHREADS) void grouped_generic_kernel(GroupedArgs a)
{
    int32_t e, start, len;
    int64_t m0, n0;
    if (RAGGED_K) {
        int32_t end;
        e = (int32_t)(blockIdx.x / a.tiles);
        const uint32_t t = blockIdx.x % a.tiles;
        group_rows(a.offsets, a.rows, e, start, end);
        len = end - start;
        m0 = (int64_t)(t / a.tiles_n) * GT;
        n0 = (int64_t)(t % a.tiles_n) * GT;
    } else {
        const GroupTile t =
            find_group_tile<GT>(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x);
        if (t.group < 0)
            return;
        e = t.group;
        start = t.start;
        len = t.rows;
        m0 = (int64_t)t.row_tile * GT;
        n0 = (int64_t)t.col_tile * GT;
    }
    const GemmArgs g = group_args<RAGGED_K>(a, e, start, len);
    float acc[4][4] = {};
    if (g.alpha != 0.0f) {
        tile_product(
            acc, g.K, !RAGGED_K, g.b_col != 0,
            [&](int m, int64_t k) {
                return m0 + m < g.M ? load_as_f32(g.A, T, elem_offset(RAGGED_K, g.lda, m0 + m, k))
                                    : 0.0f;
            },
            [&](int n, int64_t k) {
                return n0 + n < g.N ? load_as_f32(g.B, T, elem_offset(g.b_col, g.ldb, k, n0 + n))
                                    : 0.0f;
            });
    }
    store_tile(g, m0, n0, acc);
}

template <int T>
__global__ __launch_bounds__(GTHREADS) void qweight_generic_kernel(QweightArgs a)
{
    GroupTile t;
    if (a.offsets) {
        t = find_group_tile<GT>(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x);
        if (t.group < 0)
            return;
    } else {
        t = GroupTile{0, 0, a.rows, blockIdx.x / a.tiles_n, blockIdx.x % a.tiles_n};
    }
    const int64_t m0 = (int64_t)t.row_tile * GT, n0 = (int64_t)t.col_tile * GT;
    const uint8_t *Q = a.Q + t.group * a.stride_q;
    const int64_t s0 = t.group * a.stride_s;
    const int64_t a0 = (int64_t)t.start * a.lda;
    float acc[4][4] = {};
    if (a.alpha != 0.0f) {
        tile_product(
            acc, a.K, true, true,
            [&](int m, int64_t k) {
                return m0 + m < t.rows ? load_as_f32(a.A, T, a0 + (m0 + m) * a.lda + k) : 0.0f;
            },
            [&](int n, int64_t k) {
                if (n0 + n >= a.N)
                    return 0.0f;
                const uint8_t two = Q[(n0 + n) * a.ldq + k / 2];
                const int32_t q = k % 2 ? two >> 4 : two & 15;
                const int64_t j = s0 + (n0 + n) * a.lds + k / a.group_size;
                const int32_t zero = a.zeros ? a.zeros[j] & 15 : 8;
                // an exact small integer times the scale: one rounding
                return (float)(q - zero) * load_as_f32(a.scales, a.scale_type, j);
            });
    }
    GemmArgs g{};
    g.M = t.rows;
    g.N = a.N;
    g.ldc = a.ldc;
    g.alpha = a.alpha;
    g.beta = a.beta;
    g.act = a.act;
    g.c_type = a.c_type;
    g.bias_type = a.bias_type;
    g.C = (char *)a.C + (int64_t)t.start * a.ldc * (a.c_type == DT_F32 ? 4 : 2);
    g.bias = a.bias ? (const char *)a.bias +
                          t.group * a.stride_bias * (a.bias_type == DT_F32 ? 4 : 2)
                    : nullptr;
    store_tile(g, m0, n0, acc);
}

template <bool RAGGED_K>
void enqueue(const GroupedArgs &a, dim3 grid, hipStream_t s)
{
    if (a.g.ab_type == DT_F32)
        hipLaunchKernelGGL((grouped_generic_kernel<DT_F32, RAGGED_K>), grid, dim3(GTHREADS), 0, s, a);
    else if (a.g.ab_type == DT_F16)
        hipLaunchKernelGGL((grouped_generic_kernel<DT_F16, RAGGED_K>), grid, dim3(GTHREADS), 0, s, a);
    else
        hipLaunchKernelGGL((grouped_generic_kernel<DT_BF16, RAGGED_K>), grid, dim3(GTHREADS), 0, s, a);
}

} // namespace

hipError_t launch_grouped_generic(const GroupedArgs &a, bool ragged_k, uint32_t programs,
                                  hipStream_t s)
{
    if (ragged_k)
        enqueue<true>(a, dim3(programs), s);
    else
        enqueue<false>(a, dim3(programs), s);
    return hipGetLastError();
}

hipError_t launch_qweight_generic(const QweightArgs &a, uint32_t programs, hipStream_t s)
{
    if (a.a_type == DT_F16)
        hipLaunchKernelGGL(qweight_generic_kernel<DT_F16>, dim3(programs), dim3(GTHREADS), 0, s, a);
    else
        hipLaunchKernelGGL(qweight_generic_kernel<DT_BF16>, dim3(programs), dim3(GTHREADS), 0, s, a);
    return hipGetLastError();
}

} // namespace dg
