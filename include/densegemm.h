/*
 * densegemm.h -- C ABI of an MI355X (gfx950) dense GEMM library.
 *
 * Operation (one call, optionally batched):
 *
 *     C[b] = act( alpha * A[b] . B[b] + beta * C[b] + bias )      b < batch
 *
 * with A[b] an M x K matrix, B[b] a K x N matrix, C[b] an M x N matrix, the
 * product accumulated in fp32 and rounded to C's dtype only after the whole
 * K loop.  The problem statement is the one of "La GEMM, de zero a cuBLAS"
 * section 2.1; the list of inputs (M, N, K, dtype, per-operand layout,
 * output dtype, epilogue with alpha / bias / activation / accumulation into
 * an existing C, batched or broadcast operands) follows "Skill: Write a
 * Triton GEMM Kernel", section "Inputs the agent should gather first"; the
 * rule that every stride is an argument and that a broadcast operand has
 * batch stride 0 follows the same page's "Kernel design rules" and
 * "Correctness requirements".
 *
 * Conventions
 *   - Plain C99.  Every pointer argument named A, B, C, bias or workspace is
 *     a DEVICE pointer; the descriptor and text buffers are HOST pointers.
 *   - Ownership: the caller owns every buffer.  The library never allocates
 *     or frees device memory and keeps no pointer after a call returns,
 *     apart from the work it has enqueued; the caller keeps the buffers alive
 *     until that work has completed on `stream`.  The descriptor is read only
 *     during the call.
 *   - Asynchrony: work is enqueued on `stream` (NULL = the null stream) and
 *     the library never synchronises.  Results of one call are ordered
 *     before later work on the same stream.
 *   - Errors: return codes only.  Every argument is validated on the host
 *     before anything is enqueued, so any status other than DG_SUCCESS and
 *     DG_ERROR_LAUNCH means nothing was enqueued.  The only mutable global
 *     state is the per-device address of dg_gemm_noalloc's scratch array,
 *     looked up once under a lock; calls are thread-safe and reentrant
 *     (dg_gemm_noalloc calls that overlap on one GPU share its scratch; see
 *     there).
 *   - Determinism: results are bitwise reproducible run to run for a given
 *     descriptor, including split-K (partials are reduced in a fixed order,
 *     never with atomics).
 */
#ifndef DENSEGEMM_H
#define DENSEGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DG_VERSION 10000 /* 1.0.0 */

/* Status codes. */
typedef enum {
    DG_SUCCESS = 0,
    DG_ERROR_INVALID_VALUE = 1,          /* malformed descriptor or pointers */
    DG_ERROR_NOT_SUPPORTED = 2,          /* valid, but not a supported combination */
    DG_ERROR_INSUFFICIENT_WORKSPACE = 3, /* forced split-K without enough workspace */
    DG_ERROR_LAUNCH = 4                  /* the runtime refused a kernel launch */
} dg_status;

/* Element types.  DG_BF16 is bfloat16: the top 16 bits of an IEEE fp32.
 * DG_F16 is IEEE 754 binary16 (5 exponent bits, 10 fraction bits; largest
 * finite value 65504).  Inputs in fp16 are the dtype of the pages' own
 * correctness check ("Skill: Write a Triton GEMM Kernel", Inputs the agent
 * should gather first, and the allclose check of "GEMM Kernel
 * Optimization", Verification). */
/* DG_I8, signed 8-bit integers, is a type of dg_gemm_scaled's A only. */
typedef enum { DG_F32 = 0, DG_BF16 = 1, DG_F16 = 2, DG_I8 = 3 } dg_dtype;

/* Storage order of one operand.  Row-major X (R x C) with leading dimension
 * ld holds X[r][c] at element r*ld + c; column-major holds it at c*ld + r. */
typedef enum { DG_ROW_MAJOR = 0, DG_COL_MAJOR = 1 } dg_order;

/* Epilogue activation, applied to alpha*acc + beta*C + bias.
 * GELU_ERF is x * Phi(x) with Phi the standard normal CDF;
 * GELU_TANH replaces Phi(x) by (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3)))/2. */
typedef enum { DG_ACT_NONE = 0, DG_ACT_GELU_ERF = 1, DG_ACT_GELU_TANH = 2 } dg_act;

/* Kernel family selection (benchmarking and ablation; 0 lets the library
 * choose).  GENERIC is the plain LDS-tiled kernel that serves every
 * layout, alignment and dtype.  For fp32 the automatic choice is the
 * matrix-core kernel (MFMA_F32) when the operands are 16-byte aligned with
 * leading dimensions and batch strides multiple of 4; VALU_F32 (the
 * register-tiled vector-FMA kernel) takes the same operands and is used
 * only when asked for.  bf16 and fp16 inputs go to their matrix-core kernel
 * (MFMA_BF16, MFMA_F16) in any order of A and B, both 16-byte aligned with
 * leading dimensions and batch strides multiple of 8 (a column-major A or
 * row-major B is transposed on its way from LDS to the matrix cores).
 * Forcing a family whose requirements the operands do not meet returns
 * DG_ERROR_NOT_SUPPORTED. */
typedef enum {
    DG_ALGO_AUTO = 0,
    DG_ALGO_GENERIC = 1,
    DG_ALGO_VALU_F32 = 2,  /* register-tiled fp32 outer-product kernel */
    DG_ALGO_MFMA_BF16 = 3, /* bf16 matrix-core kernel */
    DG_ALGO_MFMA_F32 = 4,  /* fp32 matrix-core kernel */
    DG_ALGO_MFMA_F16 = 5   /* fp16 matrix-core kernel (the bf16 kernel's twin) */
} dg_algo;

/* Work distribution over the compute units (benchmarking and ablation; 0
 * lets the library choose).  DATA_PARALLEL gives every output tile (and
 * split-K slice) to one workgroup.  STREAM_K splits work along K to keep
 * the last wave busy ("La GEMM, de zero a cuBLAS", section 2.10, on
 * Stream-K and wave quantisation): the tiles of the full waves stay
 * data-parallel, and the K range of each remaining (tail) tile is cut into
 * slices, one workgroup each, enough to fill one more wave; a second, small
 * kernel adds each tail tile's fp32 partials in slice order (fixed order, no
 * atomics) and applies the epilogue; with STREAM_K, split_k = S > 1 cuts
 * each tail tile's K range into slices of ceil(K / S) rounded up to whole K
 * steps (so possibly fewer than S slices) instead of a split-K count.  STREAM_K applies to the bf16 and fp16 matrix-core
 * kernels with batch == 1 and needs workspace
 * (see dg_gemm_workspace_size); otherwise DG_ERROR_NOT_SUPPORTED.  The
 * automatic choice uses it only for those kernels, when there is at least
 * one full wave of tiles, the last wave would be less than 85 % full,
 * K >= 2048 and the caller passes enough workspace, or where the
 * offline-tuned plan table names it for the exact shape.
 *
 * With schedule, algo and split_k all left to the library, an output whose
 * N ends 1 to 8 columns past a whole number of tile columns (for the tile
 * the plan chose), with row-major A whose rows are 16-byte aligned, at
 * least one full-width tile per compute unit, and one wave of tiles fewer
 * without the last tile column, is computed in two launches
 * on the stream: the tiled plan over the full tile columns, then a small
 * kernel over the last columns (one wavefront per row of A, each output a
 * K-long fp32 dot product, the same epilogue).  A tuned stream-K plan with
 * a tail wave keeps the whole grid instead.  Results agree with the single
 * tiled plan within the dtype's tolerance (bit for bit when every product
 * and partial sum is exact in fp32). */
typedef enum {
    DG_SCHED_AUTO = 0,
    DG_SCHED_DATA_PARALLEL = 1,
    DG_SCHED_STREAM_K = 2
} dg_schedule;

/*
 * Problem descriptor.  All integer fields are in ELEMENTS, not bytes.
 *
 *   struct_size     must be sizeof(dg_gemm_desc) (ABI versioning).
 *   M, N, K         >= 0.  M == 0 or N == 0 is a successful no-op; K == 0
 *                   gives C = act(beta*C + bias).
 *   batch           >= 0; 0 is a no-op.
 *   a_type, b_type  input types; c_type output type.  Supported
 *                   (a, b, c): (F32, F32, F32), and for 16-bit inputs
 *                   (X, X, c) with X = BF16 or F16 and c = F32, BF16 or
 *                   F16.  Accumulation is always fp32; a 16-bit output is
 *                   rounded to nearest, ties to even (fp16 beyond 65504
 *                   rounds to infinity).
 *   a_order ...     storage order of A (M x K), B (K x N), C (M x N).
 *   lda, ldb, ldc   leading dimensions, each >= max(1, length of the
 *                   contiguous dimension) (e.g. row-major A: lda >= K).
 *   stride_a/b/c    batch strides, >= 0.  stride_a == 0 (or stride_b == 0)
 *                   broadcasts one A (B) to every batch entry.
 *                   stride_c must not make two C matrices overlap.
 *   alpha, beta     host scalars.  beta == 0: C is not read (NaN in C does
 *                   not propagate).  alpha == 0: A and B are not read.
 *   bias, bias_type optional DEVICE vector of N elements (F32, BF16 or F16),
 *                   added to every row; NULL for none.
 *   act             activation, see dg_act.
 *   split_k         0: the library decides (it only splits K when the
 *                   caller passes enough workspace); 1: never split;
 *                   S > 1: split K into S slices (needs workspace); with
 *                   schedule STREAM_K, the K slices of each tail tile.
 *   group_m         output-tile group height of the swizzled tile order; 0
 *                   picks the default (4, measured best with the XCD
 *                   remap).  1 gives plain row-major order.
 *   algo            dg_algo; 0 = automatic choice.
 *   xcd_remap       1 (default when 0) spreads consecutive tile groups over
 *                   the chip's 8 XCDs so each XCD's L2 sees a contiguous
 *                   part of the swizzled order; -1 disables it.
 *   schedule        dg_schedule; 0 = automatic choice.
 */
typedef struct dg_gemm_desc {
    uint32_t struct_size;
    int32_t a_type, b_type, c_type;   /* dg_dtype */
    int64_t M, N, K, batch;
    int32_t a_order, b_order, c_order; /* dg_order */
    int32_t bias_type;                 /* dg_dtype */
    int64_t lda, ldb, ldc;
    int64_t stride_a, stride_b, stride_c;
    float alpha, beta;
    const void *bias;
    int32_t act;       /* dg_act */
    int32_t split_k;
    int32_t group_m;
    int32_t algo;      /* dg_algo */
    int32_t xcd_remap;
    int32_t schedule;  /* dg_schedule */
} dg_gemm_desc;

/* Library version, DG_VERSION of the build. */
int dg_version(void);

/* Static text for a status code; never NULL. */
const char *dg_status_string(dg_status s);

/* Device bytes of workspace that dg_gemm would use for `d` (0 when the
 * chosen plan needs none).  The workspace holds fp32 partial sums: of
 * every K slice of a split-K plan, reduced in a separate pass ("Skill:
 * Write a Triton GEMM Kernel", Kernel design rules, on split-K), or of the
 * tail tiles' K slices of a stream-K plan.  With split_k == 0 and schedule == 0 this is the
 * size that lets the library pick split-K or Stream-K where they pay.  Returns INVALID_VALUE /
 * NOT_SUPPORTED for descriptors dg_gemm would reject. */
dg_status dg_gemm_workspace_size(const dg_gemm_desc *d, size_t *bytes);

/* Enqueue C = act(alpha*A.B + beta*C + bias) on `stream`.
 *   A, B, C    device pointers to the matrices (C is read when beta != 0
 *              and written); they must be aligned to their element size.
 *              C must not overlap A, B or bias.  A and B may be NULL when
 *              alpha == 0 or K == 0.
 *   workspace  device scratch of workspace_bytes (may be NULL / 0),
 *              16-byte aligned.  The library writes it; its content before
 *              and after is unspecified.  It must not be used by other work
 *              until this call's work has completed on `stream`.
 *   stream     a hipStream_t (passed as void*), NULL for the null stream.
 * Returns DG_SUCCESS once the work is enqueued. */
dg_status dg_gemm(const dg_gemm_desc *d, const void *A, const void *B, void *C,
                  void *workspace, size_t workspace_bytes, void *stream);

/* Size in bytes of the per-GPU scratch array of dg_gemm_noalloc. */
#define DG_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* dg_gemm for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation.
 * Same operation, arguments (minus the workspace), validation, plans and
 * results as dg_gemm given DG_NOALLOC_SCRATCH_BYTES of workspace, except
 * that split-K and stream-K partials go to a scratch array of that size
 * that is part of the library's device code: each GPU the library runs on
 * holds one copy from the library's load until the process ends, and no
 * call allocates or frees anything (no hipMalloc / hipFree, no allocating
 * library routine).  The first call on a device looks up that device's copy
 * (hipGetSymbolAddress, with the device current); later calls reuse it.
 *   - The automatic choice never plans more than DG_NOALLOC_SCRATCH_BYTES
 *     of workspace.  A forced split_k or STREAM_K schedule whose workspace
 *     (see dg_gemm_workspace_size) exceeds it returns
 *     DG_ERROR_INSUFFICIENT_WORKSPACE before anything is enqueued.
 *   - Every call on one GPU shares that GPU's scratch, which keeps the last
 *     call's partials; nothing in it needs to start at zero.  Calls whose
 *     work overlaps in time on one GPU (other streams, other host threads)
 *     race on it: order them on one stream or serialise them.
 *   - DG_ERROR_LAUNCH also covers a failed device or symbol lookup. */
dg_status dg_gemm_noalloc(const dg_gemm_desc *d, const void *A, const void *B, void *C,
                          void *stream);

/* Write a one-line, NUL-terminated description of the plan dg_gemm would
 * run for `d` (kernel, tile, split, grid, workspace) into buf[len].  Pass
 * workspace_bytes as dg_gemm would receive it (it decides split-K when
 * split_k == 0).  "sliver=n" (n > 0) marks the two-launch split above:
 * the rest of the line then describes the tiled plan over the first N - n
 * columns.  "tuned=1" marks a plan taken from the library's
 * offline-tuned table: for the exact (kernel family, M, N, K, batch) of a
 * shape swept on an MI355X, the tile and schedule that measured fastest
 * replace the heuristic choice ("GEMM Kernel Optimization", Autotune
 * Configs; "Skill: Write a Triton GEMM Kernel", Required reasoning process
 * step 7; with the benchmarking done once, offline). */
dg_status dg_gemm_describe(const dg_gemm_desc *d, size_t workspace_bytes, char *buf,
                           size_t len);

/* Host-side evaluation of the tile scheduler, for checking its bijection:
 * for every program id p < P = batch * S * ceil(M/bm) * ceil(N/bn) writes
 * out[4p .. 4p+3] = (batch index, split index, tile row, tile column) that
 * a kernel launched with that grid gives program p.  `out` is a HOST array
 * of 4*P int32.  Uses exactly the code the kernels use, which is 32-bit:
 * P above 2^31 - 1 (more programs than any launch can have) returns
 * DG_ERROR_NOT_SUPPORTED. */
dg_status dg_schedule_map(int64_t M, int64_t N, int64_t batch, int32_t split_k, int32_t bm,
                          int32_t bn, int32_t group_m, int32_t xcd_remap, int32_t *out,
                          int64_t out_len);

/* ---- products over groups of rows ------------------------------------------
 *
 * A layer of experts multiplies the rows routed to each expert by that
 * expert's matrix.  The rows of one group are consecutive, the groups have
 * any lengths, and the lengths are known on the GPU only:
 *
 *   offsets  a DEVICE array of groups + 1 int32; group e is rows
 *            [offsets[e], offsets[e+1]).  Values are clamped to [0, rows]
 *            and made non-decreasing by a running maximum before use, so no
 *            content of the array makes a call read or write outside its
 *            operands; a group may be empty.  Rows before offsets[0] and
 *            from offsets[groups] on belong to no group.
 *
 * DG_RAGGED_M (a layer's forward pass, and with B transposed its input
 * gradient): for each row i of group e
 *
 *     C[i,:] = act( alpha * A[i,:] . B[e] + beta * C[i,:] + bias[e] )
 *
 *   A rows x K row-major, B[e] K x N in either order, C rows x N row-major.
 *   Rows of C that belong to no group are neither read nor written, and the
 *   same rows of A are not used.
 *
 * DG_RAGGED_K (the weight gradient): for each group e
 *
 *     C[e] = alpha * A[rows of e]^T . B[rows of e] + beta * C[e]
 *
 *   A rows x M row-major, B rows x N row-major, C[e] M x N row-major.  An
 *   empty group gives beta * C[e] (0 when beta == 0).  No bias, no
 *   activation; the bias gradient is the same call with M = 1 and an A of
 *   ones.
 *
 * Types, accumulation, rounding, ownership, streams and errors as in
 * dg_gemm; no workspace, nothing allocated, nothing read back, so calls may
 * be captured into HIP graphs (a replay reads the offsets anew).  The work
 * is planned from rows and groups; the offsets decide only which part of it
 * each workgroup does. */
typedef enum { DG_RAGGED_M = 0, DG_RAGGED_K = 1 } dg_ragged;

/*
 * All integer fields are in ELEMENTS.
 *   struct_size     sizeof(dg_grouped_desc).
 *   ragged          dg_ragged.
 *   a_type ...      as in dg_gemm_desc: (F32, F32, F32) or (X, X, c) with X
 *                   = BF16 or F16 and c any type.
 *   b_order         order of each B[e]; RAGGED_K: DG_ROW_MAJOR.
 *   groups          0 .. 65536; 0 is a no-op.
 *   rows            0 .. 2^31 - 1, the allocated rows of A (and C or B).
 *   M               RAGGED_K only.    K  RAGGED_M only.    (else ignored)
 *   lda, ldb, ldc   leading dimensions, each >= max(1, the row's length).
 *   stride_b        RAGGED_M: distance of consecutive B[e] (0: one B).
 *   stride_c        RAGGED_K: distance of consecutive C[e], which must not
 *                   overlap.
 *   bias            RAGGED_M: optional DEVICE array; bias[e] is N elements
 *                   at e * stride_bias (0: one bias).
 *   alpha, beta, act as in dg_gemm_desc.
 */
typedef struct dg_grouped_desc {
    uint32_t struct_size;
    int32_t ragged;
    int32_t a_type, b_type, c_type, bias_type;
    int32_t b_order;
    int32_t act;
    int64_t groups, rows;
    int64_t M, N, K;
    int64_t lda, ldb, ldc;
    int64_t stride_b, stride_c, stride_bias;
    float alpha, beta;
    const void *bias;
} dg_grouped_desc;

/* Enqueue the products on `stream`.  DG_ERROR_NOT_SUPPORTED also where even
 * the largest tile makes a launch of 2^32 threads or more: with rows on 16
 * bytes from about 2^24 tiles of 256 x 256 (16 bits) or 128 x 128 (fp32), else of
 * 64 x 64; a group's last tile counts whole. */
dg_status dg_gemm_grouped(const dg_grouped_desc *d, const void *A, const void *B, void *C,
                          const int32_t *offsets, void *stream);

/* One line on the kernel, tile and grid dg_gemm_grouped would run (operands
 * taken as aligned). */
dg_status dg_gemm_grouped_describe(const dg_grouped_desc *d, char *buf, size_t len);

/* ---- products with 4-bit weights --------------------------------------------
 *
 *     C = act( alpha * A . W^T + beta * C + bias )
 *     W[n][k] = scale[n][k / group_size] * (q[n][k] - zero[n][k / group_size])
 *
 * with A M x K row-major in BF16 or F16, C M x N row-major, q in 0 .. 15.
 *   Q       row n at byte n * ldq, ceil(K / 2) bytes: q[n][2j] is the low
 *           and q[n][2j+1] the high half of byte j.
 *   scales  scale[n][j] at element n * lds + j, ceil(K / group_size) of them.
 *   zeros   one byte each, laid out as the scales (values 0 .. 15; the low
 *           four bits count); NULL: every zero is 8.
 * With offsets, row i of A and C uses the weights of the group that holds
 * it, W[e] at Q + e * stride_q bytes, scales and zeros + e * stride_s, bias
 * + e * stride_bias; the offsets as above, with M in the place of rows, and
 * rows of no group left as they were.  offsets may be NULL when groups == 1:
 * all M rows then use the one W.
 * W is never rounded to 16 bits: the scales and zeros enter in fp32.
 * Infinities and NaN give what the formula does, from every kernel; an output
 * that is not finite takes longer (its k one by one).
 *
 *   struct_size  sizeof(dg_qweight_desc).
 *   a_type       BF16 or F16 (F32: DG_ERROR_NOT_SUPPORTED).
 *   c_type, scale_type, bias_type   any dg_dtype.
 *   groups       1 .. 65536 weight matrices (0 is a no-op).
 *   M            0 .. 2^31 - 1 rows.
 *   group_size   a positive multiple of 32 (else DG_ERROR_NOT_SUPPORTED);
 *                the last group of a row may be shorter.
 *   lda, ldc, lds in elements (lds also for zeros), ldq and stride_q in
 *                bytes; lda >= max(1, K), ldc >= max(1, N), ldq >=
 *                max(1, ceil(K / 2)), lds >= max(1, ceil(K / group_size)).
 */
typedef struct dg_qweight_desc {
    uint32_t struct_size;
    int32_t a_type, c_type, scale_type, bias_type;
    int32_t act;
    int64_t groups;
    int64_t M, N, K, group_size;
    int64_t lda, ldc, ldq, lds;
    int64_t stride_q, stride_s, stride_bias;
    float alpha, beta;
    const void *bias;
} dg_qweight_desc;

/* Enqueue the product on `stream`.  Needs no workspace; may be captured.
 * DG_ERROR_NOT_SUPPORTED also where even the largest tile makes a launch of
 * 2^32 threads or more: from about 2^23 tiles of 64 x 256 (64 x 512 for group
 * sizes that are multiples of 128), or 2^24 of 64 x 64 for operands off the
 * 16-byte grid or K that is no multiple of 32. */
dg_status dg_gemm_qweight(const dg_qweight_desc *d, const void *A, const void *Q,
                          const void *scales, const void *zeros, void *C,
                          const int32_t *offsets, void *stream);

/* One line on the kernel, tile and grid dg_gemm_qweight would run, with or
 * without offsets (operands taken as aligned). */
dg_status dg_gemm_qweight_describe(const dg_qweight_desc *d, char *buf, size_t len);

/* ---- tokens sorted by group, and back -----------------------------------------
 *
 * A router names top_k groups (experts) for every token.  Slot s = t * top_k
 * + j is token t's j-th choice, S = tokens * top_k slots in all, and
 * index[t][j] its group; a value outside [0, groups) names no group (padding
 * tokens, choices over an expert's capacity).  dg_dispatch sorts the slots
 * by group, those of one group in ascending order, and writes
 *
 *   offsets  groups + 1 int32, as dg_gemm_grouped reads them: group e is
 *            rows [offsets[e], offsets[e + 1]); offsets[0] = 0;
 *   order    S int32: the slot of every row, -1 from row offsets[groups] on;
 *   place    tokens x top_k int32, packed: the row of every slot, -1 for a
 *            slot of no group (so order[place[s]] == s);
 *   rows     S x width: row place[t][j] is x[t].  Rows from offsets[groups]
 *            on are left as they were.
 *
 * x and rows NULL: only the maps.  dg_spread writes the rows alone, from a
 * given place:  rows[place[t][j]] = x[t].
 *
 * dg_combine brings rows back:
 *
 *     y[t] = sum_j weights[t][j] * z[place[t][j]] + beta * y[t]
 *
 * over the slots with a row, in the order of j, in fp32, rounded once;
 * weights NULL: ones, which with z = the rows' gradients is the gradient of
 * dg_dispatch and dg_spread.  dg_combine_grad is its own gradient: for every
 * slot with a row
 *
 *     dz[place[t][j]] = weights[t][j] * dy[t]
 *     dweights[t][j]  = sum_c dy[t][c] * z[place[t][j]][c]
 *
 * and dweights 0 for a slot without; rows of dz that no slot has are left as
 * they were.  A place outside [0, rows) is one without a row, so no content
 * of the arrays makes a call read or write outside its operands.  Two slots
 * may have one row in dg_combine; in dg_spread and dg_combine_grad each element
 * of such a row then gets the value of either (dg_dispatch writes no such
 * place).
 *
 * Types, ownership, streams and errors as in dg_gemm; no workspace, nothing
 * allocated, nothing read back; calls may be captured into HIP graphs.
 *
 * All integer fields are in ELEMENTS.
 *   struct_size   sizeof(dg_dispatch_desc), sizeof(dg_combine_desc).
 *   x_type        of x and rows (any dg_dtype).
 *   index_bits    32 or 64: signed integers.
 *   tokens, top_k, rows   >= 0, tokens * top_k and rows at most 2^31 - 1.
 *   groups        0 .. 8192 (more: DG_ERROR_NOT_SUPPORTED).
 *   rows          dg_spread: allocated rows of `rows`; dg_combine and
 *                 dg_combine_grad: of z and dz.  dg_dispatch ignores it:
 *                 `rows` has S.
 *   ld_index, ldx, ldr, ldz, lddz, ldy, ldw   leading dimensions of index,
 *                 x, rows, z, dz, y (or dy) and weights; each >= max(1, the
 *                 row's length).  place and dweights are packed.
 *   z_type, y_type   of z and dz, and of y or dy: the same, or y_type F32.
 *   w_type        of weights and dweights (any dg_dtype). */
typedef struct dg_dispatch_desc {
    uint32_t struct_size;
    int32_t x_type;
    int32_t index_bits;
    int64_t tokens, top_k, groups, rows, width;
    int64_t ld_index, ldx, ldr;
} dg_dispatch_desc;

typedef struct dg_combine_desc {
    uint32_t struct_size;
    int32_t z_type, y_type, w_type;
    int64_t tokens, top_k, rows, width;
    int64_t ldz, lddz, ldy, ldw;
    float beta;
} dg_combine_desc;

dg_status dg_dispatch(const dg_dispatch_desc *d, const void *index, const void *x,
                      int32_t *offsets, int32_t *order, int32_t *place, void *rows,
                      void *stream);

dg_status dg_spread(const dg_dispatch_desc *d, const int32_t *place, const void *x, void *rows,
                    void *stream);

dg_status dg_combine(const dg_combine_desc *d, const void *z, const int32_t *place,
                     const void *weights, void *y, void *stream);

/* dz or dweights may be NULL (not wanted); z is read for dweights only, and
 * neither dy nor z where rows or width is 0.  beta is ignored.  weights NULL:
 * ones. */
dg_status dg_combine_grad(const dg_combine_desc *d, const void *dy, const void *z,
                          const int32_t *place, const void *weights, void *dz, void *dweights,
                          void *stream);

/* ---- products in 8-bit integers -------------------------------------------------
 *
 * dg_quantize makes 8-bit codes of every row of x, and its scale:
 *
 *     scales[t] = max_k |x[t][k]| / 127         (fp32)
 *     q[t][k]   = 127 * x[t][k] / max, to the nearest integer, ties to even
 *
 * the codes from the exact quotient; a row of zeros gets scale 0 and codes 0,
 * a row that holds an infinity or NaN gets scale NaN and codes 0.  With
 * `place` (tokens x top_k int32, packed, as dg_dispatch writes it) the codes
 * and scale of token t go to the rows place[t][j] of q and scales, in
 * [0, rows); other rows are left as they were.  Of a row that two tokens have,
 * each code, and the scale, is of either, and codes and scale need not be of
 * the same one.  place NULL: row t, and rows and top_k are ignored.
 *   x_type any dg_dtype; ldx, ldq >= max(1, width); tokens * top_k and rows
 *   at most 2^31 - 1. */
typedef struct dg_quantize_desc {
    uint32_t struct_size;
    int32_t x_type;
    int64_t tokens, top_k, rows, width;
    int64_t ldx, ldq;
} dg_quantize_desc;

dg_status dg_quantize(const dg_quantize_desc *d, const void *x, const int32_t *place, int8_t *q,
                      float *scales, void *stream);

/* The product of 8-bit integers with a scale for each row and each column:
 *
 *     C = act( alpha * scale_a[m] * scale_b[n] * sum_k A[m][k] * B[n][k]
 *              + beta * C + bias )
 *
 * with A M x K and B N x K (one row per column of C), both row-major, C M x N
 * row-major.  The sum is exact, in 32-bit integers; it is converted to fp32
 * (half a step of 24 bits) and multiplied by scale_a, scale_b and alpha in
 * that order.  scale_a (fp32) or scale_b NULL: ones.
 * a_type F32, BF16 or F16: A's rows are turned into codes and scales first,
 * as by dg_quantize, in the workspace if there is one; scale_a must be NULL.
 * With offsets, row i of A and C uses the B of the group that holds it, B + e
 * * stride_b, scale_b + e * stride_s, bias + e * stride_bias; the offsets as
 * in dg_gemm_grouped with M in the place of rows, and rows of no group left
 * as they were.  offsets may be NULL when groups == 1: all M rows then use
 * the one B.
 *
 *   struct_size  sizeof(dg_scaled_desc).
 *   a_type       DG_I8 or any other dg_dtype (see above).
 *   c_type, scale_type (of scale_b), bias_type   F32, BF16 or F16.
 *   groups       1 .. 65536 matrices B (0 is a no-op).
 *   M            0 .. 2^31 - 1 rows.
 *   K            0 .. 131071 (more: DG_ERROR_NOT_SUPPORTED; the sum would not
 *                fit 32 bits).
 *   lda, ldb >= max(1, K), ldc >= max(1, N); strides >= 0, in elements. */
typedef struct dg_scaled_desc {
    uint32_t struct_size;
    int32_t a_type, c_type, scale_type, bias_type;
    int32_t act;
    int64_t groups;
    int64_t M, N, K;
    int64_t lda, ldb, ldc;
    int64_t stride_b, stride_s, stride_bias;
    float alpha, beta;
    const void *bias;
} dg_scaled_desc;

/* Device bytes of workspace of dg_gemm_scaled: 0 for a_type DG_I8, and for up
 * to DG_SCALED_FEW_ROWS rows of up to DG_SCALED_FEW_ELEMENTS elements together
 * with groups 1. */
#define DG_SCALED_FEW_ROWS 4
#define DG_SCALED_FEW_ELEMENTS 8192
dg_status dg_gemm_scaled_workspace_size(const dg_scaled_desc *d, size_t *bytes);

/* Enqueue the product on `stream`; may be captured.  workspace: 16-byte
 * aligned, used until the call's work has completed; fewer bytes than
 * dg_gemm_scaled_workspace_size says are DG_ERROR_INSUFFICIENT_WORKSPACE.
 * DG_ERROR_NOT_SUPPORTED also where even the largest tile makes a launch of
 * 2^32 threads or more. */
dg_status dg_gemm_scaled(const dg_scaled_desc *d, const void *A, const float *scale_a,
                         const int8_t *B, const void *scale_b, void *C, const int32_t *offsets,
                         void *workspace, size_t workspace_bytes, void *stream);

/* One line on the kernel, tile and grid dg_gemm_scaled would run, with or
 * without offsets (operands taken as aligned). */
dg_status dg_gemm_scaled_describe(const dg_scaled_desc *d, char *buf, size_t len);

#ifdef __cplusplus
}
#endif
#endif /* DENSEGEMM_H */
