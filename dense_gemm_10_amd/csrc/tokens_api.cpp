// C ABI of the tokens sorted by group and back, and of the 8-bit codes of
// rows: host-side validation (no HIP calls) and launch.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/densegemm.h"
#include "checks.hpp"
#include "tokens.hpp"

using namespace dg;

namespace {

bool dtype_ok(int32_t t) { return t == DG_F32 || t == DG_BF16 || t == DG_F16; }

// Bytes of `rows` rows of `len` elements, `ld` apart.
bool bytes_of(int64_t rows, int64_t len, int64_t ld, int64_t es, int64_t *bytes)
{
    int64_t span;
    return matrix_span(DG_ROW_MAJOR, rows, len, ld, &span) && mul_ok(span, es, bytes);
}

// tokens * top_k, rows and a 32-bit numbering of both.
dg_status count_slots(int64_t tokens, int64_t top_k, int64_t rows, int64_t *slots)
{
    if (tokens < 0 || top_k < 0 || rows < 0)
        return DG_ERROR_INVALID_VALUE;
    if (!mul_ok(tokens, top_k, slots) || *slots > INT32_MAX || top_k > INT32_MAX || rows > INT32_MAX)
        return DG_ERROR_NOT_SUPPORTED;
    return DG_SUCCESS;
}

// A buffer of a call, for the overlap test.
struct Range {
    const void *p;
    int64_t bytes;
    bool written;
};

template <size_t N>
bool written_overlaps(const Range (&r)[N])
{
    for (size_t i = 0; i < N; ++i)
        for (size_t j = 0; r[i].written && j < N; ++j)
            if (i != j && ranges_overlap(r[i].p, r[i].bytes, r[j].p, r[j].bytes))
                return true;
    return false;
}

struct DispatchSpans {
    int64_t slots, index, x, rows;    // slots, then bytes
};

// What dg_dispatch and dg_spread share; `out_rows` rows of `rows`.
dg_status validate(const dg_dispatch_desc *d, bool spread, DispatchSpans *s)
{
    if (!d || d->struct_size != sizeof(dg_dispatch_desc))
        return DG_ERROR_INVALID_VALUE;
    if (!dtype_ok(d->x_type) || d->width < 0 || d->ldx < 1 || d->ldr < 1 || d->ldx < d->width ||
        d->ldr < d->width)
        return DG_ERROR_INVALID_VALUE;
    if (!spread && ((d->index_bits != 32 && d->index_bits != 64) || d->groups < 0 || d->ld_index < 1 ||
                    d->ld_index < d->top_k))
        return DG_ERROR_INVALID_VALUE;
    const dg_status st = count_slots(d->tokens, d->top_k, spread ? d->rows : 0, &s->slots);
    if (st != DG_SUCCESS)
        return st;
    if (!spread && d->groups > kMaxDispatchGroups)
        return DG_ERROR_NOT_SUPPORTED;
    const int64_t es = elem_size(d->x_type);
    s->index = 0;
    const bool ok = (spread || bytes_of(d->tokens, d->top_k, d->ld_index, d->index_bits / 8, &s->index)) &&
                    bytes_of(d->tokens, d->width, d->ldx, es, &s->x) &&
                    bytes_of(spread ? d->rows : s->slots, d->width, d->ldr, es, &s->rows);
    return ok ? DG_SUCCESS : DG_ERROR_INVALID_VALUE;
}

hipError_t spread_rows(const dg_dispatch_desc *d, const int32_t *place, const void *x, void *rows,
                       int64_t limit, void *stream)
{
    const int64_t es = elem_size(d->x_type);
    SpreadArgs a;
    memset(&a, 0, sizeof a);
    a.x = (const char *)x;
    a.rows = (char *)rows;
    a.place = place;
    a.ldx = d->ldx * es;
    a.ldr = d->ldr * es;
    a.width = d->width * es;
    a.tokens = d->tokens;
    a.top_k = (int32_t)d->top_k;
    a.limit = (int32_t)limit;
    a.elem = (int32_t)es;
    return launch_spread(a, (hipStream_t)stream);
}

struct CombineSpans {
    int64_t slots, z, dz, y, w, dw;
};

dg_status validate(const dg_combine_desc *d, bool grad, bool weights, CombineSpans *s)
{
    if (!d || d->struct_size != sizeof(dg_combine_desc))
        return DG_ERROR_INVALID_VALUE;
    if (!dtype_ok(d->z_type) || !dtype_ok(d->y_type) || ((grad || weights) && !dtype_ok(d->w_type)) ||
        d->width < 0)
        return DG_ERROR_INVALID_VALUE;
    if (d->ldz < 1 || d->ldz < d->width || d->ldy < 1 || d->ldy < d->width ||
        (grad && (d->lddz < 1 || d->lddz < d->width)) ||
        (weights && (d->ldw < 1 || d->ldw < d->top_k)))
        return DG_ERROR_INVALID_VALUE;
    if (d->y_type != d->z_type && d->y_type != DG_F32)
        return DG_ERROR_NOT_SUPPORTED;
    const dg_status st = count_slots(d->tokens, d->top_k, d->rows, &s->slots);
    if (st != DG_SUCCESS)
        return st;
    const int64_t ez = elem_size(d->z_type), ew = weights || grad ? elem_size(d->w_type) : 4;
    s->w = s->dz = s->dw = 0;
    const bool ok = bytes_of(d->rows, d->width, d->ldz, ez, &s->z) &&
                    bytes_of(d->tokens, d->width, d->ldy, elem_size(d->y_type), &s->y) &&
                    (!weights || bytes_of(d->tokens, d->top_k, d->ldw, ew, &s->w)) &&
                    (!grad || (bytes_of(d->rows, d->width, d->lddz, ez, &s->dz) &&
                               mul_ok(s->slots, ew, &s->dw)));
    return ok ? DG_SUCCESS : DG_ERROR_INVALID_VALUE;
}

CombineArgs combine_args(const dg_combine_desc *d, const int32_t *place, const void *weights)
{
    const int64_t ez = elem_size(d->z_type);
    CombineArgs a;
    memset(&a, 0, sizeof a);
    a.place = place;
    a.w = weights;
    a.ldz = d->ldz * ez;
    a.ldy = d->ldy * elem_size(d->y_type);
    a.ldw = d->ldw;
    a.tokens = d->tokens;
    a.width = d->width;
    a.top_k = (int32_t)d->top_k;
    a.limit = (int32_t)d->rows;
    a.z_type = d->z_type;
    a.y_type = d->y_type;
    a.w_type = d->w_type;
    return a;
}

} // namespace

extern "C" {

dg_status dg_dispatch(const dg_dispatch_desc *d, const void *index, const void *x, int32_t *offsets,
                      int32_t *order, int32_t *place, void *rows, void *stream)
{
    DispatchSpans sp;
    const dg_status st = validate(d, false, &sp);
    if (st != DG_SUCCESS)
        return st;
    const bool with_rows = x && rows;
    if ((x || rows) && !with_rows && sp.slots > 0 && d->width > 0)
        return DG_ERROR_INVALID_VALUE;
    if (!offsets || (sp.slots > 0 && (!index || !order || !place)))
        return DG_ERROR_INVALID_VALUE;
    const int64_t es = elem_size(d->x_type);
    if (!aligned_to(index, d->index_bits / 8) || !aligned_to(offsets, 4) || !aligned_to(order, 4) ||
        !aligned_to(place, 4) || !aligned_to(x, es) || !aligned_to(rows, es))
        return DG_ERROR_INVALID_VALUE;
    const Range all[] = {{index, sp.index, false},       {x, sp.x, false},
                         {offsets, (d->groups + 1) * 4, true}, {order, sp.slots * 4, true},
                         {place, sp.slots * 4, true},    {rows, sp.rows, true}};
    if (written_overlaps(all))
        return DG_ERROR_INVALID_VALUE;
    DispatchArgs a;
    memset(&a, 0, sizeof a);
    a.index = index;
    a.x = (const char *)x;
    a.offsets = offsets;
    a.order = order;
    a.place = place;
    a.rows = (char *)rows;
    a.ld_index = d->tokens > 1 ? d->ld_index : d->top_k;
    a.ldx = d->ldx * es;
    a.ldr = d->ldr * es;
    a.width = d->width * es;
    a.slots = (int32_t)sp.slots;
    a.top_k = (int32_t)d->top_k;
    a.groups = (int32_t)d->groups;
    a.index_bits = d->index_bits;
    a.elem = (int32_t)es;
    const bool move = with_rows && sp.slots > 0 && d->width > 0;
    hipError_t err;
    if (move && sp.slots <= kDispatchFewSlots) {
        err = launch_dispatch_few(a, (hipStream_t)stream);
    } else {
        err = launch_dispatch_sort(a, (hipStream_t)stream);
        if (err == hipSuccess && move)
            err = spread_rows(d, place, x, rows, sp.slots, stream);
    }
    return err == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_spread(const dg_dispatch_desc *d, const int32_t *place, const void *x, void *rows,
                    void *stream)
{
    DispatchSpans sp;
    const dg_status st = validate(d, true, &sp);
    if (st != DG_SUCCESS)
        return st;
    if (sp.slots == 0 || d->rows == 0 || d->width == 0)
        return DG_SUCCESS;
    const int64_t es = elem_size(d->x_type);
    if (!place || !x || !rows || !aligned_to(place, 4) || !aligned_to(x, es) || !aligned_to(rows, es))
        return DG_ERROR_INVALID_VALUE;
    const Range all[] = {{place, sp.slots * 4, false}, {x, sp.x, false}, {rows, sp.rows, true}};
    if (written_overlaps(all))
        return DG_ERROR_INVALID_VALUE;
    return spread_rows(d, place, x, rows, d->rows, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_combine(const dg_combine_desc *d, const void *z, const int32_t *place, const void *weights,
                     void *y, void *stream)
{
    CombineSpans sp;
    const dg_status st = validate(d, false, weights != nullptr, &sp);
    if (st != DG_SUCCESS)
        return st;
    if (d->tokens == 0 || d->width == 0)
        return DG_SUCCESS;
    const bool reads = sp.slots > 0 && d->rows > 0;
    if (!y || (reads && (!z || !place)) || !aligned_to(y, elem_size(d->y_type)) ||
        !aligned_to(z, elem_size(d->z_type)) || !aligned_to(place, 4) ||
        (weights && !aligned_to(weights, elem_size(d->w_type))))
        return DG_ERROR_INVALID_VALUE;
    const Range all[] = {{z, sp.z, false}, {place, sp.slots * 4, false}, {weights, sp.w, false}, {y, sp.y, true}};
    if (reads && written_overlaps(all))
        return DG_ERROR_INVALID_VALUE;
    CombineArgs a = combine_args(d, place, weights);
    a.z = (const char *)z;
    a.y = (char *)y;
    a.beta = d->beta;
    if (!reads)
        a.top_k = 0;                       // y = beta * y
    return launch_combine(a, (hipStream_t)stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_combine_grad(const dg_combine_desc *d, const void *dy, const void *z, const int32_t *place,
                          const void *weights, void *dz, void *dweights, void *stream)
{
    CombineSpans sp;
    const dg_status st = validate(d, true, weights != nullptr, &sp);
    if (st != DG_SUCCESS)
        return st;
    if (sp.slots == 0 || (!dz && !dweights))
        return DG_SUCCESS;
    const bool reads = d->width > 0 && d->rows > 0;
    const int64_t ez = elem_size(d->z_type), ew = elem_size(d->w_type);
    if (!place || (reads && (!dy || (dweights && !z))) || !aligned_to(dy, elem_size(d->y_type)) ||
        !aligned_to(z, ez) || !aligned_to(dz, ez) || !aligned_to(place, 4) ||
        (weights && !aligned_to(weights, ew)) || !aligned_to(dweights, ew))
        return DG_ERROR_INVALID_VALUE;
    const Range all[] = {{dy, sp.y, false}, {z, dweights ? sp.z : 0, false}, {place, sp.slots * 4, false},
                         {weights, sp.w, false}, {dz, sp.dz, true}, {dweights, sp.dw, true}};
    if (written_overlaps(all))
        return DG_ERROR_INVALID_VALUE;
    CombineArgs a = combine_args(d, place, weights);
    a.y = (char *)const_cast<void *>(dy);
    a.z = (const char *)z;
    a.dz = (char *)dz;
    a.dw = dweights;
    a.lddz = d->lddz * ez;
    if (!reads)
        a.width = 0;                       // dweights = 0; dy and z may be null
    return launch_combine_grad(a, (hipStream_t)stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_quantize(const dg_quantize_desc *d, const void *x, const int32_t *place, int8_t *q,
                      float *scales, void *stream)
{
    if (!d || d->struct_size != sizeof(dg_quantize_desc) || !dtype_ok(d->x_type) || d->width < 0 ||
        d->ldx < 1 || d->ldq < 1 || d->ldx < d->width || d->ldq < d->width || d->tokens < 0)
        return DG_ERROR_INVALID_VALUE;
    int64_t slots;
    const dg_status st = place ? count_slots(d->tokens, d->top_k, d->rows, &slots)
                               : count_slots(d->tokens, 1, 0, &slots);
    if (st != DG_SUCCESS)
        return st;
    const int64_t es = elem_size(d->x_type), rows = place ? d->rows : d->tokens;
    int64_t xb, qb;
    if (!bytes_of(d->tokens, d->width, d->ldx, es, &xb) || !bytes_of(rows, d->width, d->ldq, 1, &qb))
        return DG_ERROR_INVALID_VALUE;
    if (slots == 0 || rows == 0)
        return DG_SUCCESS;
    if (!scales || (d->width > 0 && (!x || !q)) || !aligned_to(x, es) || !aligned_to(scales, 4) ||
        !aligned_to(place, 4))
        return DG_ERROR_INVALID_VALUE;
    const Range all[] = {{x, xb, false}, {place, slots * 4, false}, {q, qb, true}, {scales, rows * 4, true}};
    if (written_overlaps(all))
        return DG_ERROR_INVALID_VALUE;
    QuantizeArgs a;
    memset(&a, 0, sizeof a);
    a.x = (const char *)x;
    a.place = place;
    a.q = q;
    a.scales = scales;
    a.ldx = d->ldx * es;
    a.ldq = d->ldq;
    a.tokens = d->tokens;
    a.width = d->width;
    a.top_k = (int32_t)d->top_k;
    a.limit = (int32_t)d->rows;
    a.x_type = d->x_type;
    return launch_quantize(a, (hipStream_t)stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

} // extern "C"
