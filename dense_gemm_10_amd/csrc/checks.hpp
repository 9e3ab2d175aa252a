// Host-side helpers of the entry points' argument checks: sizes with overflow
// tests, address ranges, alignment.  No HIP calls.
#pragma once
#include <stdint.h>

#include "../../include/densegemm.h"

namespace dg {

inline int64_t elem_size(int32_t t) { return t == DG_F32 ? 4 : 2; }

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }
inline bool add_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_add_overflow(a, b, out); }

// Elements spanned by one rows x cols matrix with the given order and ld.
inline bool matrix_span(int32_t order, int64_t rows, int64_t cols, int64_t ld, int64_t *span)
{
    if (rows == 0 || cols == 0) {
        *span = 0;
        return true;
    }
    int64_t outer = order == DG_ROW_MAJOR ? rows : cols;
    int64_t inner = order == DG_ROW_MAJOR ? cols : rows;
    int64_t t;
    return mul_ok(outer - 1, ld, &t) && add_ok(t, inner, span);
}

// Elements spanned by the whole batch.
inline bool batch_span(int64_t span, int64_t batch, int64_t stride, int64_t *total)
{
    if (span == 0 || batch == 0) {
        *total = 0;
        return true;
    }
    int64_t t;
    return mul_ok(batch - 1, stride, &t) && add_ok(t, span, total);
}

inline bool ranges_overlap(const void *p, int64_t pn, const void *q, int64_t qn)
{
    if (!p || !q || pn <= 0 || qn <= 0)
        return false;
    uintptr_t a0 = (uintptr_t)p, a1 = a0 + (uintptr_t)pn;
    uintptr_t b0 = (uintptr_t)q, b1 = b0 + (uintptr_t)qn;
    return a0 < b1 && b0 < a1;
}

inline bool aligned_to(const void *p, int64_t bytes) { return ((uintptr_t)p % bytes) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

} // namespace dg
