// call_check.h -- what the entry points over plain device arrays share: checks of
// a call's buffers before any device work, and places in a workspace.
#pragma once

#include <hip/hip_runtime.h>

#include "zero_internal.h"

namespace zero {

inline int esize(int32_t d) { return d == ZERO_BF16 ? 2 : 4; }

// A buffer of the call: `bytes` from p, elements of `align` bytes.
struct Span {
    const void *p;
    int64_t bytes;
    int align;
};

inline bool bad_dtype(int32_t d) { return d != ZERO_F32 && d != ZERO_BF16; }

// Whether n rows of `stride` elements stay within 61 bits of bytes.
inline bool stride_fits(int64_t n, int64_t stride)
{
    return stride <= (int64_t(1) << 61) / 4 / (n > 0 ? n : 1);
}

// n rows of `stride` elements of es bytes, `cols` used.
inline Span matrix(const void *p, int64_t n, int64_t cols, int64_t stride, int es)
{
    return {p, n > 0 ? ((n - 1) * stride + cols) * es : 0, es};
}

// n elements of es bytes (p NULL: none).
inline Span vec(const void *p, int64_t n, int es) { return {p, p ? n * es : 0, es}; }

inline bool overlaps(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0)
        return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// The outputs must be aligned and apart from each other and from the inputs.
inline zero_status check_spans(const Span *in, int n_in, const Span *out, int n_out)
{
    for (int i = 0; i < n_in; ++i)
        if ((uintptr_t)in[i].p % (uintptr_t)in[i].align)
            return ZERO_EALIGN;
    for (int i = 0; i < n_out; ++i)
        if ((uintptr_t)out[i].p % (uintptr_t)out[i].align)
            return ZERO_EALIGN;
    for (int i = 0; i < n_out; ++i) {
        for (int k = 0; k < n_in; ++k)
            if (overlaps(out[i], in[k]))
                return ZERO_EINVAL;
        for (int k = 0; k < i; ++k)
            if (overlaps(out[i], out[k]))
                return ZERO_EINVAL;
    }
    return ZERO_OK;
}

// A workspace that the call needs `bytes` of.
inline zero_status check_workspace_bytes(const void *ws, size_t have, int64_t bytes)
{
    if (bytes == 0)
        return ZERO_OK;
    if (!ws)
        return ZERO_EINVAL;
    if ((uintptr_t)ws % 16)
        return ZERO_EALIGN;
    return have < (size_t)bytes ? ZERO_ENOSPC : ZERO_OK;
}

// The status of a launch.
inline zero_status done(int e, const char *where) { return e == hipSuccess ? ZERO_OK : hip_fail(e, where); }

inline int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }

}  // namespace zero
