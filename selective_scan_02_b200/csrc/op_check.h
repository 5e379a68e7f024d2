// op_check.h -- host-side argument checks shared by the operators' C entry points (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "api_internal.h"

namespace ss2d {

// Sets the calling thread's error text and returns `status`.
inline int op_fail(int status, const char *fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return set_last_error(status, msg);
}

inline int op_cuda_fail(cudaError_t e, const char *what)
{
    return op_fail(SS2D_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

struct OpSpan {
    const char *name;
    const void *p;  // nullptr: an optional tensor that is not given
    size_t bytes;
    unsigned align = 16;  // 4 for what is accessed one number at a time
};

inline bool op_overlaps(const OpSpan &a, const OpSpan &b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Checks of one call's tensors: the alignment of every one, then no output overlapping an
// input or another output.  Returns SS2D_OK or the status, with the error text set.
inline int op_check_tensors(const char *call, const OpSpan *in, int n_in, const OpSpan *out, int n_out)
{
    for (int i = 0; i < n_in + n_out; ++i) {
        const OpSpan &t = i < n_in ? in[i] : out[i - n_in];
        if (reinterpret_cast<uintptr_t>(t.p) & (t.align - 1))
            return op_fail(SS2D_ERR_MISALIGNED, "%s: %s must be %u-byte aligned", call, t.name, t.align);
    }
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (op_overlaps(out[o], in[i]))
                return op_fail(SS2D_ERR_INVALID_ARG, "%s: %s overlaps %s", call, out[o].name, in[i].name);
        for (int i = 0; i < o; ++i)
            if (op_overlaps(out[o], out[i]))
                return op_fail(SS2D_ERR_INVALID_ARG, "%s: %s overlaps %s", call, out[o].name, out[i].name);
    }
    return SS2D_OK;
}

}  // namespace ss2d
