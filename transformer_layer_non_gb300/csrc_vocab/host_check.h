// host_check.h -- host-side argument checks of the vocabulary operators' C
// ABI: the per-thread error message, pointers, and overlapping buffers.
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/ls_ops.h"

namespace {

thread_local char g_last_error[512] = "";

ls_status fail(ls_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return st;
}

ls_status ok() {
    g_last_error[0] = '\0';
    return LS_OK;
}

ls_status from_cuda(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return ok();
    return fail(LS_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A byte range [p, p+n) of one argument.
struct Span {
    const char* name;
    const void* p;
    size_t n;
};

bool overlaps(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// No output (the workspace among them) may overlap another one or an input.
ls_status check_disjoint(const Span* outs, int nout, const Span* ins, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (overlaps(outs[i], outs[j]))
                return fail(LS_ERR_INVALID_ARGUMENT, "outputs %s and %s overlap", outs[i].name,
                            outs[j].name);
        for (int j = 0; j < nin; ++j)
            if (overlaps(outs[i], ins[j]))
                return fail(LS_ERR_INVALID_ARGUMENT, "output %s overlaps input %s", outs[i].name,
                            ins[j].name);
    }
    return LS_OK;
}

ls_status check_ptr(const void* p, const char* name, bool required) {
    if (!p) {
        if (required) return fail(LS_ERR_INVALID_ARGUMENT, "%s is NULL", name);
        return LS_OK;
    }
    if (!aligned16(p)) return fail(LS_ERR_MISALIGNED, "%s is not 16-byte aligned", name);
    return LS_OK;
}

#define LS_TRY(expr)                         \
    do {                                     \
        ls_status _st = (expr);              \
        if (_st != LS_OK) return _st;        \
    } while (0)

}  // namespace
