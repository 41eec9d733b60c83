// host_check.h -- host-side argument checks of the C ABIs of the vocabulary
// and the block operators: the per-thread error message, types, sizes, pointers,
// workspaces, and overlapping buffers.
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

size_t elem_size(ls_dtype dt) { return dt == LS_F32 ? 4 : 2; }

ls_status check_storage(const char* fn, ls_dtype dt, bool f32_too) {
    if (dt == LS_F16 || dt == LS_BF16 || (dt == LS_F32 && f32_too)) return LS_OK;
    return fail(LS_ERR_INVALID_ARGUMENT, "%s: unsupported storage dtype %d", fn,
                static_cast<int>(dt));
}

ls_status check_ptr_n(const void* p, const char* name, bool required, size_t bytes) {
    if (!p) {
        if (required) return fail(LS_ERR_INVALID_ARGUMENT, "%s is NULL", name);
        return LS_OK;
    }
    if (reinterpret_cast<uintptr_t>(p) & (bytes - 1))
        return fail(LS_ERR_MISALIGNED, "%s is not %zu-byte aligned", name, bytes);
    return LS_OK;
}

ls_status check_ptr4(const void* p, const char* name, bool required) {
    return check_ptr_n(p, name, required, 4);
}

// A size in [lo, hi].
ls_status check_size(const char* fn, const char* name, int64_t v, int64_t lo, int64_t hi) {
    if (v < lo)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: %s = %lld < %lld", fn, name, (long long)v,
                    (long long)lo);
    if (v > hi)
        return fail(LS_ERR_UNSUPPORTED_SHAPE, "%s: %s = %lld exceeds %lld", fn, name, (long long)v,
                    (long long)hi);
    return LS_OK;
}

ls_status check_multiple_of_8(const char* fn, const char* name, int64_t v) {
    if (v % 8 != 0)
        return fail(LS_ERR_MISALIGNED, "%s: %s = %lld is not a multiple of 8", fn, name,
                    (long long)v);
    return LS_OK;
}

ls_status check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
    if (need == 0) return LS_OK;
    if (!ws) return fail(LS_ERR_INVALID_ARGUMENT, "%s: workspace is NULL", fn);
    if (!aligned16(ws)) return fail(LS_ERR_MISALIGNED, "workspace is not 16-byte aligned");
    if (have < need)
        return fail(LS_ERR_WORKSPACE_TOO_SMALL, "%s: workspace has %zu bytes, needs %zu", fn, have,
                    need);
    return LS_OK;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace
