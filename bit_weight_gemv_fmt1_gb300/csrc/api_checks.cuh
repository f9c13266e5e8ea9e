// api_checks.cuh -- argument checks shared by the attention entry points (mla_api.cu, gqa_api.cu).
#pragma once

#include <cstdarg>
#include <cstdio>

#include "coli_internal.cuh"

namespace coli {
namespace {

int bad(int code, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_last_error(code, buf);
}

int launched(cudaError_t e, const char *what, int n) {
    if (e != cudaSuccess)
        return bad(e == cudaErrorMemoryAllocation ? COLI_ENOMEM : COLI_ECUDA, "%s: %s", what, cudaGetErrorString(e));
    count_call(n, 0);
    return COLI_OK;
}

int need(const void *p, uintptr_t align, const char *name) {
    if (!p) return bad(COLI_EINVAL, "%s is NULL", name);
    if ((uintptr_t)p & (align - 1)) return bad(COLI_EINVAL, "%s is not %d-byte aligned", name, (int)align);
    return COLI_OK;
}

int float_type(int dtype, const char *name) {
    if (dtype != COLI_F32 && dtype != COLI_BF16) return bad(COLI_EFMT, "%s must be COLI_F32 or COLI_BF16 (got %d)", name, dtype);
    return COLI_OK;
}

// No C++ exception leaves the library.
template <class F>
int guarded(F f) {
    try {
        return f();
    } catch (...) {
        return set_last_error(COLI_ENOMEM, "out of host memory");
    }
}

}  // namespace
}  // namespace coli
