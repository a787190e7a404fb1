// Argument checks shared by the operators' C ABI files: host only, before any HIP call.  Each sets
// the calling thread's la_last_error and returns the status.
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "la_layer.hpp"

namespace {

la_status fail(la_status s, const char* fmt, ...) {
    char text[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return la::report(s, text);
}
la_status ok() { return la::report(LA_OK, ""); }

la_status done(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(LA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

#define CHECK(expr)                 \
    do {                            \
        la_status s_ = (expr);      \
        if (s_ != LA_OK) return s_; \
    } while (0)

la_status check_ptr(const void* p, const char* name, bool required) {
    if (!p) return required ? fail(LA_ERR_INVALID_ARG, "%s is NULL", name) : LA_OK;
    if (reinterpret_cast<uintptr_t>(p) & 15u) return fail(LA_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
    return LA_OK;
}

la_status check_dtype(int dt, const char* name) {
    if (dt != LA_F32 && dt != LA_BF16) return fail(LA_ERR_INVALID_ARG, "unknown %s %d", name, dt);
    return LA_OK;
}

// A row stride: 0 or at least the row, a multiple of 16 bytes.
la_status check_ld(int ld, int64_t width, int dtype, const char* name) {
    const int es = dtype == LA_BF16 ? 2 : 4;
    if (width > INT32_MAX) return fail(LA_ERR_UNSUPPORTED, "%s: a row of %lld elements is too long", name, static_cast<long long>(width));
    if (ld == 0) return LA_OK;
    if (ld < width) return fail(LA_ERR_INVALID_ARG, "%s = %d is shorter than the row (%lld)", name, ld, static_cast<long long>(width));
    if (static_cast<int64_t>(ld) * es % 16 != 0)
        return fail(LA_ERR_ALIGNMENT, "%s = %d is not a multiple of 16 bytes", name, ld);
    return LA_OK;
}

la_status check_workspace(const void* ws, size_t given, size_t need) {
    CHECK(check_ptr(ws, "workspace", false));
    if (need > 0 && (!ws || given < need))
        return fail(LA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? given : static_cast<size_t>(0));
    return LA_OK;
}

// A row's codec: la_norm_config's qdq and group for rows of d columns.
la_status check_codec(int qdq, int group, int d) {
    if (qdq == LA_QDQ_NONE) return LA_OK;
    if (qdq != LA_QDQ_INT8_GROUP && qdq != LA_QDQ_E4M3_TILE)
        return fail(LA_ERR_INVALID_ARG, "unknown qdq mode %d", qdq);
    if (group != 0 && group != 16 && group != 32 && group != 64 && group != 128)
        return fail(LA_ERR_UNSUPPORTED, "group must be 0 (the row), 16, 32, 64 or 128 (group=%d)", group);
    if (group != 0 && d % group != 0)
        return fail(LA_ERR_INVALID_ARG, "group must divide d (d=%d group=%d)", d, group);
    return LA_OK;
}

}  // namespace
