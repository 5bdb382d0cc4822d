// Host-side checks of arguments that every C entry point shares, and the
// message of the thread's last failed call.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "sdpa_math.h"

namespace sdpa_api {

inline thread_local std::string g_last_error;

inline sdpa_status_t fail(sdpa_status_t st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

inline int64_t elt_size(int dtype) {
    switch (dtype) {
        case SDPA_F32: return 4;
        case SDPA_F16:
        case SDPA_BF16: return 2;
        case SDPA_BOOL:
        case SDPA_E4M3: return 1;
        default: return 0;
    }
}

inline const char* dtype_name(int dtype) {
    switch (dtype) {
        case SDPA_F32: return "f32";
        case SDPA_F16: return "f16";
        case SDPA_BF16: return "bf16";
        case SDPA_BOOL: return "bool";
        case SDPA_E4M3: return "e4m3";
        default: return "?";
    }
}

inline int64_t numel(const sdpa_tensor_t* t) {
    int64_t n = 1;
    for (int d = 0; d < t->ndim; ++d) n *= t->sizes[d];
    return n;
}

// Effective stride: a size-1 dim never advances, whatever stride it carries.
inline int64_t eff_stride(const sdpa_tensor_t* t, int d) { return t->sizes[d] == 1 ? 0 : t->strides[d]; }

// True when every row start (all dims but the last) is `align`-byte aligned.
inline bool rows_aligned(const sdpa_tensor_t* t, int64_t align) {
    const int64_t es = elt_size(t->dtype);
    if (reinterpret_cast<uintptr_t>(t->data) % align) return false;
    for (int d = 0; d + 1 < t->ndim; ++d)
        if ((eff_stride(t, d) * es) % align) return false;
    return true;
}

inline sdpa_status_t check_tensor(const sdpa_tensor_t* t, const char* name, int ndim) {
    if (!t) return fail(SDPA_ERR_INVALID_ARG, "%s is NULL", name);
    if (t->ndim != ndim) return fail(SDPA_ERR_INVALID_ARG, "%s must have %d dims, got %d", name, ndim, t->ndim);
    for (int d = 0; d < ndim; ++d)
        if (t->sizes[d] < 0) return fail(SDPA_ERR_INVALID_ARG, "%s has a negative size", name);
    if (elt_size(t->dtype) == 0) return fail(SDPA_ERR_INVALID_ARG, "%s has an unknown dtype %d", name, t->dtype);
    if (numel(t) > 0 && t->data == nullptr) return fail(SDPA_ERR_INVALID_ARG, "%s has no data pointer", name);
    if (numel(t) > 0 && t->sizes[ndim - 1] > 1 && t->strides[ndim - 1] != 1)
        return fail(SDPA_ERR_UNSUPPORTED, "%s must be contiguous in its last dim (stride %lld)", name,
                    (long long)t->strides[ndim - 1]);
    return SDPA_OK;
}

inline sdpa_status_t check_dims(const sdpa_tensor_t* t, const char* name, const int64_t* want, int ndim) {
    for (int d = 0; d < ndim; ++d)
        if (t->sizes[d] != want[d]) {
            return fail(SDPA_ERR_INVALID_ARG, "%s dim %d is %lld, expected %lld", name, d, (long long)t->sizes[d],
                        (long long)want[d]);
        }
    return SDPA_OK;
}

// Byte extent of one (batch, head) slice: `rows` rows of `cols` elements at
// a row pitch of `pitch` elements (0 rows: 0).
inline int64_t slice_extent(int64_t rows, int64_t pitch, int64_t cols, int64_t es) {
    return rows > 0 && cols > 0 ? ((rows - 1) * pitch + cols) * es : 0;
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace sdpa_api
