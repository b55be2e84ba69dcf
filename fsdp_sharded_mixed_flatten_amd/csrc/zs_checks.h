// Argument checks that the operators' host files share (zs_lm_api.cpp,
// zs_mx4_api.cpp, zs_drafts_api.cpp, zs_clip_api.cpp). Not part of the public ABI.
#pragma once

#include <cstdint>

#include "zs_lm_internal.h"

namespace zs {

constexpr int64_t kMaxVocab = int64_t(1) << 30;
// Rows of one call: a launch covers at most 2^32 - 1 work-items and a row
// takes up to 1024 of them.
constexpr int64_t kMaxRows = (int64_t(1) << 22) - 1;
// Largest row stride: 2^22 rows of 4-byte elements that far apart span 2^62
// bytes, inside int64.
constexpr int64_t kMaxStride = int64_t(1) << 38;

inline int64_t elem_bytes(int32_t dtype) { return dtype == ZS_DTYPE_BF16 ? 2 : 4; }

inline zs_status check_dtype(int32_t dtype, const char* what) {
    if (dtype != ZS_DTYPE_BF16 && dtype != ZS_DTYPE_F32)
        return report(ZS_EINVAL, "%s = %d is neither ZS_DTYPE_BF16 nor ZS_DTYPE_F32", what, dtype);
    return ZS_OK;
}

inline zs_status check_array(const void* p, uintptr_t align, const char* what) {
    if (!p) return report(ZS_EINVAL, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % align)
        return report(ZS_EALIGN, "%s (%p) is not %d-byte aligned", what, p, (int)align);
    return ZS_OK;
}

inline zs_status check_opt_array(const void* p, uintptr_t align, const char* what) {
    return p ? check_array(p, align, what) : ZS_OK;
}

inline zs_status check_stride(int64_t stride, int64_t cols, const char* what) {
    if (stride < cols || stride > kMaxStride)
        return report(ZS_EINVAL, "%s = %lld outside [%lld, 2^38]", what, (long long)stride, (long long)cols);
    return ZS_OK;
}

// A matrix of many rows: its extent stays inside 2^60 elements.
inline zs_status check_extent(int64_t rows, int64_t cols, int64_t stride, const char* what) {
    if (zs_status st = check_stride(stride, cols, what)) return st;
    if (rows > 1 && stride > ((int64_t(1) << 60) - cols) / (rows - 1))
        return report(ZS_EINVAL, "%s = %lld: %lld rows that far apart pass 2^60", what, (long long)stride,
                      (long long)rows);
    return ZS_OK;
}

// The bytes of a matrix (or, as one row, of an array): [lo, lo + row), again
// every `stride` bytes, up to hi. Empty where lo == hi.
struct Span {
    uintptr_t lo, hi;
    uintptr_t row, stride;  // stride 0: one row
};

inline Span span(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), n = p ? (uintptr_t)bytes : 0;
    return Span{a, a + n, n, 0};
}

inline Span matrix_span(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t esz) {
    if (rows <= 1 || cols == 0) return span(p, rows > 0 ? cols * esz : 0);
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + (uintptr_t)(((rows - 1) * stride + cols) * esz), (uintptr_t)(cols * esz),
                (uintptr_t)(stride * esz)};
}

// Whether no byte belongs to both. Exact for rows that repeat at one distance
// (columns of one matrix side by side, an array between two rows); matrices of
// different strides have to lie in ranges apart.
inline bool apart(const Span& a, const Span& b) {
    if (!(a.lo < b.hi && b.lo < a.hi)) return true;
    const uintptr_t stride = a.stride ? a.stride : b.stride;
    if (stride == 0 || (b.stride && b.stride != stride)) return false;
    // how far b's rows start behind a's, modulo the stride
    const uintptr_t d = b.lo >= a.lo ? (b.lo - a.lo) % stride : (stride - (a.lo - b.lo) % stride) % stride;
    return d >= a.row && b.row <= stride - d;
}

inline zs_status check_apart(const Span& a, const Span& b, const char* what_a, const char* what_b) {
    if (!apart(a, b)) return report(ZS_EINVAL, "%s overlaps %s", what_a, what_b);
    return ZS_OK;
}

// float or double, as the call takes it.
template <typename T>
zs_status check_temperature(T t) {
    if (!(t >= T(1e-6) && t <= T(1e6))) return report(ZS_EINVAL, "temperature = %g outside [1e-6, 1e6]", (double)t);
    return ZS_OK;
}

}  // namespace zs
