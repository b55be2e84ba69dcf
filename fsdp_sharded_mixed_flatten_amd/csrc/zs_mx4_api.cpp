// Host side of the microscaled 4-bit format: argument validation. As in
// zs_api.cpp every argument is checked before anything is enqueued.
#include <cstdint>

#include "zs_checks.h"
#include "zs_mx4_internal.h"

namespace {

using namespace zs;

constexpr int64_t kMaxMx4Rows = int64_t(1) << 25;
constexpr int64_t kMaxMx4Cols = int64_t(1) << 34;
// Columns of a product: blocks and bytes of a row are counted in int32.
constexpr int64_t kMaxMx4In = int64_t(1) << 29;

int64_t blocks_of(int64_t cols) { return (cols + ZS_MX4_BLOCK - 1) / ZS_MX4_BLOCK; }

zs_status check_rows(int64_t rows, const char* what) {
    if (rows < 0 || rows > kMaxMx4Rows)
        return report(ZS_EINVAL, "%s = %lld outside [0, 2^25]", what, (long long)rows);
    return ZS_OK;
}

// Strides alone: they are checked for empty matrices too.
zs_status check_mx4_strides(int64_t rows, int64_t cols, int64_t code_stride, int64_t scale_stride,
                            const char* code_what, const char* scale_what) {
    const int64_t n = blocks_of(cols);
    if (zs_status st = check_extent(rows, 16 * n, code_stride, code_what)) return st;
    if (code_stride % 16)
        return report(ZS_EALIGN, "%s = %lld is not a multiple of 16", code_what, (long long)code_stride);
    return check_extent(rows, n, scale_stride, scale_what);
}

struct Mx4Spans {
    Span codes, scales;
};

Mx4Spans mx4_spans(const void* codes, int64_t code_stride, const void* scales, int64_t scale_stride, int64_t rows,
                   int64_t cols) {
    const int64_t n = blocks_of(cols);
    return {matrix_span(codes, rows, 16 * n, code_stride, 1), matrix_span(scales, rows, n, scale_stride, 1)};
}

// What quantize and dequantize share.
zs_status check_conversion(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride,
                           const void* codes, int64_t code_stride, const void* scales, int64_t scale_stride) {
    if (zs_status st = check_dtype(dtype, "dtype")) return st;
    if (zs_status st = check_rows(rows, "rows")) return st;
    if (cols < 0 || cols > kMaxMx4Cols) return report(ZS_EINVAL, "cols = %lld outside [0, 2^34]", (long long)cols);
    if (zs_status st = check_extent(rows, cols, x_stride, "x_stride")) return st;
    if (zs_status st = check_mx4_strides(rows, cols, code_stride, scale_stride, "codes_stride", "scales_stride"))
        return st;
    if (rows == 0 || cols == 0) return ZS_OK;
    if (zs_status st = check_array(x, (uintptr_t)elem_bytes(dtype), "x")) return st;
    if (zs_status st = check_array(codes, 16, "codes")) return st;
    if (zs_status st = check_array(scales, 1, "scales")) return st;
    const Span xs = matrix_span(x, rows, cols, x_stride, elem_bytes(dtype));
    const Mx4Spans q = mx4_spans(codes, code_stride, scales, scale_stride, rows, cols);
    if (zs_status st = check_apart(xs, q.codes, "x", "codes")) return st;
    return check_apart(xs, q.scales, "x", "scales");
}

}  // namespace

extern "C" {

zs_status zs_mx4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride, void* codes,
                          int64_t codes_stride, void* scales, int64_t scales_stride, void* stream) {
    if (zs_status st = check_conversion(x, dtype, rows, cols, x_stride, codes, codes_stride, scales, scales_stride))
        return st;
    if (rows == 0 || cols == 0) return ZS_OK;
    const Mx4Spans q = mx4_spans(codes, codes_stride, scales, scales_stride, rows, cols);
    if (zs_status st = check_apart(q.codes, q.scales, "codes", "scales")) return st;
    trace_call("zs_mx4_quantize", nullptr, 0, 0, rows * cols, stream);
    return report_hip(launch_mx4_quantize(Rows{x, x_stride}, dtype, rows, cols,
                                          Mx4{codes, scales, codes_stride, scales_stride}, stream),
                      "4-bit quantization launch");
}

zs_status zs_mx4_dequantize(const void* codes, int64_t codes_stride, const void* scales, int64_t scales_stride,
                            int64_t rows, int64_t cols, void* x, int32_t dtype, int64_t x_stride, void* stream) {
    if (zs_status st = check_conversion(x, dtype, rows, cols, x_stride, codes, codes_stride, scales, scales_stride))
        return st;
    if (rows == 0 || cols == 0) return ZS_OK;
    trace_call("zs_mx4_dequantize", nullptr, 0, 0, rows * cols, stream);
    return report_hip(launch_mx4_dequantize(Mx4{codes, scales, codes_stride, scales_stride}, rows, cols,
                                            Rows{x, x_stride}, dtype, stream),
                      "4-bit decoding launch");
}

zs_status zs_mx4_matmul(const void* x_codes, int64_t x_codes_stride, const void* x_scales, int64_t x_scales_stride,
                        int64_t rows, const void* w_codes, int64_t w_codes_stride, const void* w_scales,
                        int64_t w_scales_stride, int64_t out_features, int64_t in_features, void* y, int32_t y_dtype,
                        int64_t y_stride, void* stream) {
    if (zs_status st = check_dtype(y_dtype, "y_dtype")) return st;
    if (zs_status st = check_rows(rows, "rows")) return st;
    if (zs_status st = check_rows(out_features, "out_features")) return st;
    if (in_features < 0 || in_features > kMaxMx4In)
        return report(ZS_EINVAL, "in_features = %lld outside [0, 2^29]", (long long)in_features);
    if (zs_status st = check_mx4_strides(rows, in_features, x_codes_stride, x_scales_stride, "x_codes_stride",
                                         "x_scales_stride"))
        return st;
    if (zs_status st = check_mx4_strides(out_features, in_features, w_codes_stride, w_scales_stride, "w_codes_stride",
                                         "w_scales_stride"))
        return st;
    if (zs_status st = check_extent(rows, out_features, y_stride, "y_stride")) return st;
    if (rows == 0 || out_features == 0) return ZS_OK;
    if (zs_status st = check_array(y, (uintptr_t)elem_bytes(y_dtype), "y")) return st;
    if (in_features > 0) {
        if (zs_status st = check_array(x_codes, 16, "x_codes")) return st;
        if (zs_status st = check_array(w_codes, 16, "w_codes")) return st;
        if (zs_status st = check_array(x_scales, 1, "x_scales")) return st;
        if (zs_status st = check_array(w_scales, 1, "w_scales")) return st;
        const Span ys = matrix_span(y, rows, out_features, y_stride, elem_bytes(y_dtype));
        const Mx4Spans xs = mx4_spans(x_codes, x_codes_stride, x_scales, x_scales_stride, rows, in_features);
        const Mx4Spans ws = mx4_spans(w_codes, w_codes_stride, w_scales, w_scales_stride, out_features, in_features);
        if (zs_status st = check_apart(ys, xs.codes, "y", "x_codes")) return st;
        if (zs_status st = check_apart(ys, xs.scales, "y", "x_scales")) return st;
        if (zs_status st = check_apart(ys, ws.codes, "y", "w_codes")) return st;
        if (zs_status st = check_apart(ys, ws.scales, "y", "w_scales")) return st;
    }
    trace_call("zs_mx4_matmul", nullptr, 0, 0, rows * out_features, stream);
    return report_hip(launch_mx4_matmul(Mx4{x_codes, x_scales, x_codes_stride, x_scales_stride}, rows,
                                        Mx4{w_codes, w_scales, w_codes_stride, w_scales_stride}, out_features,
                                        blocks_of(in_features), y, y_dtype, y_stride, stream),
                      "4-bit product launch");
}

}  // extern "C"
