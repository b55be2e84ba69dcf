// Kernel launchers of the microscaled 4-bit format (zs_mx4.h) and what its host
// file and kernels share. Not part of the public ABI.
#pragma once

#include <cstdint>

#include "../../include/zs_mx4.h"
#include "zs_lm_internal.h"

namespace zs {

// A quantized matrix in device memory: rows start code_stride and scale_stride
// bytes apart.
struct Mx4 {
    const void* codes;
    const void* scales;
    int64_t code_stride;
    int64_t scale_stride;
};

// Launchers; they return a hipError_t value cast to int.
int launch_mx4_quantize(Rows x, int dtype, int64_t rows, int64_t cols, const Mx4& out, void* stream);
int launch_mx4_dequantize(const Mx4& in, int64_t rows, int64_t cols, Rows x, int dtype, void* stream);
// blocks: blocks of a row of either matrix.
int launch_mx4_matmul(const Mx4& x, int64_t rows, const Mx4& w, int64_t out_features, int64_t blocks, void* y,
                      int y_dtype, int64_t y_stride, void* stream);

}  // namespace zs
