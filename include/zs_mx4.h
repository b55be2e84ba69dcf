/*
 * zs_mx4.h -- microscaled 4-bit floating point beside the shard-local step
 * (zs.h): the format that gfx950's matrix instructions multiply directly, for
 * gathered parameters and for activations.
 *
 *   zs_mx4_quantize    a matrix (or a shard, as one row) to codes and scales
 *   zs_mx4_dequantize  and back
 *   zs_mx4_matmul      the product of two quantized matrices, one row to many
 *
 * Format. A row is cut into blocks of ZS_MX4_BLOCK (32) consecutive elements,
 * its last block filled up with zeros. An element is a 4-bit code: sign, two
 * bits of exponent, one of mantissa, that is +-0, 0.5, 1, 1.5, 2, 3, 4 or 6;
 * two a byte, the even element in the low half, 16 bytes a block. A block has
 * one scale byte s that stands for 2^(s - 127); 255 stands for NaN. An
 * element's value is its code's times its block's scale.
 * codes rows start codes_stride bytes apart (a multiple of 16, at least 16 a
 * block) and are 16-byte aligned; scales rows start scales_stride bytes apart
 * (at least one a block), at any address. x and y are as in zs_lm.h: rows
 * `stride` elements apart, aligned to their elements; what lies between rows
 * is neither read nor written. Strides are at most 2^38, and no matrix spans
 * more than 2^60 elements.
 *
 * As payload of the parameter gather: zs_mx4_quantize of a bf16 shard as one
 * row of S elements gives a rank's codes (S/2 bytes) and scales (S/32). Where
 * the plan is FLAT and S is a multiple of 32, the ranks' payloads end to end
 * are the payload of the whole flat buffer, and tensor i whose offset off and
 * row length `in` are multiples of 32 is the matrix whose codes start at byte
 * off/2 with a stride of in/2 and whose scales start at byte off/32 with a
 * stride of in/32.
 *
 * Conventions are those of zs_lm.h: caller-owned device memory, no workspace,
 * no allocation, arguments validated on the host before anything is enqueued,
 * no synchronization, zs_last_error(), one ZS_LOG trace line a call, equal
 * inputs give equal bits, every call may be captured into a HIP graph.
 */
#ifndef ZS_MX4_H
#define ZS_MX4_H

#include "zs_lm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Elements of one block. */
#define ZS_MX4_BLOCK 32

/* Codes and scales of x (rows x cols of dtype). Per block, with amax the
 * largest magnitude in it: the scale's exponent is floor(log2 amax) - 2, at
 * least -127 (amax = 0: -127); a code is the value nearest to the element over
 * the scale, ties to the code whose last bit is 0, at most 6 in magnitude,
 * with the element's sign. A block with a NaN or infinity gets scale 255 and
 * codes 0. rows <= 2^25, cols <= 2^34; rows == 0 or cols == 0 does nothing.
 * Outputs may overlap neither x nor each other. */
zs_status zs_mx4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride, void* codes,
                          int64_t codes_stride, void* scales, int64_t scales_stride, void* stream);

/* x[r, i] (rows x cols of dtype) = the value of element i of row r, which is
 * exact in either type: 6 * 2^127 and more, which no quantized matrix holds,
 * is infinite; an element of a NaN block is NaN. Limits as above; x may overlap
 * neither input. */
zs_status zs_mx4_dequantize(const void* codes, int64_t codes_stride, const void* scales, int64_t scales_stride,
                            int64_t rows, int64_t cols, void* x, int32_t dtype, int64_t x_stride, void* stream);

/* y[r, o] = sum over i of X[r, i] * W[o, i], r < rows, o < out_features, with X
 * and W the values of two quantized matrices of in_features columns each (their
 * last blocks are multiplied whole: zs_mx4_quantize fills them with zeros).
 * Products and sums are held in fp32 and y, bf16 or fp32 (y_dtype), is rounded
 * once, to the nearest, ties to even. A product X * W or a sum beyond fp32's range may be infinite, and what
 * is below fp32's normal range may be taken as 0. A NaN block gives NaN in every
 * element of y that it takes part in; zeros times anything else are zeros, under
 * any scales. Many rows are multiplied fast where the rows of both matrices' codes
 * start at most 2^22 bytes apart.
 * rows, out_features <= 2^25, in_features <= 2^29. rows == 0 or out_features
 * == 0 does nothing, in_features == 0 gives zeros. y may not overlap any
 * input; X and W may be the same matrix. */
zs_status zs_mx4_matmul(const void* x_codes, int64_t x_codes_stride, const void* x_scales, int64_t x_scales_stride,
                        int64_t rows, const void* w_codes, int64_t w_codes_stride, const void* w_scales,
                        int64_t w_scales_stride, int64_t out_features, int64_t in_features, void* y, int32_t y_dtype,
                        int64_t y_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_MX4_H */
