// Products of a few rows with a weight matrix in the quantized gather's
// payload, for CDNA4 (gfx950):
//   y[r, o] = sum over i of code[o, i] * scale[o, i] * x[r, i].
//
// The payload is read once: bits/8 + 4/block bytes a weight against
// 2 * rows flops, so up to some tens of rows the product is an HBM stream and
// what has to be kept short is the arithmetic beside each load.
#include <hip/hip_runtime.h>

#include "zs_lm_internal.h"

namespace zs {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any address that is a multiple of the element's size (the
// hardware takes unaligned vector loads).
typedef u32x4 __attribute__((aligned(2))) u32x4_u2;

__device__ __forceinline__ float bf16_f32(uint32_t h) { return __uint_as_float(h << 16); }

// Round to nearest even, the only rounding of a result; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    const uint32_t r = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
    return (uint16_t)(((u & 0x7FFFFFFFu) > 0x7F800000u) ? ((u >> 16) | 0x40u) : r);
}

__device__ __forceinline__ void store_y(void* y, bool bf16, int64_t i, float v) {
    if (bf16)
        static_cast<uint16_t*>(y)[i] = f32_bf16(v);
    else
        static_cast<float*>(y)[i] = v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// ------------------------------------------------------------------ any layout
// One wave per row of W and M rows of x. The wave walks the row in units of 8
// elements of the flat buffer that start at multiples of 8: a unit never
// crosses a shard (S is a multiple of 8) or a block (blocks start at multiples
// of 8 of a shard), so it has one scale and its codes are one aligned 32- or
// 64-bit word. The units at the row's ends may reach into the neighbouring
// tensors; their elements there are left out.
constexpr int kAnyWaves = 4;

template <int BITS, int M>
__global__ __launch_bounds__(64 * kAnyWaves) void k_matvec_any(QuantWeight w, const uint16_t* __restrict__ x,
                                                              int64_t x_stride, int rows, void* __restrict__ y,
                                                              int y_bf16, int64_t y_stride) {
    const int lane = threadIdx.x & 63;
    const int64_t o = (int64_t)blockIdx.x * kAnyWaves + (threadIdx.x >> 6);
    const int r0 = blockIdx.y * M;
    if (o >= w.n_out) return;
    const int64_t j0 = w.off + o * w.n_in;
    const int64_t u_end = w.n_in > 0 ? (j0 + w.n_in + 7) >> 3 : 0;
    const int64_t q0 = w.n_in > 0 ? j0 / w.shard : 0;
    float acc[M];
#pragma unroll
    for (int m = 0; m < M; ++m) acc[m] = 0.0f;
    for (int64_t u = (j0 >> 3) + lane; u < u_end; u += 64) {
        int64_t q = q0, s = u * 8 - q0 * w.shard;
        while (s >= w.shard) {
            s -= w.shard;
            ++q;
        }
        const float scale = w.scales[q * w.n_scales + (s >> w.block_shift)];
        float c[8];
        if (BITS == 4) {
            const uint32_t d = static_cast<const uint32_t*>(w.codes)[u];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = (float)((int32_t)(d << (28 - 4 * i)) >> 28);
        } else {
            const uint2 d = static_cast<const uint2*>(w.codes)[u];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = (float)(int8_t)((i < 4 ? d.x : d.y) >> (8 * (i & 3)));
        }
        const int64_t i0 = u * 8 - j0;  // the unit's first column, negative at a row's unaligned start
        if (i0 >= 0 && i0 + 8 <= w.n_in) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (r0 + m >= rows) break;
                const u32x4 v = *reinterpret_cast<const u32x4_u2*>(x + (r0 + m) * x_stride + i0);
                float p = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p = __builtin_fmaf(c[2 * i], bf16_f32(v[i] & 0xFFFFu), p);
                    p = __builtin_fmaf(c[2 * i + 1], __uint_as_float(v[i] & 0xFFFF0000u), p);
                }
                acc[m] = __builtin_fmaf(p, scale, acc[m]);
            }
        } else {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (r0 + m >= rows) break;
                float p = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i0 + i >= 0 && i0 + i < w.n_in)
                        p = __builtin_fmaf(c[i], bf16_f32(x[(r0 + m) * x_stride + i0 + i]), p);
                acc[m] = __builtin_fmaf(p, scale, acc[m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const float v = wave_sum(acc[m]);
        if (lane == 0 && r0 + m < rows) store_y(y, y_bf16, (r0 + m) * y_stride + o, v);
    }
}

template <int BITS>
void run_any(const QuantWeight& w, Rows x, int rows, void* y, bool y_bf16, int64_t y_stride, hipStream_t s) {
    const unsigned gx = (unsigned)((w.n_out + kAnyWaves - 1) / kAnyWaves);
    const uint16_t* xp = static_cast<const uint16_t*>(x.p);
    if (rows == 1)
        hipLaunchKernelGGL((k_matvec_any<BITS, 1>), dim3(gx, 1), dim3(64 * kAnyWaves), 0, s, w, xp, x.stride, rows, y,
                           (int)y_bf16, y_stride);
    else
        hipLaunchKernelGGL((k_matvec_any<BITS, 4>), dim3(gx, (unsigned)((rows + 3) / 4)), dim3(64 * kAnyWaves), 0, s,
                           w, xp, x.stride, rows, y, (int)y_bf16, y_stride);
}

}  // namespace

int launch_quant_matvec(const QuantWeight& w, Rows x, int rows, void* y, int y_dtype, int64_t y_stride,
                        void* stream) {
    if (w.n_out > (int64_t)kAnyWaves * ((1 << 24) - 1)) return (int)hipErrorInvalidValue;  // 2^32 - 1 work-items
    const bool y_bf16 = y_dtype == ZS_DTYPE_BF16;
    if (w.bits == 4)
        run_any<4>(w, x, rows, y, y_bf16, y_stride, (hipStream_t)stream);
    else
        run_any<8>(w, x, rows, y, y_bf16, y_stride, (hipStream_t)stream);
    return (int)hipGetLastError();
}

}  // namespace zs
