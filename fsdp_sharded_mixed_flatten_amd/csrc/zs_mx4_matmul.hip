// Products of two matrices in microscaled 4-bit floating point, for CDNA4
// (gfx950):
//   y[r, o] = sum over blocks b of 2^(ex[r,b] + ew[o,b]) * sum over i in b of cx[r, i] * cw[o, i].
//
// The matrix instructions take codes and scales as they are stored: a lane gives
// the 32 codes (16 bytes) of one row's block and that block's scale byte.
#include <hip/hip_runtime.h>

#include "zs_mx4_internal.h"

namespace zs {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 scale bytes at any address (the hardware takes unaligned vector loads).
typedef u32x4 __attribute__((aligned(1))) u32x4_u1;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // the matrix instructions' name of the format

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

// 16 x 16 products of 128 columns. Lane l gives block l / 16 of row l % 16 of
// either side and has rows 4 * (l / 16) .. + 3 of x and column l % 16 of y.
__device__ __forceinline__ f32x4 mfma16(const u32x4& x, uint32_t sx, const u32x4& w, uint32_t sw, f32x4 acc) {
    const i32x8 a{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    const i32x8 b{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, kFp4, kFp4, 0, (int)sx, 0, (int)sw);
}

// ------------------------------------------------------------------ any size
// A workgroup computes 16 x 16 results; its waves take turns of 512 columns (16
// blocks of either side, four matrix instructions) and add up through shared
// memory.
constexpr int kFewWaves = 8;

struct Turn {
    u32x4 codes[4];
    u32x4 scales;
};

// A lane's part of a turn: block 4s + lane / 16 of the turn for step s.
__device__ __forceinline__ Turn load_turn(const char* codes, const uint8_t* scales, int first, int group) {
    Turn t;
#pragma unroll
    for (int s = 0; s < 4; ++s)
        t.codes[s] = *reinterpret_cast<const u32x4*>(codes + (int64_t)(first + 4 * s + group) * 16);
    t.scales = *reinterpret_cast<const u32x4_u1*>(scales + first);
    return t;
}

__global__ __launch_bounds__(64 * kFewWaves) void k_mx4_few(Mx4 x, int64_t rows, Mx4 w, int64_t out, int blocks,
                                                            void* __restrict__ y, int y_bf16, int64_t y_stride) {
    __shared__ float part[kFewWaves][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, group = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.y * 16, o0 = (int64_t)blockIdx.x * 16;
    // rows past the end repeat the last one; their results are not stored
    const int64_t r = r0 + (lane & 15) < rows ? r0 + (lane & 15) : rows - 1;
    const int64_t o = o0 + (lane & 15) < out ? o0 + (lane & 15) : out - 1;
    const char* xc = static_cast<const char*>(x.codes) + r * x.code_stride;
    const char* wc = static_cast<const char*>(w.codes) + o * w.code_stride;
    const uint8_t* xs = static_cast<const uint8_t*>(x.scales) + r * x.scale_stride;
    const uint8_t* ws = static_cast<const uint8_t*>(w.scales) + o * w.scale_stride;
    f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    const int whole = blocks / 16;
    for (int t = wave; t < whole; t += kFewWaves) {
        const Turn a = load_turn(xc, xs, t * 16, group), b = load_turn(wc, ws, t * 16, group);
#pragma unroll
        for (int s = 0; s < 4; ++s)
            acc = mfma16(a.codes[s], a.scales[s] >> (8 * group), b.codes[s], b.scales[s] >> (8 * group), acc);
    }
    // the rest, block by block: what lies behind the last is 0 with scale 1
    if (wave == whole % kFewWaves) {
        for (int s = whole * 16; s < blocks; s += 4) {
            u32x4 a{0, 0, 0, 0}, b{0, 0, 0, 0};
            uint32_t sa = 127, sb = 127;
            if (s + group < blocks) {
                a = *reinterpret_cast<const u32x4*>(xc + (int64_t)(s + group) * 16);
                b = *reinterpret_cast<const u32x4*>(wc + (int64_t)(s + group) * 16);
                sa = xs[s + group];
                sb = ws[s + group];
            }
            acc = mfma16(a, sa, b, sb, acc);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    if (threadIdx.x < 256) {
        const int i = threadIdx.x >> 6;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kFewWaves; ++k) sum += part[k][i][lane];
        const int64_t row = r0 + 4 * group + i, col = o0 + (lane & 15);
        if (row < rows && col < out) store_y(y, y_bf16, row * y_stride + col, sum);
    }
}

}  // namespace

int launch_mx4_matmul(const Mx4& x, int64_t rows, const Mx4& w, int64_t out_features, int64_t blocks, void* y,
                      int y_dtype, int64_t y_stride, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int esz = y_dtype == ZS_DTYPE_BF16 ? 2 : 4;
    // a launch covers at most 2^32 - 1 work-items and 65535 tiles of rows
    const int64_t tiles = (out_features + 15) / 16;
    const int64_t fit = ((int64_t(1) << 32) - 1) / (tiles * 64 * kFewWaves);
    const int64_t most = 16 * (fit < 1 ? 1 : fit > 65535 ? 65535 : fit);
    for (int64_t lo = 0; lo < rows; lo += most) {
        const int64_t n = rows - lo < most ? rows - lo : most;
        const Mx4 part{static_cast<const char*>(x.codes) + lo * x.code_stride,
                       static_cast<const char*>(x.scales) + lo * x.scale_stride, x.code_stride, x.scale_stride};
        k_mx4_few<<<dim3((unsigned)tiles, (unsigned)((n + 15) / 16)), 64 * kFewWaves, 0, s>>>(
            part, n, w, out_features, (int)blocks, static_cast<char*>(y) + lo * y_stride * esz,
            y_dtype == ZS_DTYPE_BF16, y_stride);
        if (hipError_t e = hipGetLastError()) return (int)e;
    }
    return 0;
}

}  // namespace zs
