// Microscaled 4-bit floating point for CDNA4 (gfx950): a matrix to codes and
// scales and back.
//
// Per element 2 or 4 bytes of x and 17/32 byte of payload: HBM streams in both
// directions. The instruction set converts pairs of values to and from 4-bit
// codes under a power-of-two scale. The conversion to codes was compared with
// the definition (nearest, ties to even, at most 6, the sign kept) over all
// finite fp32 and bf16 values at the scales that a block can give them, the
// conversion back over all codes and scales: no value differs.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "zs_mx4_internal.h"

namespace zs {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any multiple of the element's size: rows of an odd stride start
// anywhere (the hardware takes unaligned vector accesses).
typedef u32x4 __attribute__((aligned(2))) u32x4_u2;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 128;  // and blocks of a workgroup

// The largest of v over each four (and eight) consecutive lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kQuadSwap1 = 0xB1, kQuadSwap2 = 0x4E;  // lanes 1 0 3 2 and 2 3 0 1 of each four
constexpr int kHalfMirror = 0x141;                   // lanes 7 .. 0 of each eight
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    v = max(v, moved<kQuadSwap1>(v));
    v = max(v, moved<kQuadSwap2>(v));
    if constexpr (LANES == 8) v = max(v, moved<kHalfMirror>(v));
    return v;
}

// The fp32 that a scale byte stands for; 2^-127 lies under the normal range.
__device__ __forceinline__ float scale_f32(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
}

// By value: a bit cast of a vector's element in place would read the first one.
__device__ __forceinline__ bf16x2 pair(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

// Sixteen bytes of x: kN elements, of which a block takes kLanes lanes.
template <typename T>
struct Elems;
template <>
struct Elems<uint16_t> {
    static constexpr int kN = 8, kLanes = 4;
    typedef uint32_t Code;  // codes of kN elements
    // bits of the largest magnitude, as fp32's
    static __device__ __forceinline__ uint32_t amax(const u32x4& v) {
        u16x2 m = __builtin_bit_cast(u16x2, v[0] & 0x7FFF7FFFu);
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
        return (uint32_t)max(m[0], m[1]) << 16;
    }
    static __device__ __forceinline__ Code encode(const u32x4& v, float s) {
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v[0]), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v[1]), s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v[2]), s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v[3]), s, 3);
        return c;
    }
    static __device__ __forceinline__ u32x4 decode(Code c, float s) {
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
    }
};
template <>
struct Elems<uint32_t> {
    static constexpr int kN = 4, kLanes = 8;
    typedef uint16_t Code;
    static __device__ __forceinline__ uint32_t amax(const u32x4& v) {
        return max(max(v[0] & 0x7FFFFFFFu, v[1] & 0x7FFFFFFFu), max(v[2] & 0x7FFFFFFFu, v[3] & 0x7FFFFFFFu));
    }
    static __device__ __forceinline__ Code encode(const u32x4& v, float s) {
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v[0]), __uint_as_float(v[1]), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v[2]), __uint_as_float(v[3]), s, 1);
        return (Code)c;
    }
    static __device__ __forceinline__ u32x4 decode(Code c, float s) {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)c, s, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)c, s, 1);
        return u32x4{__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(b[0]), __float_as_uint(b[1])};
    }
};

// Where a workgroup's blocks lie. It takes kThreads of them in order, counted
// through the rows; ONE: there is one row (or rows follow each other without a
// gap in all three arrays), so that no block has to be looked for.
template <bool ONE>
struct Place {
    int64_t row;    // the first block's row
    uint32_t first;  // and number in it (rows hold at most 2^29 blocks)
    uint32_t blocks;
    int64_t left;   // blocks from the first to the matrix's end

    __device__ __forceinline__ Place(int64_t rows, int64_t nb) {
        const int64_t id = (int64_t)blockIdx.x * kThreads;
        left = rows * nb - id;
        if constexpr (!ONE) {
            row = id / nb;
            first = (uint32_t)(id - row * nb);
            blocks = (uint32_t)nb;
        }
    }
    // block i of the workgroup's: row and number in the row
    __device__ __forceinline__ void at(int i, int64_t& r, int64_t& b) const {
        if constexpr (ONE) {
            r = 0;
            b = (int64_t)blockIdx.x * kThreads + i;
        } else {
            const uint32_t n = first + (uint32_t)i, down = n / blocks;
            r = row + down;
            b = n - down * blocks;
        }
    }
};

// A workgroup takes a block per thread, in kLanes steps of 16-byte loads that a
// thread holds together. The lanes of a block agree on the largest magnitude by
// lane moves. Codes and scales pass through shared memory, so that a thread stores
// its block's 16 bytes at once. x is read past the caches (it is larger than they
// are where time counts), the codes, which a product reads next, are not written
// past them. 28672 x 8192 of fp32, 1.06 GB: 187 us, 5.7 TB/s; with ordinary loads
// 241, without the staging 195; codes written past the caches 172, and their next
// reader 18 slower. 256 and 512 threads 191 and 189. 20 x 8192 of bf16: 3 us.
template <typename T, bool ONE>
__global__ __launch_bounds__(kThreads) void k_mx4_quantize(const T* __restrict__ x, int64_t x_stride, int64_t rows,
                                                           int64_t cols, int64_t nb, char* __restrict__ codes,
                                                           int64_t code_stride, uint8_t* __restrict__ scales,
                                                           int64_t scale_stride) {
    using E = Elems<T>;
    constexpr int kSteps = E::kLanes, kPerStep = kThreads / E::kLanes;
    __shared__ __attribute__((aligned(16))) typename E::Code staged[kThreads * E::kLanes];
    __shared__ uint8_t staged_scales[kThreads];
    const Place<ONE> place(rows, nb);
    const int lane = threadIdx.x % E::kLanes, mine = threadIdx.x / E::kLanes;
    u32x4 v[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int i = u * kPerStep + mine;
        int64_t row, block;
        place.at(i, row, block);
        const int64_t e = block * 32 + lane * E::kN;
        v[u] = u32x4{0, 0, 0, 0};
        if (i < place.left && e < cols) {
            const T* p = x + row * x_stride + e;
            if (e + E::kN <= cols) {
                v[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_u2*>(p));
            } else {
#pragma unroll
                for (int k = 0; k < E::kN; ++k)
                    if (e + k < cols) v[u][k * (int)sizeof(T) / 4] |= (uint32_t)p[k] << (k * 8 * (int)sizeof(T) % 32);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const uint32_t exponent = group_max<E::kLanes>(E::amax(v[u])) >> 23;
        const bool bad = exponent == 255;
        const uint32_t s = bad ? 255u : exponent > 2 ? exponent - 2 : 0u;
        const typename E::Code c = E::encode(v[u], scale_f32(bad ? 127u : s));
        staged[u * kThreads + threadIdx.x] = bad ? 0 : c;
        if (lane == 0) staged_scales[u * kPerStep + mine] = (uint8_t)s;
    }
    __syncthreads();
    if (threadIdx.x >= place.left) return;
    int64_t row, block;
    place.at(threadIdx.x, row, block);
    *reinterpret_cast<u32x4_u2*>(codes + row * code_stride + block * 16) =
        reinterpret_cast<const u32x4*>(staged)[threadIdx.x];
    scales[row * scale_stride + block] = staged_scales[threadIdx.x];
}

// The same way back: a thread loads its block's 16 bytes of codes, and the block's
// lanes store 16 bytes of x each. 28672 x 8192 to fp32: 159 us, 6.7 TB/s (x is
// written past the caches; 183 with ordinary stores, 171 with 256 threads and 166
// with 64, 227 with 2-byte loads in the place of the staging).
template <typename T, bool ONE>
__global__ __launch_bounds__(kThreads) void k_mx4_dequantize(const char* __restrict__ codes, int64_t code_stride,
                                                             const uint8_t* __restrict__ scales, int64_t scale_stride,
                                                             int64_t rows, int64_t cols, int64_t nb,
                                                             T* __restrict__ x, int64_t x_stride) {
    using E = Elems<T>;
    constexpr int kSteps = E::kLanes, kPerStep = kThreads / E::kLanes;
    __shared__ __attribute__((aligned(16))) typename E::Code staged[kThreads * E::kLanes];
    __shared__ uint8_t staged_scales[kThreads];
    const Place<ONE> place(rows, nb);
    const int lane = threadIdx.x % E::kLanes, mine = threadIdx.x / E::kLanes;
    if (threadIdx.x < place.left) {
        int64_t row, block;
        place.at(threadIdx.x, row, block);
        reinterpret_cast<u32x4*>(staged)[threadIdx.x] =
            *(reinterpret_cast<const u32x4_u2*>(codes + row * code_stride + block * 16));
        staged_scales[threadIdx.x] = scales[row * scale_stride + block];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int i = u * kPerStep + mine;
        int64_t row, block;
        place.at(i, row, block);
        const int64_t e = block * 32 + lane * E::kN;
        if (i >= place.left || e >= cols) continue;
        const u32x4 v = E::decode(staged[u * kThreads + threadIdx.x], scale_f32(staged_scales[i]));
        T* p = x + row * x_stride + e;
        if (e + E::kN <= cols) {
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_u2*>(p));
        } else {
#pragma unroll
            for (int k = 0; k < E::kN; ++k)
                if (e + k < cols) p[k] = (T)(v[k * (int)sizeof(T) / 4] >> (k * 8 * (int)sizeof(T) % 32));
        }
    }
}

// Blocks of one launch: a launch covers at most 2^32 - 1 work-items.
constexpr int64_t kMostBlocks = int64_t(1) << 31;

// One row where rows follow each other without a gap in all three arrays.
bool one_row(int64_t rows, int64_t cols, int64_t x_stride, const Mx4& q) {
    return rows == 1 ||
           (cols % 32 == 0 && x_stride == cols && q.code_stride == cols / 2 && q.scale_stride == cols / 32);
}

// Calls launch(one, first row, rows, first column, columns) for parts of the
// matrix that fit a launch: rows, or, of one row, its columns.
template <typename F>
int by_parts(bool one, int64_t rows, int64_t cols, F launch) {
    if (one) {
        const int64_t all = rows * cols, most = kMostBlocks * 32;
        for (int64_t lo = 0; lo < all; lo += most)
            if (int e = launch(0, 1, lo, all - lo < most ? all - lo : most)) return e;
        return 0;
    }
    const int64_t nb = (cols + 31) / 32, most = kMostBlocks / nb;
    for (int64_t lo = 0; lo < rows; lo += most)
        if (int e = launch(lo, rows - lo < most ? rows - lo : most, 0, cols)) return e;
    return 0;
}

unsigned grid_of(int64_t rows, int64_t nb) { return (unsigned)((rows * nb + kThreads - 1) / kThreads); }

template <typename T, bool ONE>
int quantize(Rows x, int64_t rows, int64_t cols, const Mx4& out, hipStream_t s) {
    return by_parts(ONE, rows, cols, [&](int64_t r0, int64_t nr, int64_t c0, int64_t nc) {
        const int64_t nb = (nc + 31) / 32;
        k_mx4_quantize<T, ONE><<<grid_of(nr, nb), kThreads, 0, s>>>(
            static_cast<const T*>(x.p) + r0 * x.stride + c0, x.stride, nr, nc, nb,
            static_cast<char*>(const_cast<void*>(out.codes)) + r0 * out.code_stride + c0 / 2, out.code_stride,
            static_cast<uint8_t*>(const_cast<void*>(out.scales)) + r0 * out.scale_stride + c0 / 32, out.scale_stride);
        return (int)hipGetLastError();
    });
}

template <typename T, bool ONE>
int dequantize(const Mx4& in, int64_t rows, int64_t cols, Rows x, hipStream_t s) {
    return by_parts(ONE, rows, cols, [&](int64_t r0, int64_t nr, int64_t c0, int64_t nc) {
        const int64_t nb = (nc + 31) / 32;
        k_mx4_dequantize<T, ONE><<<grid_of(nr, nb), kThreads, 0, s>>>(
            static_cast<const char*>(in.codes) + r0 * in.code_stride + c0 / 2, in.code_stride,
            static_cast<const uint8_t*>(in.scales) + r0 * in.scale_stride + c0 / 32, in.scale_stride, nr, nc, nb,
            static_cast<T*>(const_cast<void*>(x.p)) + r0 * x.stride + c0, x.stride);
        return (int)hipGetLastError();
    });
}

}  // namespace

int launch_mx4_quantize(Rows x, int dtype, int64_t rows, int64_t cols, const Mx4& out, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool one = one_row(rows, cols, x.stride, out);
    if (dtype == ZS_DTYPE_BF16)
        return one ? quantize<uint16_t, true>(x, rows, cols, out, s) : quantize<uint16_t, false>(x, rows, cols, out, s);
    return one ? quantize<uint32_t, true>(x, rows, cols, out, s) : quantize<uint32_t, false>(x, rows, cols, out, s);
}

int launch_mx4_dequantize(const Mx4& in, int64_t rows, int64_t cols, Rows x, int dtype, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool one = one_row(rows, cols, x.stride, in);
    if (dtype == ZS_DTYPE_BF16)
        return one ? dequantize<uint16_t, true>(in, rows, cols, x, s)
                   : dequantize<uint16_t, false>(in, rows, cols, x, s);
    return one ? dequantize<uint32_t, true>(in, rows, cols, x, s) : dequantize<uint32_t, false>(in, rows, cols, x, s);
}

}  // namespace zs
