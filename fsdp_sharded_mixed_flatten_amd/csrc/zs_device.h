// Device code that the files of the step's kernels share (zs_kernels.hip,
// zs_clip.hip): bf16, the AdamW element, accesses to global memory, the sum of a
// wave. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include "zs_internal.h"

namespace zs {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ bf16

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// fp32 -> bf16 bits, IEEE round to nearest even; NaN -> quiet NaN, sign kept.
__device__ __forceinline__ uint32_t bf16_rne(float f) {
    uint32_t u = __float_as_uint(f);
    uint32_t r = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
    return ((u & 0x7FFFFFFFu) > 0x7F800000u) ? ((u >> 16) | 0x40u) : r;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) { return bf16_rne(a) | (bf16_rne(b) << 16); }

// ------------------------------------------------------------------ AdamW element

__device__ __forceinline__ void adamw_elem(const AdamCoef& c, float gf, float& w, float& m, float& v) {
    float wd = w * c.decay;
    float mn = c.b1 * m + c.omb1 * gf;
    float vn = c.b2 * v + c.omb2 * (gf * gf);
    float mh = mn / c.bc1;
    float vh = vn / c.bc2;
    float den = sqrtf(vh) + c.eps;
    w = wd - c.lr * (mh / den);
    m = mn;
    v = vn;
}

__device__ __forceinline__ void adamw_unit(const AdamCoef& c, u32x2 g, f32x4& w, f32x4& m, f32x4& v) {
    float w0 = w.x, w1 = w.y, w2 = w.z, w3 = w.w;
    float m0 = m.x, m1 = m.y, m2 = m.z, m3 = m.w;
    float v0 = v.x, v1 = v.y, v2 = v.z, v3 = v.w;
    adamw_elem(c, lo_bf16(g.x), w0, m0, v0);
    adamw_elem(c, hi_bf16(g.x), w1, m1, v1);
    adamw_elem(c, lo_bf16(g.y), w2, m2, v2);
    adamw_elem(c, hi_bf16(g.y), w3, m3, v3);
    w = f32x4{w0, w1, w2, w3};
    m = f32x4{m0, m1, m2, m3};
    v = f32x4{v0, v1, v2, v3};
}

__device__ __forceinline__ u32x2 to_bf16x4(const f32x4& w) {
    u32x2 p;
    p.x = pack2(w.x, w.y);
    p.y = pack2(w.z, w.w);
    return p;
}

// ------------------------------------------------------------------ global memory

// Every access goes through a global-address-space pointer. Pointers read
// from a device table (the multi-tensor pieces) are generic to the compiler,
// which would emit flat memory instructions for them; flat loads count
// against both wait counters and serialize the grouped loads. Every buffer
// here is global memory.
template <typename T>
using gptr = __attribute__((address_space(1))) T*;

template <typename T>
__device__ __forceinline__ T ld_nt(const T* p) { return __builtin_nontemporal_load((gptr<const T>)p); }
template <typename T>
__device__ __forceinline__ void st_nt(T* p, T x) { __builtin_nontemporal_store(x, (gptr<T>)p); }

// Plain (cached) global load, for table records.
template <typename T>
__device__ __forceinline__ T ld_g(const T* p) { return *(gptr<const T>)p; }

// Rows: lane L of the wave accesses unit L of a row of kBlockThreads consecutive
// units, which starts at p - L. Such an access can go through a buffer
// resource based at the row's first unit (the same address in every lane,
// taken into scalar registers) and bounded by the row's bytes, with the
// lane's byte offset as its vector offset; a buffer access carries the full
// cache-policy field, a global one written in HIP only nt.
constexpr int kBufferWord3 = 0x00020000;  // raw (untyped) buffer: 32-bit data format

template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const T* p) {
    static_assert(kBlockThreads == 64, "a row is one wave: blocks are single waves");
    const uintptr_t row = reinterpret_cast<uintptr_t>(p - threadIdx.x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)row);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(row >> 32));
    void* base = reinterpret_cast<void*>(((uintptr_t)hi << 32) | lo);
    return __builtin_amdgcn_make_buffer_rsrc(base, (short)0, kBlockThreads * (int)sizeof(T), kBufferWord3);
}

// Row stores: nontemporal with sc1 set. At the Llama-7B shape this is 2-3%
// faster for the fused step and up to 4% for AdamW than the global
// nontemporal store (nt alone, which a buffer store with nt alone times the
// same as); sc1 without nt is slower than both.
constexpr int kStreamAux = 2 | 16;  // nt | sc1

template <typename T>
__device__ __forceinline__ void st_lane(T* p, T x) {
    const __amdgpu_buffer_rsrc_t r = row_rsrc(p);
    const int off = (int)(threadIdx.x * sizeof(T));
    if constexpr (sizeof(T) == 16)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, off, 0, kStreamAux);
    else {
        static_assert(sizeof(T) == 8, "rows of 8- or 16-byte units");
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), r, off, 0, kStreamAux);
    }
}

// ------------------------------------------------------------------ a wave's sum

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
    return x;
}

}  // namespace zs
