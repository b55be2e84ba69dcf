// Products of a few rows with a weight matrix in the quantized gather's
// payload, for CDNA4 (gfx950):
//   y[r, o] = sum over i of code[o, i] * scale[o, i] * x[r, i].
//
// The payload is read once: bits/8 + 4/block bytes a weight against
// 2 * rows flops, so up to some tens of rows the product is an HBM stream and
// what has to be kept short is the arithmetic beside each load.
#include <hip/hip_runtime.h>

#include <type_traits>

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

// ------------------------------------------------------------------ whole blocks: matrix instructions
// Where tensor offset, n_in and S are multiples of a block of 32 or more
// elements, every 32 columns of a row lie in one block and are 16 bytes (4
// bits) or 32 bytes (8 bits) at an aligned address, and scale i of the payload
// belongs to elements [i * block, (i + 1) * block).
//
// A wave takes 16 * RT rows of W and, of every row, 128 columns at a time
// (a chunk): lane (g, r) = (lane / 16, lane % 16) loads the 32 codes of row r
// in columns 32 g ... 32 g + 31. Codes become bf16 (exact: they have at most
// 8 significant bits) and multiply x in v_mfma_f32_16x16x32_bf16 with x as the
// first operand (its 16 rows are rows of x) and W as the second (its 16
// columns are rows of W), so the scale, one a row of W, is one a lane of the
// result and is applied in fp32 to sums over whole blocks.
//
// One such instruction sums 32 columns, 8 from each group of 16 lanes. With
// blocks of 128 or more the order of the columns inside a chunk is free, and
// instruction j takes word j of every lane. With smaller blocks (NB = 4 or 2
// a chunk) it has to take the four groups' words from one block: the 4 x 4
// words are transposed between the groups of lanes, one exchange a word.
//
// The waves of a workgroup share its rows and take turns over the chunks;
// their sums meet in shared memory. No partial sum leaves the workgroup.
//
// 16 rows of x fill the instruction; with fewer, the unused rows repeat one and
// the rows are spread over the lane groups so that the result's first NI
// registers hold them all (row i * 4 + g of x is register i of group g).

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kChunk = 128;

template <int BITS>
struct Codes;  // the 32 codes of a lane's part of a chunk, and word j (8 codes) as bf16
template <>
struct Codes<4> {
    u32x4 w;
    __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void load(const char* p) {
        w = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    }
    __device__ __forceinline__ void transpose() {
        auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
        auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
        w = u32x4{c[0], c[1], d[0], d[1]};
    }
    // The conversion takes a byte's low 4 bits as a signed value / 16.
    static constexpr float kUnit = 16.0f;
    static __device__ __forceinline__ float low(uint32_t d, int byte) {
        return __builtin_amdgcn_cvt_off_f32_i4((int)((d >> (8 * byte)) & 0xFFu));
    }
    __device__ __forceinline__ bf16x8 word(int j) const {
        const uint32_t even = w[j];
        uint32_t odd = even >> 4;
        asm("" : "+v"(odd));  // one shift for the four high codes: their bytes are then picked by the conversions
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __builtin_amdgcn_perm(__float_as_uint(low(odd, i)), __float_as_uint(low(even, i)), 0x07060302u);
        return __builtin_bit_cast(bf16x8, v);
    }
};
template <>
struct Codes<8> {
    u32x4 w[2];
    __device__ __forceinline__ void zero() { w[0] = w[1] = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void load(const char* p) {
        w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
        w[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p) + 1);
    }
    __device__ __forceinline__ void transpose() {
        // word j is the pair (w[j / 2][2 (j % 2)], w[j / 2][2 (j % 2) + 1])
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            auto a = __builtin_amdgcn_permlane32_swap(w[0][h], w[1][h], false, false);
            auto b = __builtin_amdgcn_permlane32_swap(w[0][2 + h], w[1][2 + h], false, false);
            auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
            auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
            w[0][h] = c[0];
            w[0][2 + h] = c[1];
            w[1][h] = d[0];
            w[1][2 + h] = d[1];
        }
    }
    static constexpr float kUnit = 1.0f;
    __device__ __forceinline__ bf16x8 word(int j) const {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t d = w[j / 2][2 * (j % 2) + i / 2];
            const float a = (float)(int8_t)(d >> (16 * (i & 1))), b = (float)(int8_t)(d >> (16 * (i & 1) + 8));
            v[i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
        }
        return __builtin_bit_cast(bf16x8, v);
    }
};

// NB: blocks a chunk (1: blocks of 128 or 256). MT: 16-row tiles of x. NI: of a
// tile's 4 result registers, those that hold rows of x. RT: 16-row tiles of W
// a wave. SPAN: chunks a wave loads together.
template <int BITS, int NB, int MT, int NI, int RT, int SPAN>
__global__ __launch_bounds__(512) void k_matvec_block(QuantWeight w, const uint16_t* __restrict__ x, int64_t x_stride,
                                                      int rows, void* __restrict__ y, int y_bf16, int64_t y_stride) {
    extern __shared__ float sums[];  // [waves - 1][RT * MT * NI][64]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int g = lane >> 4, r = lane & 15;
    const int64_t o0 = (int64_t)blockIdx.x * (16 * RT);
    const int n_in = (int)w.n_in;

    const char* code[RT];
    const float* scale[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        int64_t o = o0 + 16 * t + r;
        if (o >= w.n_out) o = w.n_out - 1;  // rows behind the last one repeat it and are not stored
        const int64_t j = w.off + o * w.n_in;
        code[t] = static_cast<const char*>(w.codes) + (j + 32 * g) * BITS / 8;
        scale[t] = w.scales + (j >> w.block_shift);
    }
    // the row of x this lane feeds, and its columns inside a chunk
    const int token = (r & 3) * 4 + (r >> 2);
    const uint16_t* xp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        // lanes without a row of x repeat one: their row of the result is not stored
        const int row = 16 * m + token < rows ? 16 * m + token : 0;
        xp[m] = x + row * x_stride + (NB == 1 ? 32 : 8) * g;
    }

    f32x4 acc[RT][MT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // One span of columns from k0; TAIL: it reaches past the row's end, where
    // codes, scales and x count as zero.
    auto span = [&](int k0, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        Codes<BITS> c[SPAN][RT];
        float s[SPAN][RT][NB];
#pragma unroll
        for (int p = 0; p < SPAN; ++p) {
            const int k = k0 + p * kChunk;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                if (!TAIL || k + 32 * g < n_in)
                    c[p][t].load(code[t] + (int64_t)k * BITS / 8);
                else
                    c[p][t].zero();
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int kb = k + b * (kChunk / NB);
                    s[p][t][b] = !TAIL || kb < n_in ? scale[t][kb >> w.block_shift] : 0.0f;
                }
            }
        }
#pragma unroll
        for (int p = 0; p < SPAN; ++p) {
            const int k = k0 + p * kChunk;
            if (TAIL && k >= n_in) break;
            bf16x8 xv[MT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kj = k + (NB == 1 ? 8 : 32) * j;  // this lane's columns: kj + (32 or 8) g ...
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    u32x4 v = u32x4{0, 0, 0, 0};
                    if (!TAIL || kj + (NB == 1 ? 32 : 8) * g < n_in)
                        v = *reinterpret_cast<const u32x4_u2*>(xp[m] + kj);
                    xv[m][j] = __builtin_bit_cast(bf16x8, v);
                }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                if (NB > 1) c[p][t].transpose();
                f32x4 part[MT];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 cv = c[p][t].word(j);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                        part[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[m][j], cv,
                                                                          j % (4 / NB) == 0 ? zero : part[m], 0, 0, 0);
                    }
                    if ((j + 1) % (4 / NB) == 0) {
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int i = 0; i < NI; ++i)
                                acc[t][m][i] = __builtin_fmaf(part[m][i], s[p][t][j * NB / 4], acc[t][m][i]);
                    }
                }
            }
        }
    };
    int k0 = wave * (SPAN * kChunk);
    for (; k0 + SPAN * kChunk <= n_in; k0 += waves * (SPAN * kChunk)) span(k0, std::false_type{});
    if (k0 < n_in) span(k0, std::true_type{});

    // the waves' sums, in the order of the waves
    if (wave > 0) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    sums[((wave - 1) * (RT * MT * NI) + (t * MT + m) * NI + i) * 64 + lane] = acc[t][m][i];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float v = acc[t][m][i];
                for (int q = 1; q < waves; ++q)
                    v += sums[((q - 1) * (RT * MT * NI) + (t * MT + m) * NI + i) * 64 + lane];
                const int row = 16 * m + 4 * i + g;
                const int64_t o = o0 + 16 * t + r;
                if (row < rows && o < w.n_out) store_y(y, y_bf16, row * y_stride + o, v * Codes<BITS>::kUnit);
            }
}

template <int BITS, int NB, int MT, int NI, int RT>
void run_block_t(const QuantWeight& w, Rows x, int rows, void* y, bool y_bf16, int64_t y_stride, hipStream_t s) {
    constexpr int kSpan = RT * MT * BITS > 8 ? 2 : 4;
    const int64_t spans = (w.n_in + kSpan * kChunk - 1) / (kSpan * kChunk);
    const int waves = spans < 8 ? (int)spans : 8;
    const size_t lds = (size_t)(waves - 1) * (RT * MT * NI) * 64 * sizeof(float);
    hipLaunchKernelGGL((k_matvec_block<BITS, NB, MT, NI, RT, kSpan>),
                       dim3((unsigned)((w.n_out + 16 * RT - 1) / (16 * RT))), dim3(64 * waves), lds, s, w,
                       static_cast<const uint16_t*>(x.p), x.stride, rows, y, (int)y_bf16, y_stride);
}

template <int BITS, int NB>
void run_block_n(const QuantWeight& w, Rows x, int rows, void* y, bool y_bf16, int64_t y_stride, hipStream_t s) {
    if (rows <= 4)
        run_block_t<BITS, NB, 1, 1, 1>(w, x, rows, y, y_bf16, y_stride, s);
    else if (rows <= 8)
        run_block_t<BITS, NB, 1, 2, 1>(w, x, rows, y, y_bf16, y_stride, s);
    else if (rows <= 16)
        run_block_t<BITS, NB, 1, 4, 1>(w, x, rows, y, y_bf16, y_stride, s);
    else if (rows <= 32)
        run_block_t<BITS, NB, 2, 4, 1>(w, x, rows, y, y_bf16, y_stride, s);
    else
        run_block_t<BITS, NB, 4, 4, 1>(w, x, rows, y, y_bf16, y_stride, s);
}

template <int BITS>
void run_block(const QuantWeight& w, Rows x, int rows, void* y, bool y_bf16, int64_t y_stride, hipStream_t s) {
    if (w.block_shift == 5)
        run_block_n<BITS, 4>(w, x, rows, y, y_bf16, y_stride, s);
    else if (w.block_shift == 6)
        run_block_n<BITS, 2>(w, x, rows, y, y_bf16, y_stride, s);
    else
        run_block_n<BITS, 1>(w, x, rows, y, y_bf16, y_stride, s);
}

}  // namespace

int launch_quant_matvec(const QuantWeight& w, Rows x, int rows, void* y, int y_dtype, int64_t y_stride,
                        void* stream) {
    if (w.n_out > (int64_t)kAnyWaves * ((1 << 24) - 1)) return (int)hipErrorInvalidValue;  // 2^32 - 1 work-items
    const bool y_bf16 = y_dtype == ZS_DTYPE_BF16;
    const int64_t block = int64_t(1) << w.block_shift;
    const bool whole = block >= 32 && w.n_in > 0 && w.off % block == 0 && w.n_in % block == 0 && w.shard % block == 0;
    if (whole && w.bits == 4)
        run_block<4>(w, x, rows, y, y_bf16, y_stride, (hipStream_t)stream);
    else if (whole)
        run_block<8>(w, x, rows, y, y_bf16, y_stride, (hipStream_t)stream);
    else if (w.bits == 4)
        run_any<4>(w, x, rows, y, y_bf16, y_stride, (hipStream_t)stream);
    else
        run_any<8>(w, x, rows, y, y_bf16, y_stride, (hipStream_t)stream);
    return (int)hipGetLastError();
}

}  // namespace zs
