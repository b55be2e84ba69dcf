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
// Blocks of 8, blocks of 16 out of line with the rows, rows of less than 32
// columns and shards shorter than a row.
// One wave per row of W and M rows of x. The wave walks the row in units of 8
// elements of the flat buffer that start at multiples of 8: a unit never
// crosses a shard (S is a multiple of 8) or a block (blocks start at multiples
// of 8 of a shard), so it has one scale and its codes are one aligned 32- or
// 64-bit word. The units at the row's ends may reach into the neighbouring
// tensors; their elements there are left out.
// 8192 x 8192 int4 in blocks of 8 takes 18 us with one row of x, 28 with 4, 94
// with 16 and 350 with 64 (67 MB, 10.5 us at 6.4 TB/s); blocks of 16 with one row
// 18 and with 4 28 (50 MB, 7.9 us). An fp32 multiply-add a weight and row, every
// unit's loads waited for before the next, and W read again for every 4 rows.
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
// A wave takes 16 rows of W and, of every row, 128 columns at a time (a
// chunk): lane (g, r) = (lane / 16, lane % 16) loads the 32 codes of row r in
// columns 32 g ... 32 g + 31. Codes become bf16 (exact: they have at most 8
// significant bits) and multiply x in v_mfma_f32_16x16x32_bf16 with x as the
// first operand (its 16 rows are rows of x) and W as the second (its 16
// columns are rows of W), so the scale, one a row of W, is one a lane of the
// result and is applied in fp32 to sums over whole blocks. Against fp32
// multiply-adds this leaves 1.6 vector instructions a weight instead of more
// than 3 and about none a row of x.
//
// One such instruction sums 32 columns, 8 from each group of 16 lanes. With
// blocks of 128 or more the order of the columns inside a chunk is free, and
// instruction j takes word j of every lane. With smaller blocks (NB = 4 or 2
// a chunk) it has to take the four groups' words from one block: the 4 x 4
// words are transposed between the groups of lanes, one exchange a word.
//
// Row i * 4 + g of 16 rows of x is register i of lane group g in the result,
// so that up to 4 rows take one register. Lanes without a row of x repeat
// another's: their rows of the result are not stored.
//
// A wave loads spans of SPAN chunks at once (codes, the span's scales as
// 16-byte loads) and the next span's before it computes a span. Plain loads:
// a row's 64 bytes of a chunk are half a cache line, and with the nontemporal
// hint the line's other half came from memory again (28672 x 8192 int4, one
// row of x: 30.5 against 26.9 us).
//
// Times in this file are of calls on three sets of inputs in turn, unless they
// say one set: 125 MB of codes used again at once are partly held by the last
// cache (the 26.9 us are then 24.1).

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 __attribute__((aligned(4))) f32x4_u4;
typedef u32x4 __attribute__((aligned(4))) u32x4_u4;

constexpr int kChunk = 128;

template <int BITS>
struct Codes;  // the 32 codes of a lane's part of a chunk, and word j (8 codes) as bf16
template <>
struct Codes<4> {
    u32x4 w;
    __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void load(const char* p) {
        w = *reinterpret_cast<const u32x4*>(p);
    }
    __device__ __forceinline__ void transpose() {
        auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
        auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
        w = u32x4{c[0], c[1], d[0], d[1]};
    }
    // The conversion takes a byte's low 4 bits as a signed value / 16.
    __device__ __forceinline__ void set(const uint32_t* d) { w = u32x4{d[0], d[1], d[2], d[3]}; }
    // Leaves out codes of word j (8 bits: of its halves).
    __device__ __forceinline__ void keep(int j, uint32_t m, uint32_t) { w[j] &= m; }
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
        w[0] = *reinterpret_cast<const u32x4*>(p);
        w[1] = reinterpret_cast<const u32x4*>(p)[1];
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
    __device__ __forceinline__ void set(const uint32_t* d) {
        w[0] = u32x4{d[0], d[1], d[2], d[3]};
        w[1] = u32x4{d[4], d[5], d[6], d[7]};
    }
    __device__ __forceinline__ void keep(int j, uint32_t m0, uint32_t m1) {
        w[j / 2][2 * (j % 2)] &= m0;
        w[j / 2][2 * (j % 2) + 1] &= m1;
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

// What a wave loads of W for one span of columns, whole blocks.
template <int BITS, int SHIFT, int SPAN_>
struct Span {
    static constexpr int SPAN = SPAN_, kBits = BITS;
    static constexpr int NB = SHIFT >= 7 ? 1 : kChunk >> SHIFT;  // blocks a chunk (1: a block is a chunk or two)
    static constexpr int kScales = SPAN * kChunk >= 1 << SHIFT ? SPAN * kChunk >> SHIFT : 1;
    static constexpr int kBeyond = 0;       // columns behind a span that its loads may touch
    static constexpr bool kRagged = false;  // rows may end inside 8 columns
    Codes<BITS> c[SPAN];
    float s[kScales];

    // The codes and scales of the row of W that this lane loads, from its column
    // 32 g on. Rows behind the last one repeat it and are not stored.
    struct Row {
        const char* code;
        const float* scale;
        __device__ __forceinline__ Row(const QuantWeight& w, int64_t o, int g) {
            const int64_t j = w.off + (o < w.n_out ? o : w.n_out - 1) * w.n_in;
            code = static_cast<const char*>(w.codes) + (j + 32 * g) * BITS / 8;
            scale = w.scales + (j >> SHIFT);
        }
    };

    // The span of columns from k0. TAIL: it may reach past the row's end, where
    // codes and scales count as zero.
    template <bool TAIL>
    __device__ __forceinline__ void load(const Row& row, int k0, int n_in, int g) {
#pragma unroll
        for (int p = 0; p < SPAN; ++p) {
            const int k = k0 + p * kChunk;
            if (!TAIL || k + 32 * g < n_in)
                c[p].load(row.code + (int64_t)k * BITS / 8);
            else
                c[p].zero();
        }
        const float* sp = row.scale + (k0 >> SHIFT);
        if (TAIL) {
#pragma unroll
            for (int i = 0; i < kScales; ++i) s[i] = k0 + (i << SHIFT) < n_in ? sp[i] : 0.0f;
            return;
        }
#pragma unroll
        for (int i = 0; i < kScales; i += 4) {
            if (kScales - i >= 4) {
                const f32x4 v = *reinterpret_cast<const f32x4_u4*>(sp + i);
                s[i] = v[0], s[i + 1] = v[1], s[i + 2] = v[2], s[i + 3] = v[3];
            } else {
#pragma unroll
                for (int n = i; n < kScales; ++n) s[n] = sp[n];
            }
        }
    }

    // acc += scales * (chunk p of W times x): xv[m][j] is the lane's operand for
    // instruction j of tile m of x.
    template <int MT, int NI>
    __device__ __forceinline__ void multiply(int p, const u32x4 (&xv)[MT][4], f32x4 (&acc)[MT]) {
        if (NB > 1) c[p].transpose();
        f32x4 part[MT];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x8 cv = c[p].word(j);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                part[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[m][j]), cv,
                                                                  j % (4 / NB) == 0 ? zero : part[m], 0, 0, 0);
            }
            if ((j + 1) % (4 / NB) == 0) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        acc[m][i] = __builtin_fmaf(part[m][i], s[(p * kChunk + j * 32) >> SHIFT], acc[m][i]);
            }
        }
    }
    // Columns of a chunk between a lane's operands for instructions j and j + 1,
    // and between lane groups, in units of 8.
    static constexpr int kUnitJ = NB == 1 ? 1 : 4, kUnitG = NB == 1 ? 4 : 1;
};

// ------------------------------------------------------------------ split blocks
// What a wave loads of W for one span where blocks of 32 or more elements start
// anywhere in a row: tensor offset, n_in or S are no multiples of block. A
// window of 32 columns then holds parts of at most two blocks, A before and B
// behind a boundary, and is multiplied twice, with the codes of B and then those
// of A left out: two partial sums, each with its own scale. Where a shard's
// last block is shorter than 32, the window around it holds a third, C. Scales
// follow one another from boundary to boundary, also from one shard to the next.
// Whole blocks of 16 go this way too: A and B are then halves of a window.
//
// A row's first code may lie at any 4 or 8 bits: a lane loads the words around
// its 32 codes and shifts them into place. Lane (g, r) works out boundary and
// scales of row r in window g of a chunk; the other lane groups ask it for them.
// More than twice the arithmetic and loads of whole blocks, which bound it: 8191
// x 8191 int4, blocks of 128, takes 24 us with one row of x, 28 with 4 and 16 and
// 67 with 64 (8192 x 8192 in whole blocks 10, 13, 15 and 29; k_matvec_any 21, 49,
// 165 and 633: with one row alone it is ahead).
template <int BITS, int SPAN_>
struct SplitSpan {
    static constexpr int SPAN = SPAN_, kBits = BITS;
    static constexpr int kWords = BITS;        // 32-bit words of 32 codes
    static constexpr int kPer = 32 / BITS;     // codes a word
    static constexpr int kBeyond = kPer;       // the word behind the lane's codes
    static constexpr bool kRagged = true;
    Codes<BITS> c[SPAN];
    float sa[SPAN], sb[SPAN], sc[SPAN];
    int edge[SPAN], edge2[SPAN];  // columns of the lane's window before the boundaries (32 and more: all)

    struct Row {
        const uint32_t* word;  // the one that holds the lane's first code
        const uint32_t* end;   // of the payload's codes
        int shift;             // of that code in its word, in bits
        const float* scale;    // of the row's first element
        int first;             // of the row's first element in its block
        int left;              // elements of the row's first shard from there on (or more than the row has)
        int log2_block;
        __device__ __forceinline__ Row(const QuantWeight& w, int64_t o, int g) {
            const int64_t j = w.off + (o < w.n_out ? o : w.n_out - 1) * w.n_in;
            const int64_t jg = j + 32 * g, q = j / w.shard, s = j - q * w.shard;
            const uint32_t* words = static_cast<const uint32_t*>(w.codes);
            word = words + jg / kPer;
            end = words + w.shard * w.world / kPer;
            shift = (int)(jg % kPer) * BITS;
            log2_block = w.block_shift;
            scale = w.scales + q * w.n_scales + (s >> log2_block);
            first = (int)(s & ((1 << log2_block) - 1));
            const int64_t rest = w.shard - s;
            left = rest < w.n_in ? (int)rest : INT32_MAX / 2;
        }
    };

    template <bool TAIL>
    __device__ __forceinline__ void load(const Row& row, int k0, int n_in, int g) {
#pragma unroll
        for (int p = 0; p < SPAN; ++p) {
            const int k = k0 + p * kChunk, kg = k + 32 * g;
            const uint32_t* at = row.word + k / kPer;
            uint32_t d[kWords + 1];
            if (!TAIL) {
#pragma unroll
                for (int i = 0; i < kWords; i += 4) {
                    const u32x4 v = *reinterpret_cast<const u32x4_u4*>(at + i);
                    d[i] = v[0], d[i + 1] = v[1], d[i + 2] = v[2], d[i + 3] = v[3];
                }
                d[kWords] = at[kWords];
            } else {
                const int used = n_in - kg;  // codes from the lane's first column on
#pragma unroll
                for (int i = 0; i <= kWords; ++i) d[i] = (i - 1) * kPer < used && at + i < row.end ? at[i] : 0u;
            }
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                d[i] = __builtin_amdgcn_alignbit(d[i + 1], d[i], row.shift);
                if (TAIL) d[i] &= mask(n_in - kg - i * kPer);
            }
            c[p].set(d);
            // boundary and scales of window g
            int index, next;
            if (kg < row.left) {
                index = (row.first + kg) >> row.log2_block;
                next = ((index + 1) << row.log2_block) - row.first;
                next = next < row.left ? next : row.left;
            } else {
                const int b = (kg - row.left) >> row.log2_block;
                index = ((row.first + row.left - 1) >> row.log2_block) + 1 + b;
                next = ((b + 1) << row.log2_block) + row.left;
            }
            edge[p] = next - kg;
            sa[p] = !TAIL || kg < n_in ? row.scale[index] : 0.0f;
            sb[p] = next < n_in && edge[p] < 32 ? row.scale[index + 1] : 0.0f;
            int last = next + (1 << row.log2_block);
            if (next < row.left && last > row.left) last = row.left;
            edge2[p] = last - kg;
            sc[p] = last < n_in && edge2[p] < 32 ? row.scale[index + 2] : 0.0f;
        }
    }

    // The first n codes of a word.
    static __device__ __forceinline__ uint32_t mask(int n) {
        return n >= kPer ? ~0u : n <= 0 ? 0u : (1u << (n * BITS)) - 1u;
    }

    template <int MT, int NI>
    __device__ __forceinline__ void multiply(int p, const u32x4 (&xv)[MT][4], f32x4 (&acc)[MT]) {
        const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
        c[p].transpose();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int from = 16 * j + r;
            const int n = __shfl(edge[p], from, 64) - 8 * g;  // this lane's codes of window j before the boundary
            auto part = [&](const Codes<BITS>& codes, float scale) {
                const bf16x8 cv = codes.word(j);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                    const f32x4 v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[m][j]), cv,
                                                                            zero, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < NI; ++i) acc[m][i] = __builtin_fmaf(v[i], scale, acc[m][i]);
                }
            };
            const float a = __shfl(sa[p], from, 64);
            if (__all(n >= 8)) {  // no row has a boundary in this window
                part(c[p], a);
                continue;
            }
            Codes<BITS> before = c[p], behind = c[p];
            before.keep(j, mask(n), mask(n - kPer));
            behind.keep(j, ~mask(n), ~mask(n - kPer));
            part(before, a);
            const int n2 = __shfl(edge2[p], from, 64) - 8 * g;
            if (__any(n2 < 8)) {
                Codes<BITS> third = behind;
                behind.keep(j, mask(n2), mask(n2 - kPer));
                third.keep(j, ~mask(n2), ~mask(n2 - kPer));
                part(third, __shfl(sc[p], from, 64));
            }
            part(behind, __shfl(sb[p], from, 64));
        }
    }
    static constexpr int kUnitJ = 4, kUnitG = 1;
};

// 8 columns of a row of x from k on, zero from the row's end; RAGGED: the row
// may end inside them.
template <bool RAGGED>
__device__ __forceinline__ u32x4 load_x(const uint16_t* x, int k, int n_in) {
    u32x4 v = u32x4{0, 0, 0, 0};
    if (k + 8 <= n_in || (!RAGGED && k < n_in)) {
        v = *reinterpret_cast<const u32x4_u2*>(x + k);
    } else if (RAGGED) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < n_in) v[i >> 1] |= (uint32_t)x[k + i] << (16 * (i & 1));
    }
    return v;
}

// Up to 4 rows of x, ROWS of them through shared memory: a wave loads its
// span's columns of each row once, contiguously, and its lanes read their
// operands from there (loading operands straight from x issues 4 wide loads a
// chunk that mostly repeat each other, and took 36 instead of 24.5 us at 28672
// x 8192 int4, one set of inputs). The waves of a workgroup share its 16 rows of
// W and take turns over the spans; their sums meet in shared memory at the end.
// Reads at 4.6 TB/s at 28672 x 8192 int4 (26.9 us, one row), 5.2 TB/s at 8192 x
// 128256 int8 (210 us, 4 rows, blocks of 128, fp32 results); bound by memory
// there and by latency in products of a few MB (4096 x 4096 int4 4.0 us in a
// captured graph, an empty launch 1.6 us).
template <typename S, int ROWS>
__global__ __launch_bounds__(512) void k_matvec_few(QuantWeight w, const uint16_t* __restrict__ x, int64_t x_stride,
                                                    int rows, void* __restrict__ y, int y_bf16, int64_t y_stride) {
    constexpr int SPAN = S::SPAN;
    constexpr int kUnits = SPAN * kChunk / 8;  // 16-byte units of a row of x in a span: a lane each
    constexpr int kPitch = kUnits + 4;
    static_assert(kUnits <= 64, "a wave loads a row of x at once");
    extern __shared__ u32x4 shared[];  // [waves][ROWS][kPitch], then the sums of waves 1 ... [waves - 1][64]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int g = lane >> 4, r = lane & 15;
    const int64_t o = (int64_t)blockIdx.x * 16 + r;
    const int n_in = (int)w.n_in;
    const typename S::Row row(w, o, g);
    u32x4* const xs = shared + wave * (ROWS * kPitch);
    const int token = (r & 3) * 4 + (r >> 2);
    const u32x4* const xr = xs + (token < rows ? token : 0) * kPitch + S::kUnitG * g;

    f32x4 acc[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
    struct Loaded {
        S s;
        u32x4 x[ROWS];
    };
    auto load = [&](Loaded& b, int k0, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        b.s.template load<TAIL>(row, k0, n_in, g);
        const int k = k0 + 8 * lane;
#pragma unroll
        for (int m = 0; m < ROWS; ++m) {
            b.x[m] = u32x4{0, 0, 0, 0};
            if (m < rows && lane < kUnits) {
                if (TAIL)
                    b.x[m] = load_x<S::kRagged>(x + m * x_stride, k, n_in);
                else
                    b.x[m] = *reinterpret_cast<const u32x4_u2*>(x + m * x_stride + k);
            }
        }
    };
    auto compute = [&](Loaded& b, int k0, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        // written and read by this wave's lanes only: in order, no barrier
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int m = 0; m < ROWS; ++m)
            if (lane < kUnits) xs[m * kPitch + lane] = b.x[m];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        u32x4 xv[SPAN][1][4];
#pragma unroll
        for (int p = 0; p < SPAN; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) xv[p][0][j] = xr[p * (kChunk / 8) + S::kUnitJ * j];
#pragma unroll
        for (int p = 0; p < SPAN; ++p) {
            if (TAIL && k0 + p * kChunk >= n_in) break;
            b.s.template multiply<1, 1>(p, xv[p], acc);
        }
    };
    // spans that lie in the row with all their loads touch, then the others
    constexpr int kSpan = SPAN * kChunk, kWhole = kSpan + S::kBeyond;
    const int step = waves * kSpan;
    int k0 = wave * kSpan;
    if (k0 + kWhole <= n_in) {
        Loaded a, b;
        load(a, k0, std::false_type{});
        while (true) {
            const bool more = k0 + step + kWhole <= n_in;
            if (more) load(b, k0 + step, std::false_type{});
            compute(a, k0, std::false_type{});
            k0 += step;
            if (!more) break;
            const bool again = k0 + step + kWhole <= n_in;
            if (again) load(a, k0 + step, std::false_type{});
            compute(b, k0, std::false_type{});
            k0 += step;
            if (!again) break;
        }
    }
    for (; k0 < n_in; k0 += step) {
        Loaded a;
        load(a, k0, std::true_type{});
        compute(a, k0, std::true_type{});
    }
    // the waves' sums, in the order of the waves
    float* const sums = reinterpret_cast<float*>(shared + waves * (ROWS * kPitch));
    if (wave > 0) sums[(wave - 1) * 64 + lane] = acc[0][0];
    __syncthreads();
    if (wave > 0) return;
    float v = acc[0][0];
    for (int q = 1; q < waves; ++q) v += sums[(q - 1) * 64 + lane];
    if (g < rows && o < w.n_out) store_y(y, y_bf16, g * y_stride + o, v * Codes<S::kBits>::kUnit);
}

// 5 and more rows of x, MT tiles of 16 a workgroup (further tiles take further
// workgroups, which find the codes in a cache): what costs here is bringing x
// to the waves (each needs all of it), so RW waves with 16 rows of W each share
// a span of x in shared memory, and KW such groups take turns over the spans.
// One barrier a turn; x of the next turn is loaded beside its codes and goes
// into the other half of the buffer.
// 28672 x 8192 int4 with 16 rows: 43 us against 76 with each wave loading its
// own operands, 64 rows 97 against 258; at 2048 x 11008 with 16 rows 9.2
// against 10.8 (one set of inputs, an earlier form; 45, 102 and 8.8 us with
// three sets now). Far from memory's speed, 2.8 TB/s with 16 rows and 1.2 with
// 64: vector instructions take 17 and 50 us of these, shared memory 6 and 24, and
// the waves wait half of their time.
template <typename S, int MT, int RW, int KW>
__global__ __launch_bounds__(64 * RW * KW) void k_matvec_rows(QuantWeight w, const uint16_t* __restrict__ x,
                                                              int64_t x_stride, int rows, void* __restrict__ y,
                                                              int y_bf16, int64_t y_stride) {
    const int row0 = blockIdx.y * (16 * MT);  // this workgroup's first row of x
    x += row0 * x_stride;
    rows = rows - row0 < 16 * MT ? rows - row0 : 16 * MT;
    constexpr int SPAN = S::SPAN;
    constexpr int kSpan = SPAN * kChunk;
    constexpr int kUnits = kSpan / 8;           // 16-byte units of a row of x in a span
    constexpr int kPitch = kUnits + 1;          // rows start in different banks
    constexpr int kTile = 16 * MT * kPitch;     // one group's x
    constexpr int kLoads = 16 * MT * kUnits / (64 * RW);
    static_assert(kLoads * 64 * RW == 16 * MT * kUnits, "a group loads whole spans of x");
    constexpr int kX = 2 * KW * kTile * 16, kS = (KW - 1) * RW * MT * 4 * 64 * 4;
    __shared__ __attribute__((aligned(16))) char shared[kX > kS ? kX : kS];
    u32x4* const xl = reinterpret_cast<u32x4*>(shared);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rw = wave % RW, kw = wave / RW;
    const int g = lane >> 4, r = lane & 15;
    const int64_t o = ((int64_t)blockIdx.x * RW + rw) * 16 + r;
    const int n_in = (int)w.n_in;
    const int turns = (n_in + KW * kSpan - 1) / (KW * kSpan);
    const typename S::Row wrow(w, o, g);
    const int token = (r & 3) * 4 + (r >> 2);
    int xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xrow[m] = (16 * m + token < rows ? 16 * m + token : 0) * kPitch + S::kUnitG * g;

    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 xn[kLoads];
    auto load = [&](S& b, int turn) {
        const int k0 = (turn * KW + kw) * kSpan;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int u = rw * 64 + lane + i * (64 * RW), row = u / kUnits, k = k0 + u % kUnits * 8;
            xn[i] = row < rows ? load_x<S::kRagged>(x + row * x_stride, k, n_in) : u32x4{0, 0, 0, 0};
        }
        if (k0 + kSpan + S::kBeyond <= n_in)
            b.template load<false>(wrow, k0, n_in, g);
        else
            b.template load<true>(wrow, k0, n_in, g);
    };
    auto store = [&](int turn) {
        u32x4* to = xl + ((turn & 1) * KW + kw) * kTile;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int u = rw * 64 + lane + i * (64 * RW);
            to[u / kUnits * kPitch + u % kUnits] = xn[i];
        }
    };
    auto compute = [&](S& b, int turn) {
        const u32x4* from = xl + ((turn & 1) * KW + kw) * kTile;
#pragma unroll
        for (int p = 0; p < SPAN; ++p) {
            u32x4 xv[MT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int m = 0; m < MT; ++m) xv[m][j] = from[xrow[m] + p * (kChunk / 8) + S::kUnitJ * j];
            b.template multiply<MT, 4>(p, xv, acc);
        }
    };
    S a, b;
    load(a, 0);
    store(0);
    __syncthreads();
    for (int turn = 0; turn < turns; turn += 2) {
        if (turn + 1 < turns) load(b, turn + 1);
        compute(a, turn);
        if (turn + 1 >= turns) break;
        store(turn + 1);
        __syncthreads();
        if (turn + 2 < turns) load(a, turn + 2);
        compute(b, turn + 1);
        if (turn + 2 < turns) store(turn + 2);
        __syncthreads();
    }
    if (KW > 1) {  // the groups' sums, in the order of the groups
        float* const sums = reinterpret_cast<float*>(shared);
        __syncthreads();
        if (kw > 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[(((kw - 1) * RW + rw) * (MT * 4) + m * 4 + i) * 64 + lane] = acc[m][i];
        }
        __syncthreads();
        if (kw > 0) return;
#pragma unroll
        for (int q = 1; q < KW; ++q)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][i] += sums[(((q - 1) * RW + rw) * (MT * 4) + m * 4 + i) * 64 + lane];
    }
    if (o >= w.n_out) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * m + 4 * i + g;
            if (row < rows) store_y(y, y_bf16, (row0 + row) * y_stride + o, acc[m][i] * Codes<S::kBits>::kUnit);
        }
}

struct Product {
    const QuantWeight& w;
    Rows x;
    int rows;
    void* y;
    int y_bf16;
    int64_t y_stride;
    hipStream_t s;
};

template <typename S, int ROWS>
void run_few(const Product& a) {
    constexpr int kSpan = S::SPAN * kChunk;
    const int64_t tiles = (a.w.n_out + 15) / 16, spans = (a.w.n_in + kSpan - 1) / kSpan;
    // 8 waves a workgroup while a workgroup a CU is about all there is (4096 x
    // 4096 int4 4.0 us against 4.4 with 4), else 4 (28672 x 8192 int4 26.9 us
    // against 28.3 with 8, 8192 x 128256 107 against 152)
    const int most = tiles <= 256 ? 8 : 4;
    const int waves = spans < most ? (int)spans : most;
    const size_t lds = (size_t)waves * ROWS * (kSpan / 8 + 4) * 16 + (size_t)(waves - 1) * 64 * 4;
    hipLaunchKernelGGL((k_matvec_few<S, ROWS>), dim3((unsigned)tiles), dim3(64 * waves), lds, a.s, a.w,
                       static_cast<const uint16_t*>(a.x.p), a.x.stride, a.rows, a.y, a.y_bf16, a.y_stride);
}

template <typename S, int MT, int RW, int KW>
void run_rows(const Product& a) {
    const dim3 grid((unsigned)((a.w.n_out + 16 * RW - 1) / (16 * RW)), (unsigned)((a.rows + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((k_matvec_rows<S, MT, RW, KW>), grid, dim3(64 * RW * KW), 0, a.s, a.w,
                       static_cast<const uint16_t*>(a.x.p), a.x.stride, a.rows, a.y, a.y_bf16, a.y_stride);
}

// S<SPAN>: what loads W, in spans of SPAN chunks. The choices were measured
// against each other (1 to 4 tiles of x, 1 to 8 waves that share it, 1 to 16
// groups that split the columns, spans of 1 to 4) at the sizes in the comments
// (columns x rows of W), int4, in us, one set of inputs.
template <template <int> class S>
void run_block(const Product& a) {
    constexpr bool kSplit = S<1>::kRagged;
    const int64_t n_out = a.w.n_out;
    // From here on 128 rows of W a workgroup fill the chip and all 8 waves share
    // x (8192 x 128256, 16 rows: 131 against 192 with 4 groups of 4).
    const bool wide = n_out >= 128 * 256;
    // Up to here 32 rows a workgroup leave compute units idle: fewer rows of W
    // and of x each, the tiles of x in workgroups of their own.
    const bool narrow = n_out <= 4096;
    if (a.rows == 1)
        run_few<S<4>, 1>(a);
    else if (a.rows <= 4)
        run_few<S<4>, 4>(a);
    else if (a.rows <= 16) {
        if (wide)
            run_rows<S<4>, 1, 8, 1>(a);
        else if constexpr (kSplit) {
            if (n_out <= 8192)  // 8191 x 8191: 31 against 39
                run_rows<S<1>, 1, 1, 8>(a);
            else
                run_rows<S<2>, 1, 2, 4>(a);
        } else if (narrow)  // 4096 x 4096: 7.5 against 8.4, 8192 x 512: 10.4 against 12.2
            run_rows<S<2>, 1, 1, 8>(a);
        else if (n_out <= 8192 && a.w.n_in > 2048)  // 28672 x 8192: 43 against 57
            run_rows<S<4>, 1, 2, 4>(a);
        else  // 4096 x 16384: 12.2 against 15.9, 2048 x 11008: 9.2 against 11.6
            run_rows<S<2>, 1, 2, 4>(a);
    } else if (a.rows <= 32) {
        if (wide)
            run_rows<S<2>, 2, 8, 1>(a);
        else if constexpr (kSplit) {
            if (narrow)  // 7253 x 271: 24 against 46
                run_rows<S<1>, 1, 1, 8>(a);
            else
                run_rows<S<2>, 2, 2, 4>(a);
        } else if (narrow)  // 4096 x 4096: 10.4 against 12.2
            run_rows<S<2>, 1, 2, 4>(a);
        else  // 8192 x 8192: 22.7 against 25.9
            run_rows<S<2>, 2, 2, 4>(a);
    } else if (wide) {
        run_rows<S<1>, 4, 8, 1>(a);
    } else if constexpr (kSplit) {
        if (narrow)  // 1995 x 3769, 60 rows: 15.5 against 21.8
            run_rows<S<1>, 2, 2, 4>(a);
        else  // 8191 x 8191, 40 rows: 62 against 88
            run_rows<S<1>, 4, 2, 4>(a);
    } else if (narrow) {  // 4096 x 4096, 64 rows: 12.3 against 19.0
        run_rows<S<2>, 2, 2, 4>(a);
    } else if (S<1>::kBits == 4) {  // 28672 x 8192, 64 rows: 97 against 121
        run_rows<S<1>, 2, 2, 4>(a);
    } else {  // 8 bits, read twice by two tiles of x: 2304 x 13200, 53 rows 24 against 31
        run_rows<S<1>, 4, 2, 4>(a);
    }
}

template <int SPAN>
using Whole4x32 = Span<4, 5, SPAN>;
template <int SPAN>
using Whole4x64 = Span<4, 6, SPAN>;
template <int SPAN>
using Whole4x128 = Span<4, 7, SPAN>;
template <int SPAN>
using Whole4x256 = Span<4, 8, SPAN>;
template <int SPAN>
using Whole8x32 = Span<8, 5, SPAN>;
template <int SPAN>
using Whole8x64 = Span<8, 6, SPAN>;
template <int SPAN>
using Whole8x128 = Span<8, 7, SPAN>;
template <int SPAN>
using Whole8x256 = Span<8, 8, SPAN>;
// Two chunks a span at most: their boundaries and scales take registers too
// (2049 x 60001 int4, one row: 46 us against 72 with 4; 16 rows 59 against 88).
template <int SPAN>
using Split4 = SplitSpan<4, (SPAN < 2 ? SPAN : 2)>;
template <int SPAN>
using Split8 = SplitSpan<8, (SPAN < 2 ? SPAN : 2)>;

}  // namespace

int launch_quant_matvec(const QuantWeight& w, Rows x, int rows, void* y, int y_dtype, int64_t y_stride,
                        void* stream) {
    const Product a{w, x, rows, y, y_dtype == ZS_DTYPE_BF16, y_stride, (hipStream_t)stream};
    const int64_t block = int64_t(1) << w.block_shift;
    const bool four = w.bits == 4;
    const bool whole = w.off % block == 0 && w.n_in % block == 0 && w.shard % block == 0;
    // split blocks: at most one shard's end in a row, and no more than two
    // boundaries inside 32 columns (whole blocks of 16 have one: 8192 x 8192 int4
    // with 16 rows 28 us against 97 a wave a row, with 5 28 against 43, with 4 30
    // against 28, with one 29 against 18)
    const bool split = w.shard >= w.n_in && (block >= 32 || (block == 16 && whole && rows > 4));
    if (block >= 32 && w.n_in > 0 && whole) {
        switch (w.block_shift) {
            case 5: four ? run_block<Whole4x32>(a) : run_block<Whole8x32>(a); break;
            case 6: four ? run_block<Whole4x64>(a) : run_block<Whole8x64>(a); break;
            case 7: four ? run_block<Whole4x128>(a) : run_block<Whole8x128>(a); break;
            default: four ? run_block<Whole4x256>(a) : run_block<Whole8x256>(a); break;
        }
    } else if (w.n_in >= 32 && split) {
        four ? run_block<Split4>(a) : run_block<Split8>(a);
    } else if (four) {
        run_any<4>(w, x, rows, y, a.y_bf16, y_stride, a.s);
    } else {
        run_any<8>(w, x, rows, y, a.y_bf16, y_stride, a.s);
    }
    return (int)hipGetLastError();
}

}  // namespace zs
