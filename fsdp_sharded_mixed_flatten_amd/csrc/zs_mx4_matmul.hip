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
typedef uint32_t __attribute__((aligned(1))) u32_u1;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // the matrix instructions' name of the format

// Two results as bf16 in one word: the hardware's conversion, which rounds to
// nearest even (compared with the rounding by integers over all 2^32 fp32 values:
// no bit differs), the only rounding of a result; NaN stays NaN.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ void store_y(void* y, bool bf16, int64_t i, float v) {
    if (bf16)
        static_cast<uint16_t*>(y)[i] = (uint16_t)pack_bf16(v, v);
    else
        static_cast<float*>(y)[i] = v;
}

// Four results side by side, `left` of which there are, k elements behind `at`.
typedef uint32_t u32x2_u2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_u4 __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void store4(char* at, bool bf16, int k, const float (&v)[4], int left) {
    if (left >= 4) {
        if (bf16)
            *reinterpret_cast<u32x2_u2*>(at + 2 * k) = u32x2_u2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        else
            *reinterpret_cast<f32x4_u4*>(at + 4 * k) = f32x4_u4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) store_y(at, bf16, k + i, v[i]);
    }
}

// 16 x 16 products of 128 columns. Lane l gives block l / 16 of row l % 16 of
// either side and has rows 4 * (l / 16) .. + 3 of x and column l % 16 of y.
__device__ __forceinline__ f32x4 mfma16(const u32x4& x, uint32_t sx, const u32x4& w, uint32_t sw, f32x4 acc) {
    const i32x8 a{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    const i32x8 b{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, kFp4, kFp4, 0, (int)sx, 0, (int)sw);
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// 32 x 32 products of 64 columns, with byte STEP of each side's scales. Lane l gives
// one block of row l % 32 of either side and has column l % 32 (x) and rows 8 (e / 4)
// + 4 (l / 32) + e % 4 (W) of the result.
template <int STEP>
__device__ __forceinline__ f32x16 mfma32(const u32x4& w, uint32_t sw, const u32x4& x, uint32_t sx, f32x16 acc) {
    const i32x8 a{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const i32x8 b{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, kFp4, kFp4, STEP, (int)sw, STEP, (int)sx);
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

// 1 x 4096 x 4096: 3.9 us, a few dependent steps (its bytes take 1.4).
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

// Up to 64 rows of x, 32 rows of W: the waves of a workgroup take turns of 512
// columns, whose operands they hold in registers (eight instructions of 64
// columns, of which a lane of the upper half gives the second block), and add up
// through shared memory.
constexpr int kRowsX = 64;
__global__ __launch_bounds__(64 * kFewWaves) void k_mx4_rows(Mx4 x, int rows, Mx4 w, int out, int blocks,
                                                             void* __restrict__ y, int y_bf16, int64_t y_stride) {
    constexpr int TX = kRowsX / 32;
    __shared__ float part[kFewWaves][16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int r0 = blockIdx.y * 32 * TX, o0 = blockIdx.x * 32;
    const int64_t o = min(o0 + (lane & 31), out - 1);
    const char* wc = static_cast<const char*>(w.codes) + o * w.code_stride;
    const uint8_t* ws = static_cast<const uint8_t*>(w.scales) + o * w.scale_stride;
    const char* xc[TX];
    const uint8_t* xs[TX];
#pragma unroll
    for (int j = 0; j < TX; ++j) {
        const int64_t r = min(r0 + 32 * j + (lane & 31), rows - 1);
        xc[j] = static_cast<const char*>(x.codes) + r * x.code_stride;
        xs[j] = static_cast<const uint8_t*>(x.scales) + r * x.scale_stride;
    }
    f32x16 acc[TX];
#pragma unroll
    for (int j = 0; j < TX; ++j) acc[j] = f32x16{};
    const int whole = blocks / 16;
    for (int t = wave; t < whole; t += kFewWaves) {
        u32x4 a[8], b[TX][8], sa, sb[TX];
#pragma unroll
        for (int s = 0; s < 8; ++s)
            a[s] = *reinterpret_cast<const u32x4*>(wc + (int64_t)(t * 16 + 2 * s + half) * 16);
        sa = *reinterpret_cast<const u32x4_u1*>(ws + t * 16);
#pragma unroll
        for (int j = 0; j < TX; ++j) {
#pragma unroll
            for (int s = 0; s < 8; ++s)
                b[j][s] = *reinterpret_cast<const u32x4*>(xc[j] + (int64_t)(t * 16 + 2 * s + half) * 16);
            sb[j] = *reinterpret_cast<const u32x4_u1*>(xs[j] + t * 16);
        }
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int j = 0; j < TX; ++j)
                acc[j] = s & 1 ? mfma32<2>(a[s], sa[s / 2] >> (8 * half), b[j][s], sb[j][s / 2] >> (8 * half), acc[j])
                               : mfma32<0>(a[s], sa[s / 2] >> (8 * half), b[j][s], sb[j][s / 2] >> (8 * half), acc[j]);
    }
    // the rest, two blocks at a time: what lies behind the last is 0 with scale 1
    if (wave == whole % kFewWaves) {
        for (int s = whole * 16; s < blocks; s += 2) {
            const bool in = s + half < blocks;
            const int at = in ? s + half : s;
            u32x4 a = *reinterpret_cast<const u32x4*>(wc + (int64_t)at * 16);
            if (!in) a = u32x4{0, 0, 0, 0};
            const uint32_t sa = in ? ws[at] : 127u;
#pragma unroll
            for (int j = 0; j < TX; ++j) {
                const u32x4 b = *reinterpret_cast<const u32x4*>(xc[j] + (int64_t)at * 16);
                acc[j] = mfma32<0>(a, sa, b, in ? xs[j][at] : 127u, acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < TX; ++j) {
        if (j > 0) __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; ++e) part[wave][e][lane] = acc[j][e];
        __syncthreads();
        // thread i has values 2 (i / 64) and the next of lane i % 64
#pragma unroll
        for (int q = 0; q < 16 / kFewWaves; ++q) {
            const int e = (16 / kFewWaves) * wave + q;
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kFewWaves; ++k) sum += part[k][e][lane];
            const int row = r0 + 32 * j + (lane & 31), col = o0 + 8 * (e / 4) + 4 * half + e % 4;
            if (row < rows && col < out) store_y(y, y_bf16, row * y_stride + col, sum);
        }
    }
}

// ------------------------------------------------------------------ many rows
// A workgroup computes BW columns of y (rows of W) for BX rows of x, its WW x WX
// waves 32 TW x 32 TX each. Both sides' codes go straight from global to shared
// memory, 128 columns (a turn) at a time through a ring of four stages: while
// a turn is multiplied the next three are on their way or there. A row's 64
// bytes are four 16-byte blocks; block c of row r lies at place c ^ (r / 4 % 4),
// so that the sixteen lanes that are served together reach all banks. (The narrow
// tile's turn is 256 columns, eight blocks: place c ^ (r / 2 % 8).)
// 4096 x 8192 x 28672: 541 to 565 us, 3.4 to 3.6 PFLOP/s, where a loop of the
// instructions alone reaches 6.5 on such codes (8.7 on zeros). The matrix unit is
// busy 46% of the cycles (1.64 GHz while counted; that loop 91% at 1.71 GHz), 54%
// with twice the columns, and no access to shared memory conflicts. A form with four
// waves came from 49 to 57% with its global loads left out: most of the waiting is
// for the workgroup itself, one a compute unit, whose waves meet at a barrier every
// 128 columns and then all read operands. 20 x 8192 x 128256: 104 to 112 us, 5.2 to
// 5.6 TB/s; runs of two lines of a row with 32 rows of x a tile take 127.
// A lane of a 32 x 32 instruction gives one block of row l % 32. Which 64
// columns an instruction takes is free as long as both sides agree: the lower
// lanes take blocks 0 and 1 of a turn's four, the upper ones 2 and 3, so that a
// lane's two scales are neighbouring bytes, which the instruction's operand
// selection picks. W gives the rows of an instruction's result, so that a lane
// holds four columns of y side by side.
template <int TW_, int TX_, int WW_, int WX_, int BLOCKS_, int STAGES_, int PER_SIMD_>
struct Tile {
    static constexpr int TW = TW_, TX = TX_, WW = WW_, WX = WX_, kStages = STAGES_, kPerSimd = PER_SIMD_;
    // 32-column blocks of a turn, 64-column steps of it, turns of a group of 512 columns
    static constexpr int kBlocks = BLOCKS_, kSteps = BLOCKS_ / 2, kTurns = 16 / BLOCKS_;
    static constexpr int kThreads = 64 * WW * WX, BW = 32 * TW * WW, BX = 32 * TX * WX, kRows = BW + BX;
    // 16-byte loads of a thread a turn, the same number in all waves: loads behind
    // the last row are of nothing
    static constexpr int kLoads = (kRows * kBlocks + kThreads - 1) / kThreads;
    static constexpr int kScaleLoads = (kRows + kThreads - 1) / kThreads;
    static_assert(BW * kBlocks % kThreads == 0, "a load is of one side");
    static_assert(kBlocks == 4 || kBlocks == 8, "the layout of shared memory");
};

typedef __attribute__((address_space(3))) void* lds_ptr;

template <typename T>
struct Shared {
    u32x4 codes[T::kStages][T::kLoads * T::kThreads];
    uint32_t scales[4][T::kRows];  // of 512 columns: a word a turn and row
};

// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ char* uniform(const void* p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
    return reinterpret_cast<char*>(((uintptr_t)hi << 32) | lo);
}

// One 64-column step's operands of a wave.
template <typename T>
struct Step {
    u32x4 w[T::TW], x[T::TX];
};
template <typename T>
struct Scales {
    uint32_t w[T::TW], x[T::TX];
};

// What a load leaves out (rows past the end, blocks past the last) is asked
// for behind the buffer's end, where a load gives 0. Buffers are of at most 2^30
// bytes (256 rows of 2^22), offsets inside them are smaller, and a sum of two such
// places is below 2^32.
constexpr uint32_t kNowhere = 0x7FFFFFF0u;

// Rows of W that many bytes apart, or a multiple of it, have the same columns in
// the same part of the memory, which workgroups that all begin with a row's first
// columns would ask at once: each begins elsewhere in its rows. us with and without:
//   bytes apart         4096        8192       12288      16384      32768
//   1 x 8192 rows    9.5  10.5   16.3 17.2   18.9 22.1   23.7 33.9   42.9 58.4
//   20 x 8192         10  10.8   18.8 18.3   23.9 25.3   28.1 36.3   51.9 61.7
//   1 x 28672       24.4  27.4   47.5 51.4   64.5 68.1   79.9  102    154  171
//   20 x 28672      31.6  32.2   55.4 57.4   83.8 95.7    101  112    203  209
//   1 x 128256        88  99.2    171  192    255  266    319  401
//   20 x 128256      108   115    180  213    279  300    332  382
// Where rows are 2048 or 6144 bytes apart it costs: 1 x 28672 16.1 and 15.4, 35 and
// 34; and where W is read by several tiles (4096 rows of x) 583 and 563.
constexpr int kCrowded = 4096;

template <typename T>
struct Tiled {
    Shared<T>& sh;
    __amdgpu_buffer_rsrc_t wr, xr;
    int blocks, groups, first;  // groups of 512 columns, and the one that the tile begins with
    bool once;                  // no other tile reads this one's rows of W
    int wave, lblock;           // the block of a turn that this thread's loads take
    uint32_t from[T::kLoads];   // and where in W and x they find it in turn 0
    int read_w, read_x;      // the rows of the tile's sides whose blocks this lane reads first
    int swizzle, half;
    const uint8_t* scale_row[T::kScaleLoads];
    u32x4 held[T::kScaleLoads];

    // W where no other tile reads its rows: whole lines that leave the cache to x and
    // the scales, whose lines are read a piece at a time (20 rows x 8192 x 128256:
    // 114 us against 125). With half lines a turn the other half would be lost.
    static constexpr int kNontemporal = 2;
    static constexpr bool kElsewhere = T::kBlocks == 8;  // of the tiles, the narrow one may be alone over its rows of W
    static constexpr int kLoadRows = T::kThreads / T::kBlocks;
    __device__ __forceinline__ void fetch(int turn, int stage) {
        int real = turn;
        if constexpr (kElsewhere) {
            const int turns = groups * T::kTurns, at = turn + first * T::kTurns;
            real = turn >= turns ? turns : at - (at >= turns ? turns : 0);
        }
        const uint32_t add = real * T::kBlocks + lblock < blocks ? real * (T::kBlocks * 16u) : kNowhere;
#pragma unroll
        for (int u = 0; u < T::kLoads; ++u) {
            const lds_ptr to = (lds_ptr)&sh.codes[stage][u * T::kThreads + wave * 64];
            if (u >= T::BW / kLoadRows)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, to, 16, (int)(from[u] + add), 0, 0, 0);
            else if (T::kBlocks == 8 && once)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, to, 16, (int)(from[u] + add), 0, 0, kNontemporal);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, to, 16, (int)(from[u] + add), 0, 0, 0);
        }
    }
    // Scales of 512 columns (16 bytes a row) go through registers.
    __device__ __forceinline__ void fetch_scales(int turn_group) {
        int group = turn_group;
        if constexpr (kElsewhere) group = group + first - (group + first >= groups ? groups : 0);
        if ((group + 1) * 16 <= blocks) {
#pragma unroll
            for (int k = 0; k < T::kScaleLoads; ++k)
                held[k] = *reinterpret_cast<const u32x4_u1*>(scale_row[k] + group * 16);
        } else {  // the last: what lies behind the row's end is 1
#pragma unroll
            for (int k = 0; k < T::kScaleLoads; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t b[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) b[e] = scale_row[k][min(group * 16 + 4 * i + e, blocks - 1)];
#pragma unroll
                    for (int e = 0; e < 4; ++e) b[e] = group * 16 + 4 * i + e < blocks ? b[e] : 127;
                    held[k][i] = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
                }
        }
    }
    // The words of turns FIRST to LAST.
    template <int FIRST, int LAST>
    __device__ __forceinline__ void put_scales() {
#pragma unroll
        for (int k = 0; k < T::kScaleLoads; ++k) {
            const int row = k * T::kThreads + threadIdx.x;
            if (T::kRows % T::kThreads == 0 || row < T::kRows)
#pragma unroll
                for (int i = FIRST; i <= LAST; ++i) sh.scales[i][row] = held[k][i];
        }
    }
    __device__ __forceinline__ void read(int stage, int step, Step<T>& f) const {
        const int place = (T::kSteps * half + step) ^ swizzle;
        constexpr int kUp = 32 * T::kBlocks;
#pragma unroll
        for (int i = 0; i < T::TW; ++i) f.w[i] = sh.codes[stage][read_w * T::kBlocks + kUp * i + place];
#pragma unroll
        for (int i = 0; i < T::TX; ++i) f.x[i] = sh.codes[stage][(T::BW + read_x) * T::kBlocks + kUp * i + place];
    }
    // A lane's scales of a turn, the first step's in the lowest byte.
    __device__ __forceinline__ void read_scales(int turn, Scales<T>& s) const {
        const uint32_t* words = sh.scales[T::kBlocks == 4 ? turn : 2 * turn + half];
        const int shift = T::kBlocks == 4 ? 16 * half : 0;
#pragma unroll
        for (int i = 0; i < T::TW; ++i) s.w[i] = words[read_w + 32 * i] >> shift;
#pragma unroll
        for (int i = 0; i < T::TX; ++i) s.x[i] = words[T::BW + read_x + 32 * i] >> shift;
    }
    template <int STEP>
    __device__ __forceinline__ void multiply(const Step<T>& f, const Scales<T>& s, f32x16 (&acc)[T::TW][T::TX]) const {
#pragma unroll
        for (int i = 0; i < T::TW; ++i)
#pragma unroll
            for (int j = 0; j < T::TX; ++j) acc[i][j] = mfma32<STEP>(f.w[i], s.w[i], f.x[j], s.x[j], acc[i][j]);
    }
    // All steps of a turn but the last, whose operands are read.
    template <int STEP>
    __device__ __forceinline__ void steps(int stage, Step<T> (&f)[2], const Scales<T>& s,
                                          f32x16 (&acc)[T::TW][T::TX]) const {
        read(stage, STEP + 1, f[(STEP + 1) & 1]);
        multiply<STEP>(f[STEP & 1], s, acc);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (STEP + 2 < T::kSteps) steps<STEP + 1>(stage, f, s, acc);
    }
};

// All but the N youngest of this wave's loads are there, and all waves are here.
// (A barrier of the language would wait for all loads.)
template <int N>
__device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename T>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void k_mx4_tiled(Mx4 x, int rows, Mx4 w, int out, int blocks,
                                                           void* __restrict__ y, int y_bf16, int64_t y_stride,
                                                           int tiles_x) {
    __shared__ Shared<T> sh;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tile = blockIdx.x;
    const int r0 = tile % tiles_x * T::BX, o0 = tile / tiles_x * T::BW;
    const int mine_x = min(rows - r0, T::BX), mine_w = min(out - o0, T::BW);
    const int xs = (int)x.code_stride, ws = (int)w.code_stride;
    const int wave_w = wave % T::WW, wave_x = wave / T::WW;
    const int groups = (blocks + 15) / 16;  // turns behind the last block multiply zeros
    Tiled<T> t{sh,
               __builtin_amdgcn_make_buffer_rsrc(uniform(static_cast<const char*>(w.codes) + o0 * w.code_stride),
                                                 (short)0, (mine_w - 1) * ws + blocks * 16, 0x00020000),
               __builtin_amdgcn_make_buffer_rsrc(uniform(static_cast<const char*>(x.codes) + r0 * x.code_stride),
                                                 (short)0, (mine_x - 1) * xs + blocks * 16, 0x00020000),
               blocks, groups, tiles_x == 1 && ws % kCrowded == 0 ? tile % groups : 0, tiles_x == 1, wave,
               (tid & (T::kBlocks - 1)) ^ (tid >> 4 & (T::kBlocks - 1)), {},
               32 * T::TW * wave_w + (lane & 31), 32 * T::TX * wave_x + (lane & 31),
               T::kBlocks == 4 ? lane >> 2 & 3 : lane >> 1 & 7,
               lane >> 5, {}, {}};
#pragma unroll
    for (int u = 0; u < T::kLoads; ++u) {
        const int row = u * Tiled<T>::kLoadRows + tid / T::kBlocks, in_x = row - T::BW;
        t.from[u] = row < T::BW ? (row < mine_w ? (uint32_t)(row * ws + t.lblock * 16) : kNowhere)
                                : (in_x < mine_x ? (uint32_t)(in_x * xs + t.lblock * 16) : kNowhere);
    }
#pragma unroll
    for (int k = 0; k < T::kScaleLoads; ++k) {
        const int row = k * T::kThreads + tid;
        t.scale_row[k] =
            row < T::BW ? static_cast<const uint8_t*>(w.scales) + (o0 + min(row, mine_w - 1)) * w.scale_stride
                        : static_cast<const uint8_t*>(x.scales) + (r0 + min(row - T::BW, mine_x - 1)) * x.scale_stride;
    }
    f32x16 acc[T::TW][T::TX];
#pragma unroll
    for (int i = 0; i < T::TW; ++i)
#pragma unroll
        for (int j = 0; j < T::TX; ++j) acc[i][j] = f32x16{};

    t.fetch_scales(0);
#pragma unroll
    for (int i = 0; i < T::kStages; ++i) t.fetch(i, i);
    t.template put_scales<0, 3>();
    if (T::kTurns == 2) t.fetch_scales(groups > 1 ? 1 : 0);
    // all but the youngest kStages - 1 turns' loads (and the scales')
    arrive<(T::kStages - 1) * T::kLoads>();
    Step<T> f[2];
    Scales<T> s[2];
    t.read(0, 0, f[0]);
    t.read_scales(0, s[0]);
    int at = 0;  // the present turn's stage
    for (int g = 0; g < groups; ++g) {
        // A turn's loads are asked for in order, so that waiting for all but the
        // youngest kStages - 2 turns' leaves the next turn's there. Of four turns,
        // the first asks for the next group's scales, between the loads of turns
        // kStages - 1 and kStages; of two, the second for those of the one after
        // next. They are put down when the words they replace have been read.
#pragma unroll
        for (int turn = 0; turn < T::kTurns; ++turn) {
            constexpr bool kFixed = T::kTurns % T::kStages == 0;
            const int stage = kFixed ? turn % T::kStages : at;
            const int then = kFixed ? (turn + 1) % T::kStages : (at + 1 == T::kStages ? 0 : at + 1);
            t.template steps<0>(stage, f, s[turn & 1], acc);
            // the next turn's codes are there, and this one's have been read
            if (T::kTurns == 4 && turn >= 1 && turn <= T::kStages - 2)
                arrive<(T::kStages - 2) * T::kLoads + T::kScaleLoads>();
            else
                arrive<(T::kStages - 2) * T::kLoads>();
            if constexpr (T::kTurns == 4) {
                if (turn == 0) t.fetch_scales(g + 1 < groups ? g + 1 : g);
                if (turn == 2) t.template put_scales<0, 2>();
                if (turn == 3) t.template put_scales<3, 3>();
            } else {
                if (turn == 0) t.template put_scales<0, 1>();
                if (turn == 1) t.template put_scales<2, 3>();
                if (turn == 1) t.fetch_scales(g + 2 < groups ? g + 2 : g);
            }
            t.fetch(T::kTurns * g + turn + T::kStages, stage);
            t.read(then, 0, f[0]);
            t.read_scales((turn + 1) % T::kTurns, s[(turn + 1) & 1]);
            t.template multiply<T::kSteps - 1>(f[1], s[turn & 1], acc);
            __builtin_amdgcn_sched_barrier(0);
            at = then;
        }
    }
    arrive<0>();  // the loads behind the last turn write shared memory, too
    // Lane l has row l % 32 of y and columns 8 * (e / 4) + 4 * (l / 32) + e % 4.
    const int row0 = r0 + 32 * T::TX * wave_x + (lane & 31);
    const int col0 = o0 + 32 * T::TW * wave_w + 4 * (lane >> 5);
#pragma unroll
    for (int j = 0; j < T::TX; ++j) {
        if (row0 + 32 * j >= rows) continue;
        char* at = static_cast<char*>(y) + ((row0 + 32 * j) * y_stride + col0) * (y_bf16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < T::TW; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 32 * i + 8 * e;
                const float v[4] = {acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
                store4(at, y_bf16, k, v, out - col0 - k);
            }
    }
}

template <typename T>
int launch_tiled(const Mx4& x, int64_t rows, const Mx4& w, int64_t out, int64_t blocks, void* y, int y_bf16,
                 int64_t y_stride, hipStream_t s) {
    const int64_t tx = (rows + T::BX - 1) / T::BX, tw = (out + T::BW - 1) / T::BW;
    k_mx4_tiled<T><<<(unsigned)(tx * tw), T::kThreads, 0, s>>>(x, (int)rows, w, (int)out, (int)blocks, y, y_bf16,
                                                              y_stride, (int)tx);
    return (int)hipGetLastError();
}

int launch_few(const Mx4& x, int64_t rows, const Mx4& w, int64_t out, int64_t blocks, void* y, int y_bf16,
               int64_t y_stride, hipStream_t s) {
    // a launch covers at most 2^32 - 1 work-items and 65535 tiles of rows
    const int64_t tiles = (out + 15) / 16;
    const int64_t fit = ((int64_t(1) << 32) - 1) / (tiles * 64 * kFewWaves);
    const int64_t most = 16 * (fit < 1 ? 1 : fit > 65535 ? 65535 : fit);
    for (int64_t lo = 0; lo < rows; lo += most) {
        const int64_t n = rows - lo < most ? rows - lo : most;
        const Mx4 part{static_cast<const char*>(x.codes) + lo * x.code_stride,
                       static_cast<const char*>(x.scales) + lo * x.scale_stride, x.code_stride, x.scale_stride};
        k_mx4_few<<<dim3((unsigned)tiles, (unsigned)((n + 15) / 16)), 64 * kFewWaves, 0, s>>>(
            part, n, w, out, (int)blocks, static_cast<char*>(y) + lo * y_stride * (y_bf16 ? 2 : 4), y_bf16, y_stride);
        if (hipError_t e = hipGetLastError()) return (int)e;
    }
    return 0;
}

// ------------------------------------------------------------------ few rows, many of W
// Up to 32 rows of x, 32 TW rows of W. The workgroup's WAVES waves share a row's
// columns, 256 each in turn, so that together they read runs of WAVES * 128 bytes
// of a row. A wave's
// columns are its own: codes go through its own ring of STAGES turns in shared
// memory with waits by count and no barrier, scales through registers. At the
// end the waves' sums are added up through shared memory.
template <int TW_, int WAVES_, int STAGES_>
struct Long {
    static constexpr int TW = TW_, kWaves = WAVES_, kStages = STAGES_;
    static constexpr int kThreads = 64 * WAVES_, BW = 32 * TW_, kRows = BW + 32;
    static constexpr int kWLoads = BW / 8, kLoads = kRows / 8;  // of a wave a turn, 16 bytes a lane
    static constexpr int kTurnLoads = kLoads + TW_ + 1;         // with the scales'
    static constexpr int kQuarter = 16 * TW_ / WAVES_;          // values of a lane that a wave adds up
    static_assert(kQuarter % 4 == 0, "whole stores");
    static_assert((kStages - 1) * kTurnLoads < 64, "what a wait can count");
};

template <typename T>
struct LongWave {
    u32x4 (&ring)[T::kStages][T::kLoads * 64];
    __amdgpu_buffer_rsrc_t wr, xr;
    const uint8_t* scale_row[T::TW + 1];
    uint32_t from[T::kLoads];
    int blocks, slices, first, lblock, half;  // first: the slice of 256 columns that this workgroup begins with

    // The slice of the row that the workgroup's slice number `slice` is; behind the
    // last, what is behind the row's end.
    __device__ __forceinline__ int place_of(int slice) const {
        return slice >= slices ? slices : slice + first - (slice + first >= slices ? slices : 0);
    }
    // Loads of W leave the caches to x and the scales, whose lines are read a piece
    // at a time.
    __device__ __forceinline__ void fetch(int slice, int stage, uint32_t (&scales)[T::TW + 1]) {
        const int real = place_of(slice), at_block = min(real * 8 + 4 * half, blocks - 4);
#pragma unroll
        for (int i = 0; i <= T::TW; ++i) scales[i] = *reinterpret_cast<const u32_u1*>(scale_row[i] + at_block);
#pragma unroll
        for (int u = 0; u < T::kLoads; ++u) {
            const lds_ptr to = (lds_ptr)&ring[stage][u * 64];
            const int block = real * 8 + (lblock ^ (4 * (u & 1)));
            const uint32_t at = from[u] + (block < blocks ? real * 128u : kNowhere);
            if (u < T::kWLoads)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, to, 16, (int)at, 0, 0, 2);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, to, 16, (int)at, 0, 0, 0);
        }
    }
    // Scales that reach behind the row's end were read from its last four on; what
    // lies behind is 1.
    __device__ __forceinline__ void mend(int slice, uint32_t (&scales)[T::TW + 1]) const {
        const int over = min(max(place_of(slice) * 8 + 4 * half - (blocks - 4), 0), 4);
#pragma unroll
        for (int i = 0; i <= T::TW; ++i)
            scales[i] = (uint32_t)((uint64_t(0x7F7F7F7F) << 32 | scales[i]) >> (8 * over));
    }
    template <int STEP>
    __device__ __forceinline__ void step(int stage, int lane, const uint32_t (&scales)[T::TW + 1],
                                         f32x16 (&acc)[T::TW]) const {
        const int place = (lane & 31) * 8 + ((4 * half + STEP) ^ (lane >> 1 & 7));
        const u32x4 x = ring[stage][T::BW * 8 + place];
#pragma unroll
        for (int i = 0; i < T::TW; ++i)
            acc[i] = mfma32<STEP>(ring[stage][256 * i + place], scales[i], x, scales[T::TW], acc[i]);
    }
};

template <typename T>
__global__ __launch_bounds__(T::kThreads) void k_mx4_long(Mx4 x, int rows, Mx4 w, int out, int blocks,
                                                          void* __restrict__ y, int y_bf16, int64_t y_stride) {
    __shared__ u32x4 ring[T::kWaves][T::kStages][T::kLoads * 64];
    static_assert(sizeof(ring) >= sizeof(float) * T::kWaves * T::TW * 16 * 64, "the sums fit");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int o0 = blockIdx.x * T::BW, mine_w = min(out - o0, T::BW);
    const int xs = (int)x.code_stride, ws = (int)w.code_stride;
    const int slices = (blocks + 7) / 8;
    LongWave<T> t{ring[wave],
                  __builtin_amdgcn_make_buffer_rsrc(uniform(static_cast<const char*>(w.codes) + o0 * w.code_stride),
                                                    (short)0, (mine_w - 1) * ws + blocks * 16, 0x00020000),
                  __builtin_amdgcn_make_buffer_rsrc(uniform(x.codes), (short)0, (rows - 1) * xs + blocks * 16,
                                                    0x00020000),
                  {}, {}, blocks, slices, ws % kCrowded == 0 ? (int)(blockIdx.x % (unsigned)slices) : 0,
                  (lane & 7) ^ (lane >> 4), lane >> 5};
#pragma unroll
    for (int u = 0; u < T::kLoads; ++u) {
        const int row = u * 8 + lane / 8, in_x = row - T::BW, at = (t.lblock ^ (4 * (u & 1))) * 16;
        t.from[u] = row < T::BW ? (row < mine_w ? (uint32_t)(row * ws + at) : kNowhere)
                                : (in_x < rows ? (uint32_t)(in_x * xs + at) : kNowhere);
    }
#pragma unroll
    for (int i = 0; i < T::TW; ++i)
        t.scale_row[i] =
            static_cast<const uint8_t*>(w.scales) + (o0 + min(32 * i + (lane & 31), mine_w - 1)) * w.scale_stride;
    t.scale_row[T::TW] = static_cast<const uint8_t*>(x.scales) + min(lane & 31, rows - 1) * x.scale_stride;
    f32x16 acc[T::TW];
#pragma unroll
    for (int i = 0; i < T::TW; ++i) acc[i] = f32x16{};
    uint32_t scales[T::kStages][T::TW + 1];
#pragma unroll
    for (int i = 0; i < T::kStages; ++i) {
        t.fetch(wave + i * T::kWaves, i, scales[i]);
        asm volatile("" ::: "memory");
    }
    // a turn's codes and scales are asked for together, the oldest first
    // (turns behind the last multiply zeros)
    for (int slice = wave; slice < slices;) {
#pragma unroll
        for (int stage = 0; stage < T::kStages; ++stage) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((T::kStages - 1) * T::kTurnLoads) : "memory");
            t.mend(slice, scales[stage]);
            t.template step<0>(stage, lane, scales[stage], acc);
            t.template step<1>(stage, lane, scales[stage], acc);
            t.template step<2>(stage, lane, scales[stage], acc);
            t.template step<3>(stage, lane, scales[stage], acc);
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the turn has been read
            t.fetch(slice + T::kStages * T::kWaves, stage, scales[stage]);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            slice += T::kWaves;
        }
    }
    arrive<0>();  // the loads behind the last turn write shared memory, too
    float* sums = reinterpret_cast<float*>(&ring[0][0][0]);
#pragma unroll
    for (int i = 0; i < T::TW; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) sums[((wave * T::TW + i) * 16 + e) * 64 + lane] = acc[i][e];
    __syncthreads();
    const int row = lane & 31;
    if (row >= rows) return;
    char* at = static_cast<char*>(y) + (row * y_stride + o0) * (y_bf16 ? 2 : 4);
#pragma unroll
    for (int q = 0; q < T::kQuarter; q += 4) {
        const int first = wave * T::kQuarter + q, i = first / 16, e0 = first % 16;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = 0.0f;
#pragma unroll
            for (int k = 0; k < T::kWaves; ++k) v[e] += sums[((k * T::TW + i) * 16 + e0 + e) * 64 + lane];
        }
        const int col = 32 * i + 2 * e0 + 4 * t.half;
        store4(at, y_bf16, col, v, out - o0 - col);
    }
}

template <typename T>
int launch_long(const Mx4& x, int64_t rows, const Mx4& w, int64_t out, int64_t blocks, void* y, int y_bf16,
                int64_t y_stride, hipStream_t s) {
    k_mx4_long<T><<<(unsigned)((out + T::BW - 1) / T::BW), T::kThreads, 0, s>>>(x, (int)rows, w, (int)out,
                                                                              (int)blocks, y, y_bf16, y_stride);
    return (int)hipGetLastError();
}

int launch_rows(const Mx4& x, int64_t rows, const Mx4& w, int64_t out, int64_t blocks, void* y, int y_bf16,
                int64_t y_stride, hipStream_t s) {
    k_mx4_rows<<<dim3((unsigned)((out + 31) / 32), (unsigned)((rows + kRowsX - 1) / kRowsX)), 64 * kFewWaves, 0, s>>>(
        x, (int)rows, w, (int)out, (int)blocks, y, y_bf16, y_stride);
    return (int)hipGetLastError();
}

// 32 columns of y for 32 rows of x: two turns of 256 columns in each of four waves,
// two workgroups a compute unit. us, 28672 x 8192 with 20 rows: 26; three turns and
// 64 columns of y 43 (half as many workgroups), four turns 27 and two waves 30. The
// narrower tile's share of x costs where there are many: 20 rows, 8192 x 128256 123
// against 118 with 128 columns of y in two waves, which takes 77 at 28672 x 8192.
using LongRows = Long<1, 4, 2>;
// 128 columns of y for 64 rows of x: three stages of 256 columns.
using Narrow = Tile<2, 1, 2, 2, 8, 3, 2>;
// 128 for 128: four stages of 128 columns, two workgroups a compute unit.
using Middle = Tile<2, 2, 2, 2, 4, 4, 2>;
// 256 for 256: eight waves, each of which reads six operands for eight instructions
// (four for four in the tile above, three for two in the narrow one).
using Wide = Tile<2, 4, 4, 2, 4, 4, 2>;

enum Shape { kFew, kRows, kLong, kNarrow, kMiddle, kWide };

// The shape for rows of x, out rows of W and blocks of either, by how many
// workgroups each gives the 256 compute units. us, columns x rows of W:
//   rows of x                   few  rows     long  narrow  middle  wide
//   1, 4096 x 4096              4.1           5.1                        up to 16 rows few below 256 tiles of 32
//   16, 4096 x 4096             4.7      6.7  5.5      10      11    23
//   16, 4096 x 6400             6.9           5.8
//   1, 4096 x 11008             6.9           8.3
//   16, 8192 x 6400              13           9.2
//   16, 16384 x 6400             24            16                        (where the rule errs most)
//   16, 8192 x 8192              13            10
//   1, 28672 x 8192              26            21
//   1, 8192 x 128256            111      168   89     102     115   131
//   8, 8192 x 128256                          103     106                narrow from 800 tiles of 128 on above
//   16, 8192 x 128256                         117     105                8 rows, and where rows are short
//   1, 8192 x 76800                            56      82
//   8, 8192 x 102400                           82      95                (800 tiles)
//   16, 8192 x 102400                          93      97
//   16, 8192 x 51200                           49      47
//   1, 16384 x 128256                         171     167
//   16, 16384 x 128256                        218     178
//   16, 16384 x 51200                          96      83
//   1, 4096 x 76800                            33      39
//   1, 4096 x 102400                           42      44
//   1, 4096 x 128256                           51      48
//   16, 4096 x 128256                          63      54
//   1, 4096 x 151936                           59      63
//   16, 4096 x 151936                          73      70
//   1, 2048 x 28672                            11      10                (of fewer than 128 blocks: from 200 on)
//   1, 2048 x 76800                            22      22
//   1, 2048 x 151936                           38      35
//   16, 2048 x 40000                           14      13
//   16, 8192 x 28672             41       50   28      30      32    51
//   20, 2048 x 11008            8.7      9.0  6.8     6.5     7.6    14  above 16 rows narrow from 200 on
//   20, 28672 x 8192             63       43   26      83      79   155
//   32, 4096 x 4096                      7.8  6.2
//   32, 8192 x 28672                           35      32
//   64, 28672 x 8192            133       70           90      87   168
//   77, 28672 x 8192            162       98           74      88   170  narrow up to 256 tiles
//   192, 2048 x 11008            36       27           14      11    20
//   256, 8192 x 28672           495      234           97      66    74  wide from 160 tiles on
//   384, 8192 x 28672                                 144      94    77
//   1024, 2048 x 11008                                 33      29    27
Shape choose(int64_t rows, int64_t out, int64_t blocks) {
    const int64_t narrow = (out + Narrow::BW - 1) / Narrow::BW;
    if (rows <= 32 && blocks >= 8) {
        if (rows > 16) return narrow >= 200 ? kNarrow : kLong;
        if ((out + LongRows::BW - 1) / LongRows::BW < 256) return kFew;
        return (narrow >= 200 && blocks < 128) || (narrow >= 800 && (blocks <= 128 || rows > 8)) ? kNarrow : kLong;
    }
    if (rows <= Narrow::BX) {
        if (narrow >= 200 || (rows > 16 && narrow >= 80)) return kNarrow;
        return rows <= 16 ? kFew : kRows;
    }
    const int64_t wide = ((rows + Wide::BX - 1) / Wide::BX) * ((out + Wide::BW - 1) / Wide::BW);
    if (rows > Middle::BX && wide >= 160) return kWide;
    return ((rows + Narrow::BX - 1) / Narrow::BX) * narrow <= 256 ? kNarrow : kMiddle;
}

// A tile spans at most 2^30 bytes: 256 rows of 2^22 (2^23 columns). Rows farther
// apart take the shape of few rows, whatever their number: 1600 x 4096 x 1600 with
// rows 2^22 bytes apart 25 us, 16 bytes more 83 (2064 bytes: 19).
constexpr int64_t kTiledStride = int64_t(1) << 22;

}  // namespace

int launch_mx4_matmul(const Mx4& x, int64_t rows, const Mx4& w, int64_t out_features, int64_t blocks, void* y,
                      int y_dtype, int64_t y_stride, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int bf16 = y_dtype == ZS_DTYPE_BF16;
    const bool tiled = blocks > 0 && x.code_stride <= kTiledStride && w.code_stride <= kTiledStride;
    switch (tiled ? choose(rows, out_features, blocks) : kFew) {
        case kRows: return launch_rows(x, rows, w, out_features, blocks, y, bf16, y_stride, s);
        case kLong: return launch_long<LongRows>(x, rows, w, out_features, blocks, y, bf16, y_stride, s);
        case kNarrow: return launch_tiled<Narrow>(x, rows, w, out_features, blocks, y, bf16, y_stride, s);
        case kMiddle: return launch_tiled<Middle>(x, rows, w, out_features, blocks, y, bf16, y_stride, s);
        case kWide: return launch_tiled<Wide>(x, rows, w, out_features, blocks, y, bf16, y_stride, s);
        default: return launch_few(x, rows, w, out_features, blocks, y, bf16, y_stride, s);
    }
}

}  // namespace zs
