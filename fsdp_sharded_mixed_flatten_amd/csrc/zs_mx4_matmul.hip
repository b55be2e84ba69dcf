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

// ------------------------------------------------------------------ many rows
// A workgroup computes a tile of BM rows of x by BN of W, its WM x WN waves
// 32 TM x 32 TN each. Both sides' codes go through shared memory, 256 columns
// at a time, straight from global memory: the next 256 are on their way while
// the present ones are multiplied. A row's 128 bytes are eight 16-byte blocks,
// and block c of row r lies at place c ^ (r % 8), so that lanes that read one
// block of many rows spread over the banks.
// A lane of a 32 x 32 instruction gives block l / 32 of row l % 32. Which 64
// columns an instruction takes is free as long as both sides agree: the lower
// lanes take blocks 0 to 3 of the eight in their four turns and the upper ones 4
// to 7, so that a lane's four scales are one word, whose bytes the
// instruction's operand selection picks.
template <int TM_, int TN_, int WM_, int WN_>
struct Tile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_;
    static constexpr int kThreads = 64 * WM * WN, BM = 32 * TM * WM, BN = 32 * TN * WN;
    static constexpr int kUnits = (BM + BN) * 8 / kThreads;  // 16-byte loads of a thread a turn
    static_assert(BM * 8 % kThreads == 0 && BN * 8 % kThreads == 0 && kThreads % 64 == 0, "whole loads");
};

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int STEP>
__device__ __forceinline__ f32x16 mfma32(const u32x4& x, uint32_t sx, const u32x4& w, uint32_t sw, f32x16 acc) {
    const i32x8 a{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    const i32x8 b{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, kFp4, kFp4, STEP, (int)sx, STEP, (int)sw);
}

typedef __attribute__((address_space(3))) void* lds_ptr;

template <typename T>
struct Shared {
    u32x4 codes[2][(T::BM + T::BN) * 8];
    uint32_t scales[2][4][T::BM + T::BN];
};

template <typename T, int STEP>
__device__ __forceinline__ void turn_step(const u32x4* x, const u32x4* w, const uint32_t* sx, const uint32_t* sw,
                                          int half, f32x16 (&acc)[T::TM][T::TN]) {
    const int r = threadIdx.x & 31, place = (4 * half + STEP) ^ (r & 7);
    u32x4 a[T::TM], b[T::TN];
#pragma unroll
    for (int i = 0; i < T::TM; ++i) a[i] = x[(32 * i + r) * 8 + place];
#pragma unroll
    for (int j = 0; j < T::TN; ++j) b[j] = w[(32 * j + r) * 8 + place];
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j) acc[i][j] = mfma32<STEP>(a[i], sx[i], b[j], sw[j], acc[i][j]);
}

// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ char* uniform(const void* p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
    return reinterpret_cast<char*>(((uintptr_t)hi << 32) | lo);
}

template <typename T>
__global__ __launch_bounds__(T::kThreads) void k_mx4_tiled(Mx4 x, int rows, Mx4 w, int out, int blocks,
                                                           void* __restrict__ y, int y_bf16, int64_t y_stride,
                                                           int tiles_m) {
    __shared__ Shared<T> sh;
    const int tid = threadIdx.x, half = (tid & 63) >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tile = blockIdx.x;
    const int r0 = tile % tiles_m * T::BM, o0 = tile / tiles_m * T::BN;
    const int mine_x = min(rows - r0, T::BM), mine_w = min(out - o0, T::BN);
    const int xs = (int)x.code_stride, ws = (int)w.code_stride;
    // what a load leaves out (rows past the end, blocks past the last) is asked
    // for behind the buffer's end, where a load gives 0
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
        uniform(static_cast<const char*>(x.codes) + r0 * x.code_stride), (short)0, (mine_x - 1) * xs + blocks * 16,
        0x00020000);
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        uniform(static_cast<const char*>(w.codes) + o0 * w.code_stride), (short)0, (mine_w - 1) * ws + blocks * 16,
        0x00020000);
    constexpr int kNowhere = 0x7FFFFFF0;
    const int lrow = tid >> 3, lblock = (tid & 7) ^ (lrow & 7);
    auto fetch = [&](int turn, int stage) {
        const bool in = turn * 8 + lblock < blocks;
        const int col = (turn * 8 + lblock) * 16;
#pragma unroll
        for (int u = 0; u < T::BM * 8 / T::kThreads; ++u) {
            const int row = u * (T::kThreads / 8) + lrow;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_ptr)&sh.codes[stage][u * T::kThreads + wave * 64], 16,
                                                     in && row < mine_x ? row * xs + col : kNowhere, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < T::BN * 8 / T::kThreads; ++u) {
            const int row = u * (T::kThreads / 8) + lrow;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                wr, (lds_ptr)&sh.codes[stage][T::BM * 8 + u * T::kThreads + wave * 64], 16,
                in && row < mine_w ? row * ws + col : kNowhere, 0, 0, 0);
        }
    };
    // scales of 512 columns of a row: 16 bytes, through registers
    constexpr int kScaleRows = (T::BM + T::BN) / T::kThreads;
    static_assert(kScaleRows * T::kThreads == T::BM + T::BN, "a thread fetches the scales of whole rows");
    u32x4 held[kScaleRows];
    const uint8_t* sp[kScaleRows];
#pragma unroll
    for (int k = 0; k < kScaleRows; ++k) {
        const int row = k * T::kThreads + tid;
        sp[k] = row < T::BM ? static_cast<const uint8_t*>(x.scales) + (r0 + min(row, mine_x - 1)) * x.scale_stride
                            : static_cast<const uint8_t*>(w.scales) + (o0 + min(row - T::BM, mine_w - 1)) * w.scale_stride;
    }
    auto fetch_scales = [&](int pair) {
        if ((pair + 1) * 16 <= blocks) {
#pragma unroll
            for (int k = 0; k < kScaleRows; ++k) held[k] = *reinterpret_cast<const u32x4_u1*>(sp[k] + pair * 16);
        } else {  // the last, byte by byte; nothing reads this half of sh.scales now
#pragma unroll
            for (int k = 0; k < kScaleRows; ++k) {
                uint8_t* to = reinterpret_cast<uint8_t*>(&sh.scales[pair & 1][0][k * T::kThreads + tid]);
                uint8_t b[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) b[i] = sp[k][min(pair * 16 + i, blocks - 1)];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    to[i / 4 * 4 * (T::BM + T::BN) + i % 4] = pair * 16 + i < blocks ? b[i] : (uint8_t)127;
            }
        }
    };
    auto put_scales = [&](int pair) {
        if ((pair + 1) * 16 <= blocks) {
#pragma unroll
            for (int k = 0; k < kScaleRows; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) sh.scales[pair & 1][i][k * T::kThreads + tid] = held[k][i];
        }
    };
    f32x16 acc[T::TM][T::TN];
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j) acc[i][j] = f32x16{};
    const int wm = wave % T::WM, wn = wave / T::WM;
    const int turns = (blocks + 7) / 8;
    fetch(0, 0);
    fetch_scales(0);
    put_scales(0);
    for (int t = 0; t < turns; ++t) {
        __syncthreads();  // turn t's codes and scales are there, turn t - 1's no longer read
        const int stage = t & 1, pair = t >> 1;
        if (t + 1 < turns) fetch(t + 1, stage ^ 1);
        if (stage == 0 && t + 2 < turns) fetch_scales(pair + 1);
        uint32_t sx[T::TM], sw[T::TN];
        const uint32_t* plane = sh.scales[pair & 1][2 * stage + half];
#pragma unroll
        for (int i = 0; i < T::TM; ++i) sx[i] = plane[32 * (wm * T::TM + i) + (tid & 31)];
#pragma unroll
        for (int j = 0; j < T::TN; ++j) sw[j] = plane[T::BM + 32 * (wn * T::TN + j) + (tid & 31)];
        const u32x4* xt = sh.codes[stage] + 32 * wm * T::TM * 8;
        const u32x4* wt = sh.codes[stage] + (T::BM + 32 * wn * T::TN) * 8;
        turn_step<T, 0>(xt, wt, sx, sw, half, acc);
        turn_step<T, 1>(xt, wt, sx, sw, half, acc);
        turn_step<T, 2>(xt, wt, sx, sw, half, acc);
        turn_step<T, 3>(xt, wt, sx, sw, half, acc);
        if (stage == 1 && t + 1 < turns) put_scales(pair + 1);
    }
    // lane l has column l % 32 and rows 8 * (e / 4) + 4 * (l / 32) + e % 4
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j) {
            const int col = o0 + 32 * (wn * T::TN + j) + (tid & 31);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = r0 + 32 * (wm * T::TM + i) + 8 * (e / 4) + 4 * half + e % 4;
                if (row < rows && col < out) store_y(y, y_bf16, row * y_stride + col, acc[i][j][e]);
            }
        }
}

template <typename T>
int launch_tiled(const Mx4& x, int64_t rows, const Mx4& w, int64_t out, int64_t blocks, void* y, int y_bf16,
                 int64_t y_stride, hipStream_t s) {
    const int64_t tm = (rows + T::BM - 1) / T::BM, tn = (out + T::BN - 1) / T::BN;
    k_mx4_tiled<T><<<(unsigned)(tm * tn), T::kThreads, 0, s>>>(x, (int)rows, w, (int)out, (int)blocks, y, y_bf16, y_stride,
                                                              (int)tm);
    return (int)hipGetLastError();
}

}  // namespace

int launch_mx4_matmul(const Mx4& x, int64_t rows, const Mx4& w, int64_t out_features, int64_t blocks, void* y,
                      int y_dtype, int64_t y_stride, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int esz = y_dtype == ZS_DTYPE_BF16 ? 2 : 4;
    if (rows > 64 && blocks > 0 && x.code_stride <= (1 << 22) && w.code_stride <= (1 << 22))
        return launch_tiled<Tile<4, 4, 2, 2>>(x, rows, w, out_features, blocks, y, y_dtype == ZS_DTYPE_BF16, y_stride,
                                              s);
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
