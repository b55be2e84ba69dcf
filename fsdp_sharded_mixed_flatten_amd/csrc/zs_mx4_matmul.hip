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

// Four results side by side, `left` of which there are, k elements behind `at`.
// The hardware's conversion rounds to nearest even but for one value in 2^17 next
// to a tie, half a step and 2^-16 of one off.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_u2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_u4 __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
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
// A workgroup computes BW columns of y (rows of W) for BX rows of x, its WW x WX
// waves 32 TW x 32 TX each. Both sides' codes go straight from global to shared
// memory, 128 columns (a turn) at a time through a ring of four stages: while
// a turn is multiplied the next three are on their way or there. A row's 64
// bytes are four 16-byte blocks; block c of row r lies at place c ^ (r / 4 % 4),
// so that the sixteen lanes that are served together reach all banks.
// A lane of a 32 x 32 instruction gives one block of row l % 32. Which 64
// columns an instruction takes is free as long as both sides agree: the lower
// lanes take blocks 0 and 1 of a turn's four, the upper ones 2 and 3, so that a
// lane's two scales are neighbouring bytes, which the instruction's operand
// selection picks. W gives the rows of an instruction's result, so that a lane
// holds four columns of y side by side.
template <int TW_, int TX_, int WW_, int WX_>
struct Tile {
    static constexpr int TW = TW_, TX = TX_, WW = WW_, WX = WX_;
    static constexpr int kThreads = 64 * WW * WX, BW = 32 * TW * WW, BX = 32 * TX * WX, kRows = BW + BX;
    static constexpr int kLoads = kRows * 4 / kThreads;  // 16-byte loads of a thread a turn
    static constexpr int kScaleLoads = (kRows + kThreads - 1) / kThreads;
    static_assert(BW * 4 % kThreads == 0 && BX * 4 % kThreads == 0, "whole loads");
};

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int STEP>
__device__ __forceinline__ f32x16 mfma32(const u32x4& w, uint32_t sw, const u32x4& x, uint32_t sx, f32x16 acc) {
    const i32x8 a{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const i32x8 b{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, kFp4, kFp4, STEP, (int)sw, STEP, (int)sx);
}

typedef __attribute__((address_space(3))) void* lds_ptr;

template <typename T>
struct Shared {
    u32x4 codes[4][T::kRows * 4];
    uint32_t scales[2][4][T::kRows];  // of 512 columns, two of them in turn: a word a turn and row
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

template <typename T>
struct Tiled {
    Shared<T>& sh;
    __amdgpu_buffer_rsrc_t wr, xr;
    int blocks;
    int wave, lblock;           // the block of a turn that this thread's loads take
    uint32_t from[T::kLoads];   // and where in W and x they find it in turn 0
    int read_w, read_x;      // the row of a tile whose blocks this lane reads, times 4
    int swizzle, half;
    const uint8_t* scale_row[T::kScaleLoads];
    u32x4 held[T::kScaleLoads];

    // What a load leaves out (rows past the end, blocks past the last) is asked
    // for behind the buffer's end, where a load gives 0. Buffers are shorter than
    // 2^30 bytes and offsets inside them too, so that no sum passes 2^32.
    static constexpr uint32_t kNowhere = 0x7FFFFFF0u;
    static constexpr int kLoadRows = T::kThreads / 4;
    __device__ __forceinline__ void fetch(int turn, int stage) {
        const uint32_t add = turn * 4 + lblock < blocks ? turn * 64u : kNowhere;
#pragma unroll
        for (int u = 0; u < T::kLoads; ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(u < T::BW / kLoadRows ? wr : xr,
                                                     (lds_ptr)&sh.codes[stage][u * T::kThreads + wave * 64], 16,
                                                     (int)(from[u] + add), 0, 0, 0);
    }
    // Scales of 512 columns (16 bytes a row) go through registers.
    __device__ __forceinline__ void fetch_scales(int group) {
        if ((group + 1) * 16 <= blocks) {
#pragma unroll
            for (int k = 0; k < T::kScaleLoads; ++k)
                held[k] = *reinterpret_cast<const u32x4_u1*>(scale_row[k] + group * 16);
        } else {  // the last: what lies behind the row's end is 1
#pragma unroll
            for (int k = 0; k < T::kScaleLoads; ++k) {
                uint32_t b[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) b[i] = scale_row[k][min(group * 16 + i, blocks - 1)];
#pragma unroll
                for (int i = 0; i < 16; ++i) b[i] = group * 16 + i < blocks ? b[i] : 127;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    held[k][i] = b[4 * i] | (b[4 * i + 1] << 8) | (b[4 * i + 2] << 16) | (b[4 * i + 3] << 24);
            }
        }
    }
    __device__ __forceinline__ void put_scales(int group) {
#pragma unroll
        for (int k = 0; k < T::kScaleLoads; ++k) {
            const int row = k * T::kThreads + threadIdx.x;
            if (T::kRows % T::kThreads == 0 || row < T::kRows)
#pragma unroll
                for (int i = 0; i < 4; ++i) sh.scales[group & 1][i][row] = held[k][i];
        }
    }
    __device__ __forceinline__ void read(int stage, int step, Step<T>& f) const {
        const int place = (2 * half + step) ^ swizzle;
#pragma unroll
        for (int i = 0; i < T::TW; ++i) f.w[i] = sh.codes[stage][read_w + 128 * i + place];
#pragma unroll
        for (int i = 0; i < T::TX; ++i) f.x[i] = sh.codes[stage][4 * T::BW + read_x + 128 * i + place];
    }
    __device__ __forceinline__ void read_scales(int group, int turn, Scales<T>& s) const {
#pragma unroll
        for (int i = 0; i < T::TW; ++i) s.w[i] = sh.scales[group & 1][turn][read_w / 4 + 32 * i] >> (16 * half);
#pragma unroll
        for (int i = 0; i < T::TX; ++i) s.x[i] = sh.scales[group & 1][turn][T::BW + read_x / 4 + 32 * i] >> (16 * half);
    }
    template <int STEP>
    __device__ __forceinline__ void multiply(const Step<T>& f, const Scales<T>& s, f32x16 (&acc)[T::TW][T::TX]) const {
#pragma unroll
        for (int i = 0; i < T::TW; ++i)
#pragma unroll
            for (int j = 0; j < T::TX; ++j) acc[i][j] = mfma32<STEP>(f.w[i], s.w[i], f.x[j], s.x[j], acc[i][j]);
    }
};

// All but the N youngest of this wave's loads are there, and all waves are here.
// (A barrier of the language would wait for all loads.)
template <int N>
__device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename T>
__global__ __launch_bounds__(T::kThreads) void k_mx4_tiled(Mx4 x, int rows, Mx4 w, int out, int blocks,
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
    Tiled<T> t{sh,
               __builtin_amdgcn_make_buffer_rsrc(uniform(static_cast<const char*>(w.codes) + o0 * w.code_stride),
                                                 (short)0, (mine_w - 1) * ws + blocks * 16, 0x00020000),
               __builtin_amdgcn_make_buffer_rsrc(uniform(static_cast<const char*>(x.codes) + r0 * x.code_stride),
                                                 (short)0, (mine_x - 1) * xs + blocks * 16, 0x00020000),
               blocks, wave, (tid & 3) ^ (tid >> 4 & 3), {},
               4 * (32 * T::TW * wave_w + (lane & 31)), 4 * (32 * T::TX * wave_x + (lane & 31)), lane >> 2 & 3,
               lane >> 5, {}, {}};
#pragma unroll
    for (int u = 0; u < T::kLoads; ++u) {
        const int row = u * Tiled<T>::kLoadRows + (tid >> 2), in_x = row - T::BW;
        t.from[u] = row < T::BW ? (row < mine_w ? (uint32_t)(row * ws + t.lblock * 16) : Tiled<T>::kNowhere)
                                : (in_x < mine_x ? (uint32_t)(in_x * xs + t.lblock * 16) : Tiled<T>::kNowhere);
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

    const int groups = (blocks + 15) / 16;  // of four turns; turns behind the last block multiply zeros
    t.fetch_scales(0);
    t.put_scales(0);
    t.fetch(0, 0);
    t.fetch(1, 1);
    t.fetch(2, 2);
    t.fetch(3, 3);
    arrive<3 * T::kLoads>();
    Step<T> f[2];
    Scales<T> s[2];
    t.read(0, 0, f[0]);
    t.read_scales(0, 0, s[0]);
    for (int g = 0; g < groups; ++g) {
        // A turn's loads are asked for in order, so that waiting for all but the
        // youngest two turns' leaves the next turn's there. The scales of the
        // next group are asked for in the first turn and put down in the third;
        // they are younger than two turns' loads until the fourth turn waits.
        const int next = 4 * g + 4;
#pragma unroll
        for (int turn = 0; turn < 4; ++turn) {
            t.read(turn, 1, f[1]);
            t.template multiply<0>(f[0], s[turn & 1], acc);
            __builtin_amdgcn_sched_barrier(0);
            // the next turn's codes are there, and this one's have been read
            if (turn == 1 || turn == 2)
                arrive<2 * T::kLoads + T::kScaleLoads>();
            else
                arrive<2 * T::kLoads>();
            if (turn == 0) t.fetch_scales(g + 1 < groups ? g + 1 : g);
            if (turn == 2) t.put_scales(g + 1);
            t.fetch(next + turn, turn);
            t.read((turn + 1) & 3, 0, f[0]);
            t.read_scales(turn == 3 ? g + 1 : g, (turn + 1) & 3, s[(turn + 1) & 1]);
            t.template multiply<1>(f[1], s[turn & 1], acc);
            __builtin_amdgcn_sched_barrier(0);
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
