// Losses over rows of logits for CDNA4 (gfx950): log-probabilities of given
// tokens with entropy and the best alternatives, their gradient, and
// distillation from a teacher's top logits with its gradient.
//
// Every kernel is a stream over rows of `vocab` logits (2 or 4 bytes each)
// with one exponential and a few fp32 operations an element. Differences
// from the row's maximum are taken of the logits themselves, before the
// temperature scales them; exponentials are powers of two of differences scaled
// by log2(e) / temperature. A difference of more than fp32's largest value is
// -infinity and its exponential the 0 that it is; outputs that are differences
// over the temperature, and may be finite then, take halves (quotient()).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "zs_lm_internal.h"

namespace zs {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any multiple of the element's size: rows of an odd stride start
// anywhere (the hardware takes unaligned vector accesses).
typedef u32x4 __attribute__((aligned(2))) u32x4_u2;

constexpr float kInf = __builtin_inff();
constexpr float kLn2 = 0.693147180559945309f;
// Differences d are bounded below by this where they multiply 2^d, which is 0
// long before (and the products stay far from infinity).
constexpr float kLowest = -1.0e4f;

// (x - m) / temperature. Halves differ by no more than fp32's largest value, and
// halving is exact.
__device__ __forceinline__ float quotient(float x, float m, float inv_t) {
    return (0.5f * x - 0.5f * m) * (2.0f * inv_t);
}

__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FC00000u); }

// Two fp32 values as bf16 in one word, round to nearest even by the hardware's
// conversion (the one rounding of a stored gradient); NaN stays NaN.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// A 16-byte vector of logits as fp32 values and back.
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ float get(const u32x4& v, int i) {
        return __uint_as_float((i & 1) ? (v[i >> 1] & 0xFFFF0000u) : (v[i >> 1] << 16));
    }
    static __device__ __forceinline__ float one(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
    static __device__ __forceinline__ uint16_t round(float f) { return (uint16_t)pack_bf16(f, f); }
    static __device__ __forceinline__ u32x4 pack(const float* f) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        return v;
    }
    static constexpr uint32_t kNegInf = 0xFF80FF80u, kNan = 0x7FC07FC0u;
};
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ float get(const u32x4& v, int i) { return __uint_as_float(v[i]); }
    static __device__ __forceinline__ float one(float x) { return x; }
    static __device__ __forceinline__ float round(float f) { return f; }
    static __device__ __forceinline__ u32x4 pack(const float* f) {
        return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
    static constexpr uint32_t kNegInf = 0xFF800000u, kNan = 0x7FC00000u;
};

template <typename T>
__device__ __forceinline__ u32x4 load_vec(const T* p) {
    return *reinterpret_cast<const u32x4_u2*>(p);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, u32x4 v) {
    *reinterpret_cast<u32x4_u2*>(p) = v;
}

// Vector `first` + threadIdx.x of a row: the same row and `first` in the whole
// block, so that the address is a scalar and one 32-bit offset a thread.
template <typename T>
__device__ __forceinline__ u32x4 load_at(const T* row, int64_t first) {
    return *reinterpret_cast<const u32x4_u2*>(reinterpret_cast<const char*>(row) + first * 16 + threadIdx.x * 16u);
}
// NT: nontemporal.
template <bool NT, typename T>
__device__ __forceinline__ void store_at(T* row, int64_t first, u32x4 v) {
    u32x4_u2* p = reinterpret_cast<u32x4_u2*>(reinterpret_cast<char*>(row) + first * 16 + threadIdx.x * 16u);
    if (NT)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}

// ------------------------------------------------------------------ reductions over lanes
// By data-parallel-primitive moves, an instruction a step (a shuffle through
// shared memory is an instruction, an address and its latency).

// v moved by CTRL; lanes that nothing moves into get `none`.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float moved(float v, float none) {
    return __uint_as_float(
        __builtin_amdgcn_update_dpp(__float_as_uint(none), __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
constexpr int kShr = 0x110, kMirror = 0x140, kHalfMirror = 0x141, kBcast15 = 0x142, kBcast31 = 0x143;
constexpr int kQuadSwap1 = 0xB1, kQuadSwap2 = 0x4E;  // lanes 1 0 3 2 and 2 3 0 1 of each four

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// Over the 64 lanes, the same in all: rows of 16 first, then across them.
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, moved<kShr + 1>(v, -kInf));
    v = fmaxf(v, moved<kShr + 2>(v, -kInf));
    v = fmaxf(v, moved<kShr + 4>(v, -kInf));
    v = fmaxf(v, moved<kShr + 8>(v, -kInf));
    v = fmaxf(v, moved<kBcast15, 0xA>(v, -kInf));
    v = fmaxf(v, moved<kBcast31, 0xC>(v, -kInf));
    return lane_value(v, 63);
}

__device__ __forceinline__ float wave_sum(float v) {
    v += moved<kShr + 1>(v, 0.0f);
    v += moved<kShr + 2>(v, 0.0f);
    v += moved<kShr + 4>(v, 0.0f);
    v += moved<kShr + 8>(v, 0.0f);
    v += moved<kBcast15, 0xA>(v, 0.0f);
    v += moved<kBcast31, 0xC>(v, 0.0f);
    return lane_value(v, 63);
}

// Over groups of W = 4, 8 or 16 lanes, the same in all of a group.
template <int W>
__device__ __forceinline__ float group_max(float v) {
    v = fmaxf(v, moved<kQuadSwap1>(v, v));
    v = fmaxf(v, moved<kQuadSwap2>(v, v));
    if (W > 4) v = fmaxf(v, moved<kHalfMirror>(v, v));
    if (W > 8) v = fmaxf(v, moved<kMirror>(v, v));
    return v;
}

template <int W>
__device__ __forceinline__ float group_sum(float v) {
    v += moved<kQuadSwap1>(v, v);
    v += moved<kQuadSwap2>(v, v);
    if (W > 4) v += moved<kHalfMirror>(v, v);
    if (W > 8) v += moved<kMirror>(v, v);
    return v;
}

// Gradients are not read here again: nontemporal stores leave the caches to the
// logits (4096 x 32000 bf16 87 us against 107, 1024 x 151936 fp32 321 against
// 381). Not where rows start inside a 16-byte unit: a line then takes two
// stores, and they no longer meet in a cache (301 x 100003 fp32 62 against 59).
__device__ __forceinline__ bool whole_units(const void* g) { return (reinterpret_cast<uintptr_t>(g) & 15) == 0; }

// ------------------------------------------------------------------ running softmax
// max m of the logits, s = sum of 2^((x - m) k) and t = sum of 2^d d with
// d = (x - m) k, k = log2(e) / temperature. d is bounded below in the product
// so that masked logits (d = -infinity, 2^d = 0) add 0; a NaN, or a difference
// of two infinities, makes s NaN.
struct Running {
    float m, s, t;
};

// m, or 0 where nothing has been seen yet (m = -infinity).
__device__ __forceinline__ float base_of(float m) { return m == -kInf ? 0.0f : m; }

// Moves r to the maximum m (>= r.m).
__device__ __forceinline__ void rebase(Running& r, float m, float k) {
    const float d = (r.m - base_of(m)) * k;
    const float c = exp2f(d);
    r.t = c * (r.t + r.s * fmaxf(d, kLowest));
    r.s = c * r.s;
    r.m = m;
}

__device__ __forceinline__ Running merge(Running a, Running b, float k) {
    const float m = fmaxf(a.m, b.m);
    rebase(a, m, k);
    rebase(b, m, k);
    return Running{m, a.s + b.s, a.t + b.t};
}

__device__ __forceinline__ void add_one(Running& r, float x, float k) {
    const float m = fmaxf(r.m, x);
    rebase(r, m, k);
    const float d = (x - base_of(m)) * k;
    const float e = exp2f(d);
    r.s += e;
    r.t += e * fmaxf(d, kLowest);
}

// The block's Running from its threads', the same in every thread; `part` may
// be used again after the next barrier.
template <int THREADS, int WAVES>
__device__ __forceinline__ Running block_merge(Running r, float k, Running (&part)[WAVES]) {
    static_assert(WAVES >= THREADS / 64, "an entry a wave");
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const Running o{__shfl_xor(r.m, d, 64), __shfl_xor(r.s, d, 64), __shfl_xor(r.t, d, 64)};
        r = merge(r, o, k);
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = r;
    __syncthreads();
    r = part[0];
    for (int w = 1; w < THREADS / 64; ++w) r = merge(r, part[w], k);
    return r;
}

// One thread's share of a row: vectors tid, tid + THREADS, ... and one element
// of the tail behind the last whole vector. Right for any logits.
template <typename T, int THREADS>
__device__ __forceinline__ Running row_running(const T* row, int64_t vocab, float k) {
    constexpr int N = Vec<T>::kN;
    const int64_t nv = vocab / N;
    Running r{-kInf, 0.0f, 0.0f};
    for (int64_t v = threadIdx.x; v < nv; v += THREADS) {
        const u32x4 x = load_vec(row + v * N);
        float m = r.m;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, Vec<T>::get(x, i));
        rebase(r, m, k);
        const float b = base_of(m);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float d = (Vec<T>::get(x, i) - b) * k;
            const float e = exp2f(d);
            r.s += e;
            r.t += e * fmaxf(d, kLowest);
        }
    }
    const int64_t tail = nv * N + threadIdx.x;
    if (tail < vocab) add_one(r, Vec<T>::one(row[tail]), k);
    return r;
}

// ------------------------------------------------------------------ running softmax, ordinary logits
// The same sums with one multiply-add a difference: relative to c, the rounded
// product of the maximum and k, d = x k - c is off by one rounding of d itself
// (that c is no exact multiple of k shifts every d alike). ENTROPY: t is kept.
// Products past fp32's range, infinities, NaN and maxima so large that the
// shift matters leave s 0, infinite or NaN, or are seen from the maximum
// (ordinary() is false): the row is then summed by row_running.
struct Fast {
    float m, c, s, t;
};

__device__ __forceinline__ float exp2_raw(float d) { return __builtin_amdgcn_exp2f(d); }

template <bool ENTROPY>
__device__ __forceinline__ void fast_rebase(Fast& r, float m, float k) {
    const float c = base_of(m) * k;
    const float d = r.m == -kInf ? 0.0f : r.c - c;  // nothing seen yet: s = t = 0
    const float f = exp2_raw(d);
    if (ENTROPY) r.t = f * (r.t + r.s * fmaxf(d, kLowest));
    r.s = f * r.s;
    r.m = m;
    r.c = c;
}

template <bool ENTROPY>
__device__ __forceinline__ Fast fast_merge(Fast a, Fast b, float k) {
    const float m = fmaxf(a.m, b.m);
    fast_rebase<ENTROPY>(a, m, k);
    fast_rebase<ENTROPY>(b, m, k);
    return Fast{a.m, a.c, a.s + b.s, a.t + b.t};
}

__device__ __forceinline__ Fast fast_one(float x, float k) {
    if (x == -kInf) return Fast{x, 0.0f, 0.0f, 0.0f};
    const float c = x * k;
    const float d = __builtin_fmaf(x, k, -c);  // the rounding of c
    const float e = exp2_raw(d);
    return Fast{x, c, e, e * d};
}

template <typename T, bool ENTROPY, int U>
__device__ __forceinline__ void fast_add(Fast& r, const u32x4 (&x)[U], float k) {
    constexpr int N = Vec<T>::kN;
    float m = r.m;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N; i += 2) m = fmaxf(fmaxf(m, Vec<T>::get(x[u], i)), Vec<T>::get(x[u], i + 1));
    fast_rebase<ENTROPY>(r, m, k);
    float t = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float s[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float d = __builtin_fmaf(Vec<T>::get(x[u], i), k, -r.c);
            s[i] = exp2_raw(d);
            if (ENTROPY) t = __builtin_fmaf(s[i], d, t);
        }
#pragma unroll
        for (int h = N / 2; h; h >>= 1)
#pragma unroll
            for (int i = 0; i < h; ++i) s[i] += s[i + h];
        r.s += s[0];
    }
    if (ENTROPY && __any(t != t)) {  // a masked logit (0 times an infinite d), which t has to leave out, or a NaN
        t = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            u32x4 z = x[u];
            asm("" : "+v"(z));  // worked out again: nothing is kept for this
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float d = __builtin_fmaf(Vec<T>::get(z, i), k, -r.c);
                t = __builtin_fmaf(exp2_raw(d), fmaxf(d, kLowest), t);
            }
        }
    }
    r.t += t;
}

// r and the row's vectors from `first` on, then its tail.
template <typename T, int THREADS, bool ENTROPY, int U>
__device__ __forceinline__ Fast fast_running(Fast r, const T* row, int first, int64_t vocab, float k) {
    constexpr int N = Vec<T>::kN;
    const int nv = (int)(vocab / N), tid = threadIdx.x;
    const uint32_t none = Vec<T>::kNegInf;
    int v = first;  // of the block's first thread
    u32x4 x[U];
    auto load = [&](u32x4(&to)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) to[u] = load_at(row, v + u * THREADS);
        v += U * THREADS;
    };
    if (v + U * THREADS <= nv) {  // whole groups, the next one's loads ahead of each group's arithmetic
        u32x4 y[U];
        load(x);
        while (true) {
            const bool more = v + U * THREADS <= nv;
            if (more) load(y);
            fast_add<T, ENTROPY>(r, x, k);
            if (!more) break;
            const bool again = v + U * THREADS <= nv;
            if (again) load(x);
            fast_add<T, ENTROPY>(r, y, k);
            if (!again) break;
        }
    }
    if (v < nv) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = u32x4{none, none, none, none};
            if (v + u * THREADS + tid < nv) x[u] = load_at(row, v + u * THREADS);
        }
        fast_add<T, ENTROPY>(r, x, k);
    }
    const int tail = nv * N + tid;
    if (tail < vocab) r = fast_merge<ENTROPY>(r, fast_one(Vec<T>::one(row[tail]), k), k);
    return r;
}

// A block's sums, a wave each, of either form. The forms differ in size, so
// the reductions take them as arrays whose length is checked.
template <int WAVES>
union BlockParts {
    Running any[WAVES];
    Fast fast[WAVES];
};

// The block's sums, the same in every thread: the maximum first, then each lane
// moves its sums to it once.
template <int THREADS, bool ENTROPY, int WAVES>
__device__ __forceinline__ Fast fast_block_merge(Fast r, float k, Fast (&part)[WAVES]) {
    constexpr int W = THREADS / 64;
    static_assert(WAVES >= W, "an entry a wave");
    fast_rebase<ENTROPY>(r, wave_max(r.m), k);
    r.s = wave_sum(r.s);
    if (ENTROPY) r.t = wave_sum(r.t);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = r;
    __syncthreads();
    r = part[threadIdx.x % W];
    fast_rebase<ENTROPY>(r, group_max<W>(r.m), k);
    r.s = group_sum<W>(r.s);
    if (ENTROPY) r.t = group_sum<W>(r.t);
    return r;
}

__device__ __forceinline__ bool ordinary(const Fast& r) {
    return r.s > 0.0f && r.s < kInf && fabsf(r.c) < 1048576.0f && r.t == r.t;
}

// Statistics of a row, the same in every thread of the block: its maximum, log
// s and t / s (d in powers of two), s relative to the maximum; own: this
// thread's largest logit.
struct RowStats {
    float m, logsum, mean_d, own;
};

template <typename T, int THREADS, bool ENTROPY>
__device__ __forceinline__ RowStats row_stats(const T* row, int64_t vocab, float k, BlockParts<THREADS / 64>& part) {
    const Fast own = fast_running<T, THREADS, ENTROPY, 4>(Fast{-kInf, 0.0f, 0.0f, 0.0f}, row, 0, vocab, k);
    const Fast r = fast_block_merge<THREADS, ENTROPY>(own, k, part.fast);
    if (ordinary(r)) {
        // from c to the maximum: x k - c = (x - m) k + (m k - c)
        const float shift = __builtin_fmaf(r.m, k, -r.c);
        return RowStats{r.m, logf(r.s) - kLn2 * shift, ENTROPY ? r.t / r.s - shift : 0.0f, own.m};
    }
    __syncthreads();  // every thread has read the block's parts
    const Running a = row_running<T, THREADS>(row, vocab, k);
    const Running b = block_merge<THREADS>(a, k, part.any);
    if (b.m == -kInf && b.s == 0.0f) return RowStats{-kInf, 0.0f, 0.0f, -kInf};
    if (!(b.s < kInf)) return RowStats{b.m, quiet_nan(), quiet_nan(), a.m};
    return RowStats{b.m, logf(b.s), b.t / b.s, a.m};
}

// ------------------------------------------------------------------ best alternatives

// Whether logit a of token i comes before logit b of token j.
__device__ __forceinline__ bool before(float a, int i, float b, int j) { return (a > b) | ((a == b) & (i < j)); }

// The same order as one number, larger first: the logit's bits, made to grow
// with it (-0 as +0), over the token's, made to shrink.
__device__ __forceinline__ uint64_t order_key(float x, int id) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    const uint32_t up = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return ((uint64_t)up << 32) | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ float key_logit(uint64_t key) {
    const uint32_t up = (uint32_t)(key >> 32);
    return __uint_as_float((up & 0x80000000u) ? up ^ 0x80000000u : ~up);
}
__device__ __forceinline__ int key_token(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

// The thread's first element that comes after (x0, i0) in the order of
// `before`; token INT32_MAX if there is none.
template <typename T, int THREADS>
__device__ __forceinline__ void next_own(const T* row, int64_t vocab, float x0, int i0, float* best,
                                         int* best_i) {
    constexpr int N = Vec<T>::kN;
    const int64_t nv = vocab / N;
    float b = -kInf;
    int bi = INT32_MAX;
    for (int64_t v = threadIdx.x; v < nv; v += THREADS) {
        const u32x4 x = load_vec(row + v * N);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float f = Vec<T>::get(x, i);
            const int at = (int)(v * N) + i;
            if (before(x0, i0, f, at) && before(f, at, b, bi)) {
                b = f;
                bi = at;
            }
        }
    }
    const int64_t tail = nv * N + threadIdx.x;
    if (tail < vocab) {
        const float f = Vec<T>::one(row[tail]);
        if (before(x0, i0, f, (int)tail) && before(f, (int)tail, b, bi)) {
            b = f;
            bi = (int)tail;
        }
    }
    *best = b;
    *best_i = bi;
}

// The row's `top` best elements by rounds: every thread holds the best of its
// own elements that has not been taken, the best of those is taken, and the
// thread it came from looks for its next. Right for any row (equal or masked
// logits included). Every logit is below +infinity and no NaN.
template <typename T, int THREADS, typename Put>
__device__ __forceinline__ void top_by_rounds(const T* row, int64_t vocab, int top, float* lx, int* li, Put put) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float b;
    int bi;
    next_own<T, THREADS>(row, vocab, kInf, -1, &b, &bi);
    for (int n = 0; n < top; ++n) {
        float x = b;
        int i = bi;
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            const float ox = __shfl_xor(x, d, 64);
            const int oi = __shfl_xor(i, d, 64);
            if (before(ox, oi, x, i)) {
                x = ox;
                i = oi;
            }
        }
        if (lane == 0) {
            lx[wave] = x;
            li[wave] = i;
        }
        __syncthreads();
        for (int w = 0; w < THREADS / 64; ++w)
            if (before(lx[w], li[w], x, i)) {
                x = lx[w];
                i = li[w];
            }
        __syncthreads();
        if (threadIdx.x == 0) put(n, x, i);
        if (bi == i) next_own<T, THREADS>(row, vocab, x, i, &b, &bi);
    }
}

// The row's `top` best elements, put(place, logit, token) for each; own: this
// thread's largest logit. 64 groups of threads cover the row; the
// top-th largest of the groups' maxima, or a little less, is a bound that at
// least `top` elements reach and, the elements being spread over the groups, few more do: the
// elements of the threads whose own maximum reaches it are read again (they
// come from a cache), those that reach it are listed, and the list is ranked by
// counting. The second reading is dealt out over the whole block: left to the
// threads themselves it was a chain of loads a few lanes wide. A
// row with more of them than the list holds (equal logits, an order by size)
// goes by rounds. Where fewer than `top` groups hold a logit above -infinity (most
// of the vocabulary is masked), all that are above it are listed (10 tokens of
// 128256 allowed, 20 alternatives, bf16: 17 us for one row; by rounds 347).
constexpr int kListed = 512;
struct TopShared {
    float group[64];
    uint64_t key[kListed];  // order_key of the listed elements
    float best[16];         // of the waves, for top_by_rounds
    int best_id[16];
    int owner[1024];
    int n, owners;
};

// The bound; sh.n and sh.owners are 0 afterwards.
template <int THREADS>
__device__ __forceinline__ float top_bound(int top, float own, TopShared& sh) {
    constexpr int kGroup = THREADS / 64;  // threads a group
    const int lane = threadIdx.x & 63;
    const float g = group_max<kGroup>(own);
    if (threadIdx.x % kGroup == 0) sh.group[threadIdx.x / kGroup] = g;
    if (threadIdx.x == 0) sh.n = sh.owners = 0;
    __syncthreads();
    // the largest number of 16 leading bits that at least `top` groups' maxima
    // reach, in the order of order_key
    const uint32_t key = (uint32_t)(order_key(sh.group[lane], 0) >> 32);
    uint32_t reach = 0;
    for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1)
        if ((int)__popcll(__ballot(key >= (reach | bit))) >= top) reach |= bit;
    // nothing lies between -infinity and the first 16 bits' value below it
    return reach <= 0x007F0000u ? -kInf : key_logit((uint64_t)reach << 32);
}

__device__ __forceinline__ void top_list(float f, int at, TopShared& sh) {
    const int n = atomicAdd(&sh.n, 1);
    if (n < kListed) sh.key[n] = order_key(f, at);
}

// Ranks the list.
template <typename T, int THREADS, typename Put>
__device__ __forceinline__ void top_rank(const T* row, int64_t vocab, int top, TopShared& sh, Put put) {
    const int lane = threadIdx.x & 63;
    __syncthreads();
    const int n = sh.n;
    if (n > kListed) {
        __syncthreads();
        top_by_rounds<T, THREADS>(row, vocab, top, sh.best, sh.best_id, put);
        return;
    }
    if (n <= 64) {  // the usual list: one wave, an entry a lane
        if (threadIdx.x >= 64) return;
        if (n < top) {
            // every logit above -infinity is listed: the places left go to the
            // lowest masked tokens, which are among the first `top`
            const bool masked = lane < top && Vec<T>::one(row[lane]) == -kInf;
            const int at = n + (int)__popcll(__ballot(masked) & ((1ull << lane) - 1));
            if (masked && at < top) put(at, -kInf, lane);
        }
        const uint64_t key = sh.key[lane];
        int place = 0;
        for (int o = 0; o < n; ++o) {
            const uint64_t other = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(key >> 32), o) << 32) |
                                   (uint32_t)__builtin_amdgcn_readlane((int)key, o);
            place += other > key;
        }
        if (lane < n && place < top) put(place, key_logit(key), key_token(key));
        return;
    }
    for (int c = threadIdx.x; c < n; c += THREADS) {
        const uint64_t key = sh.key[c];
        int place = 0;
#pragma unroll 8
        for (int o = 0; o < n; ++o) place += sh.key[o] > key;
        if (place < top) put(place, key_logit(key), key_token(key));
    }
}

template <typename T, int THREADS, typename Put>
__device__ __forceinline__ void top_elements(const T* row, int64_t vocab, int top, float own, TopShared& sh, Put put) {
    constexpr int N = Vec<T>::kN;
    const float bound = fmaxf(top_bound<THREADS>(top, own, sh), -FLT_MAX);
    const int64_t nv = vocab / N;
    if (own >= bound) {
        sh.owner[atomicAdd(&sh.owners, 1)] = threadIdx.x;
        const int64_t tail = nv * N + threadIdx.x;
        if (tail < vocab) {
            const float f = Vec<T>::one(row[tail]);
            if (f >= bound) top_list(f, (int)tail, sh);
        }
    }
    __syncthreads();
    // the listed threads' vectors, dealt out over the block: vector j of thread
    // o is o + j * THREADS
    const unsigned per = (unsigned)((nv + THREADS - 1) / THREADS), all = per * sh.owners;
    constexpr int U = 4;
    for (unsigned p0 = threadIdx.x; p0 < all; p0 += U * THREADS) {
        u32x4 x[U];
        int64_t v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned p = p0 + u * THREADS;
            const uint32_t none = Vec<T>::kNan;
            v[u] = p < all ? sh.owner[p / per] + (int64_t)(p % per) * THREADS : nv;
            x[u] = u32x4{none, none, none, none};
            if (v[u] < nv) x[u] = load_vec(row + v[u] * N);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            unsigned reach = 0;  // few do: those are read once more rather than picked from registers
#pragma unroll
            for (int i = 0; i < N; ++i) reach |= Vec<T>::get(x[u], i) >= bound ? 1u << i : 0u;
            for (; reach; reach &= reach - 1) {
                const int at = (int)v[u] * N + __ffs(reach) - 1;
                top_list(Vec<T>::one(row[at]), at, sh);
            }
        }
    }
    top_rank<T, THREADS>(row, vocab, top, sh, put);
}

// ------------------------------------------------------------------ log-probabilities

// The outputs of a row that is skipped.
__device__ __forceinline__ void skipped_row(int64_t r, const LogprobsOut& out) {
    if (threadIdx.x == 0) {
        if (out.logprob) out.logprob[r] = 0.0f;
        if (out.entropy) out.entropy[r] = 0.0f;
        if (out.stats) out.stats[2 * r] = out.stats[2 * r + 1] = 0.0f;
    }
    if ((int)threadIdx.x < out.top) {
        out.top_ids[r * out.top + threadIdx.x] = -1;
        out.top_logprobs[r * out.top + threadIdx.x] = 0.0f;
    }
}

// The given token's logit, NaN where it is past the vocabulary.
template <typename T>
__device__ __forceinline__ float token_logit(const T* row, int64_t token, int64_t vocab) {
    return token < vocab ? Vec<T>::one(row[token]) : quiet_nan();
}

// A row's outputs but for its alternatives; those too where it has none (a NaN
// or +infinity in the row: log s is NaN). x: the given token's logit.
__device__ __forceinline__ void row_outputs(int64_t r, const RowStats& st, float x, float inv_t,
                                            const LogprobsOut& out) {
    if (threadIdx.x == 0) {
        // m is -infinity in a row of nothing else and in one with a NaN beside (log s is NaN)
        const bool masked = st.m == -kInf && st.logsum == 0.0f && x == -kInf;
        if (out.logprob) out.logprob[r] = masked ? -kInf : quotient(x, st.m, inv_t) - st.logsum;
        if (out.entropy) out.entropy[r] = st.logsum - kLn2 * st.mean_d;
        if (out.stats) {
            out.stats[2 * r] = st.m;
            out.stats[2 * r + 1] = st.logsum;
        }
    }
    if (!(st.logsum < kInf) && (int)threadIdx.x < out.top) {
        out.top_ids[r * out.top + threadIdx.x] = -1;
        out.top_logprobs[r * out.top + threadIdx.x] = quiet_nan();
    }
}

template <typename T, int THREADS, bool ENTROPY>
__global__ __launch_bounds__(THREADS) void k_logprobs(const T* __restrict__ logits, int64_t stride, int64_t vocab,
                                                      const int32_t* __restrict__ tokens, float inv_t, float k,
                                                      LogprobsOut out) {
    __shared__ BlockParts<THREADS / 64> part;
    __shared__ TopShared sh;
    const int64_t r = blockIdx.x;
    const T* row = logits + r * stride;
    const int64_t token = tokens[r];
    if (token < 0) {
        skipped_row(r, out);
        return;
    }
    const float x = token_logit(row, token, vocab);
    const RowStats st = row_stats<T, THREADS, ENTROPY>(row, vocab, k, part);
    row_outputs(r, st, x, inv_t, out);
    if (out.top == 0 || !(st.logsum < kInf)) return;
    top_elements<T, THREADS>(row, vocab, out.top, st.own, sh, [&](int place, float x, int id) {
        out.top_ids[r * out.top + place] = id;
        out.top_logprobs[r * out.top + place] = st.m == -kInf ? -kInf : quotient(x, st.m, inv_t) - st.logsum;
    });
}

// ------------------------------------------------------------------ gradient of the log-probabilities

constexpr int kGradThreads = 256;
constexpr int kGradU = 2;  // vectors a thread handles (4096 x 128256 bf16 347 us; 4: 362, 8: 394)

// What bounds this kernel once it streams is arithmetic beside the exponential:
// with d = x k - c, c the rounded product of the maximum and k, everything else
// of p = 2^d P and of the factor gl + gh (l + H) = G d + B is a constant of the
// row (2048 x 151936 bf16: 208 us; 220 with the formula for each element and a
// comparison of its index with the token). Rows whose maximum is out of that
// form's range take the formula.
template <typename T, bool ENTROPY>
__global__ __launch_bounds__(kGradThreads) void k_logprobs_grad(const T* logits, int64_t stride, int64_t vocab,
                                                                unsigned tiles, float inv_t, float k,
                                                                LogprobsGradIn in, T* grad, int64_t grad_stride) {
    constexpr int N = Vec<T>::kN;
    const int64_t r = blockIdx.x / tiles;
    const int tile = blockIdx.x % tiles;
    const T* row = logits + r * stride;
    T* g = grad + r * grad_stride;
    const int token = in.tokens[r];
    const float m = in.stats[2 * r], logsum = in.stats[2 * r + 1];
    const bool zero = token < 0 || (m == -kInf && logsum == 0.0f);
    const float gl = token >= vocab ? quiet_nan() : in.grad_logprob[r];
    const float gh = ENTROPY ? in.grad_entropy[r] : 0.0f;
    const float h = ENTROPY ? in.entropy[r] : 0.0f;
    const int nv = (int)(vocab / N), tid = threadIdx.x;
    const int v0 = tile * (kGradThreads * kGradU);
    const float hot = gl * inv_t;
    // value: the gradient of an element of logit x but for the given token's own
    // share. Vector by vector: with more loads in flight a thread, reads and
    // writes disturb each other more (4 vectors: 398 us against 362).
    auto write = [&](auto nt, auto value) {
#pragma unroll
        for (int u = 0; u < kGradU; ++u) {
            const int v = v0 + u * kGradThreads + tid;
            if (v < nv) {
                const u32x4 x = load_at(row, v0 + u * kGradThreads);
                float f[N];
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = value(Vec<T>::get(x, i));
                if (v == token / N && !zero) {
#pragma unroll
                    for (int i = 0; i < N; ++i) f[i] += i == token % N ? hot : 0.0f;
                }
                store_at<decltype(nt)::value>(g, v0 + u * kGradThreads, Vec<T>::pack(f));
            } else {
                const int j = nv * N + (v - nv);  // the tail's elements take the threads behind the last vector
                if (j < vocab) g[j] = Vec<T>::round(value(Vec<T>::one(row[j])) + (j == token && !zero ? hot : 0.0f));
            }
        }
    };
    auto write_aligned = [&](auto value) {
        if (whole_units(g))
            write(std::true_type{}, value);
        else
            write(std::false_type{}, value);
    };
    const float c = m * k;
    if (zero) {
        write_aligned([](float) { return 0.0f; });
    } else if (fabsf(c) < 1048576.0f) {
        const float rest = __builtin_fmaf(m, k, -c);  // x k - c = (x - m) k + rest
        const float a = -exp2f(-rest - logsum * (1.0f / kLn2)) * inv_t;
        if (ENTROPY) {
            const float b = gl + gh * (h - logsum - kLn2 * rest), slope = gh * kLn2;
            write_aligned([=](float x) {
                const float d = __builtin_fmaf(x, k, -c);
                return exp2_raw(d) * a * __builtin_fmaf(slope, fmaxf(d, kLowest), b);
            });
        } else {
            const float agl = a * gl;
            write_aligned([=](float x) { return exp2_raw(__builtin_fmaf(x, k, -c)) * agl; });
        }
    } else {
        write_aligned([=](float x) {
            const float d = x - m;
            const float p = exp2f(d * k - logsum * (1.0f / kLn2));
            return -p * (gl + gh * (fmaxf(d * inv_t - logsum, kLowest) + h)) * inv_t;
        });
    }
}

// ------------------------------------------------------------------ distillation

template <typename T>
__device__ __forceinline__ void fill_row(T* g, int64_t vocab, float f) {
    constexpr int N = Vec<T>::kN;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = f;
    const u32x4 x = Vec<T>::pack(v);
    const int64_t nv = vocab / N;
    for (int64_t j = threadIdx.x; j < nv; j += blockDim.x) store_vec(g + j * N, x);
    const int64_t tail = nv * N + threadIdx.x;
    if (tail < vocab) g[tail] = Vec<T>::round(f);
}

constexpr int kSlots = 2 * ZS_DISTILL_MAX_K;  // of the table that finds equal ids

struct DistillShared {
    float t[ZS_DISTILL_MAX_K];     // the teacher's logits, -infinity for unused entries
    float x[ZS_DISTILL_MAX_K];     // the student's logits at its tokens
    int32_t id[ZS_DISTILL_MAX_K];  // its tokens, -1 for unused entries
    int32_t slot[kSlots];
    int32_t repeated;
    BlockParts<1024 / 64> part;
};

// The teacher's side of a row: its largest logit, 1 / the sum of its
// exponentials and the log of that sum. Taken from shared memory by every wave
// for itself, which costs less than a barrier.
struct TeacherStats {
    float max, inv, logsum;
    bool bad;  // an id past the vocabulary, a NaN or +infinity
};

__device__ __forceinline__ TeacherStats teacher_stats(int n, int64_t vocab, float k, const DistillShared& sh) {
    const int lane = threadIdx.x & 63;
    float m = -kInf;
    bool bad = false;
    for (int i = lane; i < n; i += 64) {
        m = fmaxf(m, sh.t[i]);
        bad = bad || sh.id[i] >= vocab || !(sh.t[i] < kInf);
    }
    m = wave_max(m);
    float s = 0.0f;
    for (int i = lane; i < n; i += 64) s += exp2f((sh.t[i] - base_of(m)) * k);
    s = wave_sum(s);
    return TeacherStats{m, 1.0f / s, logf(s), (bool)__any(bad)};
}

// Losses are summed in units of 2^24: a difference of two logits over the
// smallest temperature is below 2^150, and in units of 2^24 in fp32's range.
constexpr float kLossUnit = 16777216.0f;

// loss / T^2 in that unit = sum of q ((t - max) / T - (x - m) / T + log s - log
// sum of the teacher's exponentials); one wave.
__device__ __forceinline__ float teacher_loss(int n, const TeacherStats& ts, float m, float logsum, float inv_t,
                                              float k, const DistillShared& sh) {
    float l = 0.0f;
    for (int i = threadIdx.x & 63; i < n; i += 64) {
        const float dt = sh.t[i] - ts.max;
        const float q = exp2f(dt * k) * ts.inv;
        const float half = 0.5f * dt - (0.5f * sh.x[i] - 0.5f * m);
        if (q > 0.0f) l += q * (half * (inv_t * (2.0f / kLossUnit)) + (logsum - ts.logsum) * (1.0f / kLossUnit));
    }
    return wave_sum(l);
}

// Marks sh.repeated where an id occurs twice: every used id goes into the first
// free slot from its own on (sh.slot is -1 everywhere, and twice as long as
// there can be ids).
template <int THREADS>
__device__ __forceinline__ void find_repeated(int n, DistillShared& sh) {
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const int id = sh.id[i];
        if (id < 0) continue;
        unsigned at = ((unsigned)id * 2654435761u) >> 21;
        static_assert(kSlots == 1 << 11, "11 bits");
        for (int tries = 0; tries < kSlots; ++tries) {
            const int old = atomicCAS(&sh.slot[at], -1, id);
            if (old == -1) break;
            if (old == id) {
                sh.repeated = 1;
                break;
            }
            at = (at + 1) % kSlots;
        }
    }
}

// The entries' tokens are written again with the teacher's share, once for each
// token by the first of its entries. p(x): the student's share of the
// gradient. Behind a barrier after the row's gradient and find_repeated.
template <typename T, int THREADS, typename P>
__device__ __forceinline__ void teacher_gradient(int n, const TeacherStats& ts, float k, float scale, T* g,
                                                 const DistillShared& sh, P p) {
    const bool repeated = sh.repeated != 0;
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const int id = sh.id[i];
        if (id < 0) continue;
        float q = exp2f((sh.t[i] - ts.max) * k);
        if (repeated) {
            q = 0.0f;
            bool first = true;
            for (int j = 0; j < n; ++j) {
                if (sh.id[j] != id) continue;
                first = first && j >= i;
                q += exp2f((sh.t[j] - ts.max) * k);
            }
            if (!first) continue;
        }
        g[id] = Vec<T>::round(p(sh.x[i]) - scale * (q * ts.inv));
    }
}

// g = p(row) over the row's whole vectors from `first` on, a group's loads ahead of its
// arithmetic; g may be row.
template <typename T, int THREADS, bool NT, typename P>
__device__ __forceinline__ void map_row_as(const T* row, T* g, int first, int nv, P p) {
    constexpr int N = Vec<T>::kN;
    constexpr int U = 4;
    const int tid = threadIdx.x;
    for (int v = first; v < nv; v += U * THREADS) {
        u32x4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * THREADS + tid < nv) x[u] = load_at(row, v + u * THREADS);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v + u * THREADS + tid >= nv) break;
            float o[N];
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = p(Vec<T>::get(x[u], j));
            store_at<NT>(g, v + u * THREADS, Vec<T>::pack(o));
        }
    }
}

template <typename T, int THREADS, typename P>
__device__ __forceinline__ void map_row(const T* row, T* g, int first, int nv, P p) {
    if (first >= nv) return;
    if (whole_units(g))
        map_row_as<T, THREADS, true>(row, g, first, nv, p);
    else
        map_row_as<T, THREADS, false>(row, g, first, nv, p);
}

// One block per row. The row's first vectors, NV a thread, are held in registers
// between the pass that sums their exponentials as they arrive and the pass
// that writes the gradient, so they are read once; what lies behind them (in
// rows longer than a compute unit's registers hold) is read again.
template <typename T, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void k_distill(const T* logits, int64_t stride, int64_t vocab, Teacher te,
                                                     float temperature, float inv_t, float k,
                                                     float* __restrict__ loss, T* grad, int64_t grad_stride) {
    constexpr int N = Vec<T>::kN;
    __shared__ DistillShared sh;
    const int64_t r = blockIdx.x;
    const T* row = logits + r * stride;
    T* g = grad + r * grad_stride;
    const float w = te.row_weight ? te.row_weight[r] : 1.0f;
    if (w == 0.0f) {
        if (threadIdx.x == 0) loss[r] = 0.0f;
        if (grad) fill_row(g, vocab, 0.0f);
        return;
    }
    const int nv = (int)(vocab / N), tid = threadIdx.x;
    const int tail = nv * N + tid;
    const int n = te.k;
    // The teacher's entries, an entry a thread (more threads than entries, or
    // up to 4 a thread), asked for before the row and put down behind it.
    const int32_t* ids = te.ids + r * n;
    const float* tl = te.logits + r * n;
    int32_t id = -1;
    float t = -kInf, z = 0.0f;
    if ((int)threadIdx.x < n) {
        id = ids[threadIdx.x];
        t = tl[threadIdx.x];
    }
    u32x4 x[NV];
    const uint32_t none = Vec<T>::kNegInf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        x[i] = u32x4{none, none, none, none};
        if (i * THREADS + tid < nv) x[i] = load_at(row, i * THREADS);
    }
    if (grad)
        for (int i = threadIdx.x; i < kSlots; i += THREADS) sh.slot[i] = -1;
    if (threadIdx.x == 0) sh.repeated = 0;
    auto put = [&](int i, int32_t id_i, float t_i, float x_i) {
        sh.id[i] = id_i < 0 ? -1 : id_i;
        sh.t[i] = id_i < 0 ? -kInf : t_i;
        sh.x[i] = x_i;
    };
    auto at = [&](int32_t j) { return j >= 0 && j < vocab ? Vec<T>::one(row[j]) : 0.0f; };
    if ((int)threadIdx.x < n) z = at(id);
    if (n > THREADS)
        for (int i = threadIdx.x + THREADS; i < n; i += THREADS) put(i, ids[i], tl[i], at(ids[i]));
    Fast f{-kInf, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
        u32x4 y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) y[u] = x[i + u];
        fast_add<T, false>(f, y, k);
        __builtin_amdgcn_sched_barrier(0);  // the held vectors leave no registers for a second group in flight
    }
    f = fast_running<T, THREADS, false, NV >= 16 ? 2 : 4>(f, row, NV * THREADS, vocab, k);
    if ((int)threadIdx.x < n) put(threadIdx.x, id, t, z);
    f = fast_block_merge<THREADS, false>(f, k, sh.part.fast);  // its barrier publishes the entries
    const TeacherStats ts = teacher_stats(n, vocab, k, sh);
    if (ts.bad || ts.max == -kInf) {
        const float fill = ts.bad ? quiet_nan() : 0.0f;
        if (threadIdx.x == 0) loss[r] = fill;
        if (grad) fill_row(g, vocab, fill);
        return;
    }
    const float scale = w * temperature;
    if (ordinary(f)) {
        if (threadIdx.x < 64) {
            const float l = teacher_loss(n, ts, f.m, logf(f.s) - kLn2 * __builtin_fmaf(f.m, k, -f.c), inv_t, k, sh);
            if (threadIdx.x == 0) loss[r] = w * temperature * temperature * kLossUnit * l;
        }
        if (!grad) return;
        find_repeated<THREADS>(n, sh);
        const float c = scale / f.s;
        auto p = [&](float z) { return c * exp2_raw(__builtin_fmaf(z, k, -f.c)); };
        auto write = [&](auto nt) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float o[N];
                asm("" : "+v"(x[i]));  // unpacked again here: the first pass's fp32 values are not kept
#pragma unroll
                for (int j = 0; j < N; ++j) o[j] = p(Vec<T>::get(x[i], j));
                if (i * THREADS + tid < nv) store_at<decltype(nt)::value>(g, i * THREADS, Vec<T>::pack(o));
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (whole_units(g))
            write(std::true_type{});
        else
            write(std::false_type{});
        map_row<T, THREADS>(row, g, NV * THREADS, nv, p);
        if (tail < vocab) g[tail] = Vec<T>::round(p(Vec<T>::one(row[tail])));
        __syncthreads();
        teacher_gradient<T, THREADS>(n, ts, k, scale, g, sh, p);
        return;
    }
    // any other row: differences from the maximum first, the row read again
    __syncthreads();
    const Running a = block_merge<THREADS>(row_running<T, THREADS>(row, vocab, k), k, sh.part.any);
    const float m = base_of(a.m);
    if (threadIdx.x < 64) {
        const float l = teacher_loss(n, ts, m, logf(a.s), inv_t, k, sh);
        const bool masked = a.m == -kInf && a.s == 0.0f;
        if (threadIdx.x == 0) loss[r] = w * temperature * temperature * kLossUnit * (masked ? kInf : l);
    }
    if (!grad) return;
    find_repeated<THREADS>(n, sh);
    const float c = a.s == 0.0f ? 0.0f : scale / a.s;
    auto p = [&](float z) { return c * exp2f((z - m) * k); };
    map_row<T, THREADS>(row, g, 0, nv, p);
    if (tail < vocab) g[tail] = Vec<T>::round(p(Vec<T>::one(row[tail])));
    __syncthreads();
    teacher_gradient<T, THREADS>(n, ts, k, scale, g, sh, p);
}

}  // namespace

namespace {

template <typename T, int THREADS>
void run_logprobs(Rows logits, int64_t rows, int64_t vocab, const int32_t* tokens, double temperature,
                  const LogprobsOut& out, hipStream_t s) {
    const float inv_t = (float)(1.0 / temperature), k = (float)(M_LOG2E / temperature);
    const T* p = static_cast<const T*>(logits.p);
    if (out.entropy)
        hipLaunchKernelGGL((k_logprobs<T, THREADS, true>), dim3((unsigned)rows), dim3(THREADS), 0, s, p, logits.stride,
                           vocab, tokens, inv_t, k, out);
    else
        hipLaunchKernelGGL((k_logprobs<T, THREADS, false>), dim3((unsigned)rows), dim3(THREADS), 0, s, p,
                           logits.stride, vocab, tokens, inv_t, k, out);
}

}  // namespace

int launch_logprobs(Rows logits, int dtype, int64_t rows, int64_t vocab, const int32_t* tokens, double temperature,
                    const LogprobsOut& out, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    // 512 threads a row where rows are few or long, else 256. With 8
    // alternatives, 256 threads against 512, us: few rows 64 x 151936 fp32 23.2,
    // 16.5; about even at 512 rows of 128256 and 32000 bf16. 4096 rows of bf16:
    // 32768 53, 67; 49152 78, 82; 57344 90, 102; 65536 (128 KB) 104, 98; 81920 127,
    // 119. 4096 rows of fp32: 16384 52, 50; 20480 65, 64; 24576 (96 KB) 76, 72;
    // 28672 88, 83; 32768 101, 94. Without alternatives 512 threads gain 1 to 5%
    // from these lengths on.
    const bool bf16 = dtype == ZS_DTYPE_BF16;
    const int64_t row_bytes = vocab * (bf16 ? 2 : 4);
    const bool wide = vocab > 8192 && (rows <= 1024 || row_bytes >= (bf16 ? 128 << 10 : 96 << 10));
    if (bf16 && wide)
        run_logprobs<uint16_t, 512>(logits, rows, vocab, tokens, temperature, out, s);
    else if (bf16)
        run_logprobs<uint16_t, 256>(logits, rows, vocab, tokens, temperature, out, s);
    else if (wide)
        run_logprobs<float, 512>(logits, rows, vocab, tokens, temperature, out, s);
    else
        run_logprobs<float, 256>(logits, rows, vocab, tokens, temperature, out, s);
    return (int)hipGetLastError();
}

namespace {

template <typename T>
int run_grad(Rows logits, int64_t rows, int64_t vocab, double temperature, const LogprobsGradIn& in, void* grad,
             int64_t grad_stride, hipStream_t s) {
    constexpr int N = Vec<T>::kN;
    // the row's vectors, and one thread for each element of its tail
    const int64_t per = kGradThreads * kGradU;
    const int64_t tiles = (vocab / N + vocab % N + per - 1) / per;
    // a launch covers at most 2^32 - 1 work-items: 4 million rows of 16392 bf16
    // logits (137 GB, in place) take two
    const int64_t most = ((int64_t(1) << 32) - 1) / kGradThreads / tiles;
    const float inv_t = (float)(1.0 / temperature), k = (float)(M_LOG2E / temperature);
    for (int64_t r = 0; r < rows; r += most) {
        const T* p = static_cast<const T*>(logits.p) + r * logits.stride;
        T* g = static_cast<T*>(grad) + r * grad_stride;
        const LogprobsGradIn part{in.tokens + r, in.stats + 2 * r, in.entropy ? in.entropy + r : nullptr,
                                  in.grad_logprob + r, in.grad_entropy ? in.grad_entropy + r : nullptr};
        const dim3 grid((unsigned)((rows - r < most ? rows - r : most) * tiles));
        if (in.grad_entropy)
            hipLaunchKernelGGL((k_logprobs_grad<T, true>), grid, dim3(kGradThreads), 0, s, p, logits.stride, vocab,
                               (unsigned)tiles, inv_t, k, part, g, grad_stride);
        else
            hipLaunchKernelGGL((k_logprobs_grad<T, false>), grid, dim3(kGradThreads), 0, s, p, logits.stride, vocab,
                               (unsigned)tiles, inv_t, k, part, g, grad_stride);
        if (const hipError_t e = hipGetLastError()) return (int)e;
    }
    return (int)hipSuccess;
}

}  // namespace

int launch_logprobs_grad(Rows logits, int dtype, int64_t rows, int64_t vocab, double temperature,
                         const LogprobsGradIn& in, void* grad, int64_t grad_stride, void* stream) {
    if (dtype == ZS_DTYPE_BF16)
        return run_grad<uint16_t>(logits, rows, vocab, temperature, in, grad, grad_stride, (hipStream_t)stream);
    return run_grad<float>(logits, rows, vocab, temperature, in, grad, grad_stride, (hipStream_t)stream);
}

namespace {

template <typename T, int THREADS, int NV>
void run_distill(Rows logits, int64_t rows, int64_t vocab, const Teacher& t, double temperature, float* loss,
                 void* grad, int64_t grad_stride, hipStream_t s) {
    hipLaunchKernelGGL((k_distill<T, THREADS, NV>), dim3((unsigned)rows), dim3(THREADS), 0, s,
                       static_cast<const T*>(logits.p), logits.stride, vocab, t, (float)temperature,
                       (float)(1.0 / temperature), (float)(M_LOG2E / temperature), loss, static_cast<T*>(grad),
                       grad_stride);
}

template <typename T>
int pick_distill(Rows logits, int64_t rows, int64_t vocab, const Teacher& t, double temperature, float* loss,
                 void* grad, int64_t grad_stride, hipStream_t s) {
    // As many threads and vectors a thread as hold the row; 20 vectors are what
    // 1024 threads have registers for (4096 x 151936 bf16, 19 vectors: 487 us,
    // read twice 549; 1024 x 151936 fp32, 20 of 38 held: 271 us against 330, 252 now).
    const int64_t nv = vocab / Vec<T>::kN;  // 16-byte vectors of a row
    if (nv <= 256 * 4)
        run_distill<T, 256, 4>(logits, rows, vocab, t, temperature, loss, grad, grad_stride, s);
    else if (nv <= 512 * 8)
        run_distill<T, 512, 8>(logits, rows, vocab, t, temperature, loss, grad, grad_stride, s);
    else if (nv <= 512 * 16)
        run_distill<T, 512, 16>(logits, rows, vocab, t, temperature, loss, grad, grad_stride, s);
    else if (nv <= 1024 * 16)
        run_distill<T, 1024, 16>(logits, rows, vocab, t, temperature, loss, grad, grad_stride, s);
    else
        run_distill<T, 1024, 20>(logits, rows, vocab, t, temperature, loss, grad, grad_stride, s);
    return (int)hipGetLastError();
}

}  // namespace

int launch_distill(Rows logits, int dtype, int64_t rows, int64_t vocab, const Teacher& t, double temperature,
                   float* loss, void* grad, int64_t grad_stride, void* stream) {
    if (dtype == ZS_DTYPE_BF16)
        return pick_distill<uint16_t>(logits, rows, vocab, t, temperature, loss, grad, grad_stride,
                                      (hipStream_t)stream);
    return pick_distill<float>(logits, rows, vocab, t, temperature, loss, grad, grad_stride, (hipStream_t)stream);
}

}  // namespace zs
