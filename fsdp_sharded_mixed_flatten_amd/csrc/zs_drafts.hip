// Verification of drafted tokens for CDNA4 (gfx950).
//
// A token is drawn where a running sum over the vocabulary passes a border that
// a random number sets. 151936 tokens of like probability have borders 7e-6
// apart, so that sums of fp32 exponentials would put one draw in a hundred on
// another side of a border than the definition does. Exponentials, their sums
// and the running sums are therefore held in 64 bits.
//
// Three launches: every row's largest logit and sum of exponentials, in pieces;
// per request the number of tokens that stand and, where one fell, each piece's
// share of max(p - q, 0); per request the piece, and in it the token, that the
// border falls into.
#include <hip/hip_runtime.h>

#include "zs_drafts_internal.h"

namespace zs {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any multiple of the element's size (the hardware takes unaligned
// vector loads).
typedef u32x4 __attribute__((aligned(2))) u32x4_u2;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr double kInf = __builtin_inf();
constexpr float kInfF = __builtin_inff();

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ float get(const u32x4& v, int i) {
        return __uint_as_float((i & 1) ? (v[i >> 1] & 0xFFFF0000u) : (v[i >> 1] << 16));
    }
    static __device__ __forceinline__ float one(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
};
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ float get(const u32x4& v, int i) { return __uint_as_float(v[i]); }
    static __device__ __forceinline__ float one(float x) { return x; }
};

// What the temperature makes of a difference of logits.
struct Scale {
    double per_logit;  // log2(e) / temperature
    double lowest;     // the difference of a token 2^-1000 times as likely
    double inv_t;      // 1 / temperature
};

// 2^f for |f| <= 1/2 is the polynomial that agrees with it at the 11 Chebyshev
// points cos((2k + 1) pi / 22) / 2; it is off by 3e-16, and 1 at 0. The
// coefficients are kept in scalar registers, from which a three-operand
// multiply-add takes them (as literals each would be copied into vector registers
// first, two moves an operation).
struct Exp2 {
    double c[11] = {1.0,
                    0.69314718055995,
                    0.24022650695910097,
                    0.05550410866444772,
                    0.009618129107606888,
                    0.0013333558230164974,
                    0.0001540353044173605,
                    1.5252657260200837e-05,
                    1.321544258792169e-06,
                    1.0208690299958306e-07,
                    7.072585949269223e-09};
    double whole = 6755399441055744.0;  // 1.5 * 2^52
    double per_logit, lowest;
    __device__ __forceinline__ Exp2(const Scale& scale) : per_logit(scale.per_logit), lowest(scale.lowest) {
#pragma unroll
        for (int i = 1; i < 10; ++i) asm("" : "+s"(c[i]));
        // an instruction takes one scalar: these are operands next to another one
        asm("" : "+v"(c[10]), "+v"(whole));
    }
    // The likelihood of a logit that is d <= 0 above another, to the last digits;
    // at least 2^-1001, which no sum that has the largest logit's 1 in it sees. The
    // whole number comes out of the last bits of a sum with 1.5 * 2^52 (the
    // conversions and the scaling of doubles that this replaces run at a quarter of
    // a multiply-add's rate).
    __device__ __forceinline__ double operator()(double d) const {
        d = fmax(d, lowest);
        const double sum = fma(d, per_logit, whole), f = fma(d, per_logit, whole - sum);
        double p = c[10];
#pragma unroll
        for (int i = 9; i >= 0; --i) p = fma(p, f, c[i]);
        u32x2 bits = __builtin_bit_cast(u32x2, p);
        const u32x2 n = __builtin_bit_cast(u32x2, sum);
        bits[1] += n[0] << 20;
        return __builtin_bit_cast(double, bits);
    }
    // The same, but 0 below 2^-1000: quotients by sums of up to 2^30 such values
    // are not 0 where the value is not.
    __device__ __forceinline__ double cut(double d) const {
        const double v = (*this)(d);
        return d >= lowest ? v : 0.0;
    }
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}
// NaN if there is one.
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = __builtin_elementwise_maximum(v, __shfl_xor(v, d, 64));
    return v;
}

// Drafted tokens of request b; < 0: skipped.
__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int64_t b) {
    if (!a.lens) return a.drafts;
    const int n = a.lens[b];
    return n < a.drafts ? n : a.drafts;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const Rows& m, int64_t row) {
    return static_cast<const T*>(m.p) + row * m.stride;
}

// ------------------------------------------------------------------ 1: rows

// Where element e of a lane's part of a piece lies.
template <typename T>
__device__ __forceinline__ int place_of(int e) {
    constexpr int kN = Vec<T>::kN;
    return (e / kN * 64 + (int)(threadIdx.x & 63)) * kN + e % kN;
}

// kCount elements of a lane's part of a piece of `left` logits, from element
// `first` on; -infinity behind the end.
template <typename T, int kPiece, int kCount>
__device__ __forceinline__ void load_piece(const T* z, int left, int first, float (&x)[kCount]) {
    constexpr int kN = Vec<T>::kN;
    static_assert(kCount % kN == 0, "whole vectors");
    const int i0 = place_of<T>(0) + first * 64;
    if (left == kPiece) {
        const u32x4_u2* at = reinterpret_cast<const u32x4_u2*>(z + i0);
#pragma unroll
        for (int v = 0; v < kCount / kN; ++v) {
            const u32x4 w = at[v * 64];
#pragma unroll
            for (int e = 0; e < kN; ++e) x[v * kN + e] = Vec<T>::get(w, e);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < kCount; ++e) {
        const int i = i0 + place_of<T>(e) - place_of<T>(0);
        x[e] = i < left ? Vec<T>::one(z[i]) : -kInfF;
    }
}

template <int kPiece>
__device__ __forceinline__ int piece_len(int64_t vocab, int64_t piece) {
    const int64_t left = vocab - piece * kPiece;
    return (int)(left < kPiece ? left : kPiece);
}

// The workgroups of a row, each of which has kWaves pieces.
__host__ __device__ inline int64_t groups_of(int64_t pieces) { return (pieces + kWaves - 1) / kWaves; }

// Workgroup (group, row): a wave holds its piece in registers between the
// maximum and the sum. An element takes about 20 vector instructions, most of them
// of 64 bits at the rate of 32-bit ones, whatever its type. 576 rows of 151936 fp32
// (350 MB, 55 us at a copy's rate) take 62 to 81 us, of whose cycles the vector
// unit is busy 67%: memory and arithmetic are both near their limit (nontemporal
// loads make no difference). Of bf16, half the bytes, a call takes as long.
template <typename T, int kPiece>
__global__ __launch_bounds__(kThreads) void k_verify_rows(VerifyArgs a, Scale scale, int64_t row0,
                                                          int64_t pieces, VerifyPart* __restrict__ parts) {
    const uint32_t groups = (uint32_t)groups_of(pieces);
    const int64_t row = row0 + blockIdx.x / groups;
    const int64_t piece = (int64_t)(blockIdx.x % groups) * kWaves + (threadIdx.x >> 6);
    const int64_t targets = a.requests * (a.drafts + 1);
    const bool target = row < targets;
    const int64_t in = target ? row : row - targets;
    const int per = a.drafts + (target ? 1 : 0);
    const int64_t b = in / per;
    if (piece >= pieces) return;
    if ((int)(in - b * per) >= drafts_of(a, b) + (target ? 1 : 0)) return;  // behind the request's rows
    constexpr int kPerThread = kPiece / 64;
    float x[kPerThread];
    load_piece<T, kPiece>(row_of<T>(target ? a.target : a.draft, in) + piece * kPiece,
                          piece_len<kPiece>(a.vocab, piece), 0, x);
    float top = -kInfF;  // a NaN stays
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) top = __builtin_elementwise_maximum(top, x[e]);
    top = wave_max(top);
    const bool bad = !(top < kInfF);
    const double top64 = bad ? __builtin_nan("") : (double)top;
    double sum = 0.0;
    if (!bad && top > -kInfF) {  // the same in the whole wave
        const Exp2 exp2(scale);
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) sum += exp2((double)x[e] - top64);
        sum = wave_sum(sum);
    }
    if ((threadIdx.x & 63) == 0) parts[row * pieces + piece] = VerifyPart{top64, sum};
}

// A row's largest logit and sum, from its pieces', by kJoin lanes that take kHeld
// pieces at a time; bad rows have a NaN for the largest.
constexpr int kJoin = 16, kHeld = 8;
__device__ __forceinline__ VerifyPart join(const Exp2& exp2, const VerifyPart* parts, int64_t pieces, bool any) {
    const int lane = threadIdx.x % kJoin;
    double top = -kInf, sum = 0.0;
    int bad = 0;
    for (int64_t c0 = 0; any && c0 < pieces; c0 += kJoin * kHeld) {
        VerifyPart held[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int64_t c = c0 + i * kJoin + lane;
            held[i] = parts[c < pieces ? c : c0];
            if (c >= pieces) held[i] = VerifyPart{-kInf, 0.0};
        }
        double most = top;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            bad |= !(held[i].top < kInf);
            most = fmax(most, held[i].top);
        }
        if (!bad && most > -kInf) {
            sum *= exp2(top - most);  // 0 where top is still -infinity
#pragma unroll
            for (int i = 0; i < kHeld; ++i) sum += held[i].sum * exp2(held[i].top - most);
        }
        top = most;
    }
    double all = top;
#pragma unroll
    for (int d = kJoin / 2; d; d >>= 1) {
        all = fmax(all, __shfl_xor(all, d, 64));
        bad |= __shfl_xor(bad, d, 64);
    }
    sum = !bad && all > -kInf ? sum * exp2(top - all) : 0.0;
#pragma unroll
    for (int d = kJoin / 2; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
    return VerifyPart{bad ? __builtin_nan("") : all, sum};
}

// ------------------------------------------------------------------ 2: what stands, and the rest

// The probabilities of a row's logits.
struct Softmax {
    double top, inv_sum;
    __device__ __forceinline__ Softmax(const VerifyPart& r) {
        top = r.top > -kInf ? r.top : 0.0;  // a row of -infinity alone: every probability is 0
        inv_sum = r.sum > 0.0 ? 1.0 / r.sum : 0.0;
    }
    __device__ __forceinline__ double operator()(const Exp2& exp2, float z) const {
        return exp2.cut((double)z - top) * inv_sum;
    }
};

// Workgroup (group, request). Every one of a request finds out by itself how
// many tokens stand; the first writes it down. 64 requests of 151936 fp32: 24 us,
// of which 3 pass before the first logit is asked for (which row it is follows
// from the sums) and 12 are two rows' bytes; one request of 32000 bf16: 7. What the
// workgroups of a request repeat grows with the square of the vocabulary: calls of
// one request with 4 drafts take 15 us at 2^17 logits, 45 at 2^20, 450 at 2^24.
template <typename T, int kPiece>
__global__ __launch_bounds__(kThreads) void k_verify_rest(VerifyArgs a, Scale scale,
                                                          int64_t request0, int64_t pieces,
                                                          const VerifyPart* __restrict__ parts,
                                                          double* __restrict__ totals,
                                                          VerifyPick* __restrict__ picks) {
    __shared__ VerifyPart stats[2 * ZS_VERIFY_MAX_DRAFTS + 1];  // target rows, then draft rows
    __shared__ int first_fallen;
    const uint32_t groups = (uint32_t)groups_of(pieces);
    const int64_t b = request0 + blockIdx.x / groups, group = blockIdx.x % groups;
    const int k = a.drafts, n = drafts_of(a, b), tid = threadIdx.x;
    int32_t* out = a.out + b * (k + 1);
    float* lps = a.logprobs ? a.logprobs + b * (k + 1) : nullptr;
    if (n < 0) {
        if (group == 0) {
            for (int i = tid; i <= k; i += kThreads) {
                out[i] = -1;
                if (lps) lps[i] = 0.0f;
            }
            if (tid == 0) {
                a.accepted[b] = 0;
                picks[b].kind = kDrawNothing;
            }
        }
        return;
    }
    // thread i: token i with its logits
    int x = -1;
    bool inside = false;
    float zp = 0.0f, zq = 0.0f, u = 0.0f;
    if (tid < n) {
        x = a.tokens[b * k + tid];
        u = a.uniforms[b * (k + 1) + tid];
        inside = x >= 0 && x < a.vocab;
        if (inside) {
            zp = Vec<T>::one(row_of<T>(a.target, b * (k + 1) + tid)[x]);
            if (a.draft.p) zq = Vec<T>::one(row_of<T>(a.draft, b * k + tid)[x]);
        }
    }
    const Exp2 exp2(scale);
    const int64_t targets = a.requests * (k + 1);
    const int rows = n + 1 + (a.draft.p ? n : 0);
    for (int i0 = 0; i0 < rows; i0 += kThreads / kJoin) {
        const int i = i0 + tid / kJoin;
        const int64_t row = i <= n ? b * (k + 1) + i : targets + b * k + (i - n - 1);
        const VerifyPart s = join(exp2, parts + row * pieces, pieces, i < rows);
        if (i < rows && tid % kJoin == 0) stats[i] = s;
    }
    if (tid == 0) first_fallen = n;
    __syncthreads();
    // whether it stands (rows that cannot be used let it fall)
    double lp = 0.0;
    if (tid < n) {
        const VerifyPart ps = stats[tid];
        bool stands = inside && ps.top > -kInf;
        double q = 1.0;
        if (a.draft.p) {
            const VerifyPart qs = stats[n + 1 + tid];
            stands = stands && !(qs.top != qs.top);
            q = Softmax(qs)(exp2, zq);
        }
        stands = stands && (double)u * q < Softmax(ps)(exp2, zp);
        if (stands)
            lp = ((double)zp - ps.top) * scale.inv_t - log(ps.sum);
        else
            atomicMin(&first_fallen, tid);  // shared memory; the least is the same in any order
    }
    __syncthreads();
    const int at = first_fallen;
    const VerifyPart ps = stats[at], qs = at < n && a.draft.p ? stats[n + 1 + at] : VerifyPart{0.0, 0.0};
    const bool dead = !(ps.top > -kInf) || qs.top != qs.top;
    const int kind = dead ? kDrawNothing : at < n ? kDrawRest : kDrawTarget;
    const int fallen = at < n ? a.tokens[b * k + at] : -1;
    if (group == 0) {
        if (tid < at) {
            out[tid] = x;
            if (lps) lps[tid] = (float)lp;
        }
        for (int i = at + tid; i <= k; i += kThreads) {
            out[i] = -1;  // the token at `at` is drawn by the next launch
            if (lps) lps[i] = i == at && dead ? __builtin_nanf("") : 0.0f;
        }
        if (tid == 0) {
            a.accepted[b] = at;
            picks[b] = VerifyPick{ps.top, ps.sum, qs.top, qs.sum, at, kind, fallen, 0};
        }
    }
    if (kind != kDrawRest) return;
    const int64_t piece = group * kWaves + (tid >> 6);
    if (piece >= pieces) return;
    const int left = piece_len<kPiece>(a.vocab, piece);
    const int64_t j0 = piece * kPiece;
    const T* zs = row_of<T>(a.target, b * (k + 1) + at) + j0;
    const Softmax p(ps);
    double sum = 0.0;
    // kTogether elements at a time, with the next ones' loads in flight
    constexpr int kPerThread = kPiece / 64, kTogether = 8;
    float z[kTogether], z1[kTogether];
    load_piece<T, kPiece>(zs, left, 0, z);
    if (a.draft.p) {
        const T* ys = row_of<T>(a.draft, b * k + at) + j0;
        float y[kTogether], y1[kTogether];
        load_piece<T, kPiece>(ys, left, 0, y);
        const Softmax q(qs);
#pragma unroll 1
        for (int e0 = 0; e0 < kPerThread; e0 += kTogether) {
            if (e0 + kTogether < kPerThread) {
                load_piece<T, kPiece>(zs, left, e0 + kTogether, z1);
                load_piece<T, kPiece>(ys, left, e0 + kTogether, y1);
            }
#pragma unroll
            for (int e = 0; e < kTogether; ++e) sum += fmax(p(exp2, z[e]) - q(exp2, y[e]), 0.0);
#pragma unroll
            for (int e = 0; e < kTogether; ++e) {
                z[e] = z1[e];
                y[e] = y1[e];
            }
        }
    } else {  // q is 1 at the token that fell
#pragma unroll 1
        for (int e0 = 0; e0 < kPerThread; e0 += kTogether) {
            if (e0 + kTogether < kPerThread) load_piece<T, kPiece>(zs, left, e0 + kTogether, z1);
#pragma unroll
            for (int e = 0; e < kTogether; ++e)
                sum += j0 + place_of<T>(e) + e0 * 64 == fallen ? 0.0 : p(exp2, z[e]);
#pragma unroll
            for (int e = 0; e < kTogether; ++e) z[e] = z1[e];
        }
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) totals[b * pieces + piece] = sum;
}

// ------------------------------------------------------------------ 3: the draw

constexpr int kDrawPer = 2;  // consecutive tokens of a thread

// The running sum over a workgroup's threads before each one, and the sum of all.
template <int kW>
__device__ __forceinline__ double before(double v, double& all, double (&shared)[kW]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double run = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(run, d, 64);
        if (lane >= d) run += o;
    }
    if (lane == 63) shared[wave] = run;
    __syncthreads();
    double base = 0.0;
    all = 0.0;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        if (i < wave) base += shared[i];
        all += shared[i];
    }
    return base + run - v;
}

// The first thread with a share whose running sum passes the border, else the
// last with a share; -1 if none has one.
struct Choice {
    int first, last;
};
template <int kW>
__device__ __forceinline__ int choose(double v, double run, double border, Choice (&shared)[kW]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t some = __ballot(v > 0.0), past = __ballot(v > 0.0 && !(run + v <= border));
    if (lane == 0)
        shared[wave] = Choice{past ? wave * 64 + __builtin_ctzll(past) : -1,
                              some ? wave * 64 + 63 - __builtin_clzll(some) : -1};
    __syncthreads();
    int first = -1, last = -1;
#pragma unroll
    for (int i = kW - 1; i >= 0; --i) {
        if (shared[i].first >= 0) first = shared[i].first;
        if (last < 0) last = shared[i].last;
    }
    return first >= 0 ? first : last;
}

// A workgroup a request: the piece, then two tokens a thread of it. A chain of
// dependent steps, 4 us for one request and 9 for 64 (eight tokens a thread of 256:
// 9 and 16).
template <typename T, int kPiece>
__global__ __launch_bounds__(kPiece / kDrawPer) void k_verify_draw(VerifyArgs a, Scale scale, int64_t pieces,
                                                                   const VerifyPart* __restrict__ parts,
                                                                   const double* __restrict__ totals,
                                                                   const VerifyPick* __restrict__ picks) {
    constexpr int kT = kPiece / kDrawPer, kW = kT / 64;
    __shared__ double scans[3][kW];
    __shared__ Choice choices[2][kW];
    __shared__ int64_t chosen_piece;
    __shared__ double chosen_before;
    const int64_t b = blockIdx.x;
    const VerifyPick pick = picks[b];
    if (pick.kind == kDrawNothing) return;
    const Exp2 exp2(scale);
    const int k = a.drafts;
    const int64_t row = b * (k + 1) + pick.at;
    bool whole = pick.kind == kDrawTarget;  // drawn from p, not from max(p - q, 0)
    const double u = a.uniforms[b * (k + 1) + k], inv_sum = 1.0 / pick.p_sum;
    // the piece: each thread has a run of them
    const int64_t per = (pieces + kT - 1) / kT;
    const int64_t c0 = min(threadIdx.x * per, pieces), c1 = min(c0 + per, pieces);
    auto share = [&](int64_t c) {
        if (!whole) return totals[b * pieces + c];
        const VerifyPart s = parts[row * pieces + c];
        return s.sum > 0.0 ? s.sum * exp2.cut(s.top - pick.p_top) * inv_sum : 0.0;
    };
    double mine, all, run;
    for (int turn = 0;; ++turn) {
        mine = 0.0;
        for (int64_t c = c0; c < c1; ++c) mine += share(c);
        run = before(mine, all, scans[turn]);
        if (whole || all > 0.0) break;
        whole = true;  // p nowhere exceeds q: drawn from p
    }
    const double border = u >= 1.0 ? kInf : u * all;  // from 1 on no rounding of a running sum passes it
    int owner = choose(mine, run, border, choices[0]);
    if ((int)threadIdx.x == owner) {
        int64_t found = c0;
        double found_before = run;
        for (int64_t c = c0; c < c1; ++c) {
            const double v = share(c);
            if (v > 0.0) {
                found = c;
                found_before = run;
                if (!(run + v <= border)) break;
            }
            run += v;
        }
        chosen_piece = found;
        chosen_before = found_before;
    }
    __syncthreads();
    // the token: each thread has a run of the piece
    const int64_t j0 = chosen_piece * kPiece + threadIdx.x * kDrawPer;
    const T* z = row_of<T>(a.target, row) + j0;
    const T* y = !whole && a.draft.p ? row_of<T>(a.draft, b * k + pick.at) + j0 : nullptr;
    float zv[kDrawPer], yv[kDrawPer];
#pragma unroll
    for (int e = 0; e < kDrawPer; ++e) {
        zv[e] = j0 + e < a.vocab ? Vec<T>::one(z[e]) : -kInfF;
        yv[e] = y && j0 + e < a.vocab ? Vec<T>::one(y[e]) : -kInfF;
    }
    const Softmax p(VerifyPart{pick.p_top, pick.p_sum}), q(VerifyPart{pick.q_top, pick.q_sum});
    double v[kDrawPer];
    mine = 0.0;
#pragma unroll
    for (int e = 0; e < kDrawPer; ++e) {
        v[e] = p(exp2, zv[e]);
        if (y)
            v[e] = fmax(v[e] - q(exp2, yv[e]), 0.0);
        else if (!whole && j0 + e == pick.token)
            v[e] = 0.0;
        mine += v[e];
    }
    run = chosen_before + before(mine, all, scans[2]);
    owner = choose(mine, run, border, choices[1]);
    if ((int)threadIdx.x == owner) {
        int64_t token = j0;
        float logit = zv[0];
        bool done = false;
#pragma unroll
        for (int e = 0; e < kDrawPer; ++e) {
            if (!done && v[e] > 0.0) {
                token = j0 + e;
                logit = zv[e];
                done = !(run + v[e] <= border);
            }
            run += v[e];
        }
        a.out[row] = (int32_t)token;
        if (a.logprobs) a.logprobs[row] = (float)(((double)logit - pick.p_top) * scale.inv_t - log(pick.p_sum));
    }
}

template <typename T, int kPiece>
int verify(const VerifyArgs& a, const VerifyLayout& l, double temperature, void* workspace, hipStream_t s) {
    char* ws = static_cast<char*>(workspace);
    VerifyPart* parts = reinterpret_cast<VerifyPart*>(ws);
    double* totals = reinterpret_cast<double*>(ws + l.totals_off);
    VerifyPick* picks = reinterpret_cast<VerifyPick*>(ws + l.picks_off);
    const double per_logit = 1.44269504088896340736 / temperature;
    const Scale scale{per_logit, -1000.0 / per_logit, 1.0 / temperature};
    // a launch covers at most 2^32 - 1 work-items
    const int64_t groups = groups_of(l.pieces), most = ((int64_t(1) << 32) - 1) / (groups * kThreads);
    const int64_t rows = a.draft.p ? l.rows : a.requests * (a.drafts + 1);
    for (int64_t lo = 0; lo < rows; lo += most) {
        const int64_t n = rows - lo < most ? rows - lo : most;
        k_verify_rows<T, kPiece><<<(unsigned)(n * groups), kThreads, 0, s>>>(a, scale, lo, l.pieces, parts);
        if (hipError_t e = hipGetLastError()) return (int)e;
    }
    for (int64_t lo = 0; lo < a.requests; lo += most) {
        const int64_t n = a.requests - lo < most ? a.requests - lo : most;
        k_verify_rest<T, kPiece><<<(unsigned)(n * groups), kThreads, 0, s>>>(a, scale, lo, l.pieces, parts, totals,
                                                                             picks);
        if (hipError_t e = hipGetLastError()) return (int)e;
    }
    k_verify_draw<T, kPiece><<<(unsigned)a.requests, kPiece / kDrawPer, 0, s>>>(a, scale, l.pieces, parts, totals,
                                                                                picks);
    return (int)hipGetLastError();
}

template <typename T>
int verify(const VerifyArgs& a, double temperature, void* workspace, hipStream_t s) {
    const VerifyLayout l = verify_layout(a.requests, a.drafts, a.vocab);
    return l.piece == kVerifyPiece ? verify<T, kVerifyPiece>(a, l, temperature, workspace, s)
                                   : verify<T, kVerifySmallPiece>(a, l, temperature, workspace, s);
}

}  // namespace

int launch_verify(const VerifyArgs& a, int dtype, double temperature, void* workspace, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == ZS_DTYPE_BF16 ? verify<uint16_t>(a, temperature, workspace, s)
                                  : verify<float>(a, temperature, workspace, s);
}

}  // namespace zs
