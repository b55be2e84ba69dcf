// Verification of drafted tokens for CDNA4 (gfx950).
//
// A token is drawn where a running sum over the vocabulary passes a border that
// a random number sets. 151936 tokens of like probability have borders 7e-6
// apart, so that sums of fp32 exponentials would put one draw in a hundred on
// another side of a border than the definition does. Exponentials, their sums
// and the running sums are therefore held in 64 bits.
//
// Three launches: every row's largest logit and sum of exponentials, in chunks;
// per request the number of tokens that stand and, where one fell, each chunk's
// share of max(p - q, 0); per request the chunk, and in it the token, that the
// border falls into.
#include <hip/hip_runtime.h>

#include "zs_drafts_internal.h"

namespace zs {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any multiple of the element's size (the hardware takes unaligned
// vector loads).
typedef u32x4 __attribute__((aligned(2))) u32x4_u2;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPerThread = (int)kVerifyChunk / kThreads;
static_assert(kVerifyChunk % kThreads == 0, "a chunk is whole turns of a workgroup");
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

// 2^t for t <= 0, to a few units in the 15th digit: the series of 2^f around
// the nearest whole number, |f| <= 1/2, whose first term left out is below
// 7e-15. Below 2^-1000 it is 0, so that quotients of what is not 0 are not 0
// either.
__device__ __forceinline__ double exp2_neg(double t) {
    if (!(t >= -1000.0)) return 0.0;
    const double n = __builtin_rint(t), f = t - n;
    constexpr double kLn2 = 0.693147180559945309417;
    constexpr double c1 = kLn2, c2 = c1 * kLn2 / 2, c3 = c2 * kLn2 / 3, c4 = c3 * kLn2 / 4, c5 = c4 * kLn2 / 5,
                     c6 = c5 * kLn2 / 6, c7 = c6 * kLn2 / 7, c8 = c7 * kLn2 / 8, c9 = c8 * kLn2 / 9,
                     c10 = c9 * kLn2 / 10, c11 = c10 * kLn2 / 11;
    double p = c11;
    p = fma(p, f, c10);
    p = fma(p, f, c9);
    p = fma(p, f, c8);
    p = fma(p, f, c7);
    p = fma(p, f, c6);
    p = fma(p, f, c5);
    p = fma(p, f, c4);
    p = fma(p, f, c3);
    p = fma(p, f, c2);
    p = fma(p, f, c1);
    p = fma(p, f, 1.0);
    return ldexp(p, (int)n);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmax(v, __shfl_xor(v, d, 64));
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

// Workgroup (chunk, row) holds its chunk in registers between the maximum and
// the sum.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_verify_rows(VerifyArgs a, double per_logit, int64_t row0,
                                                          int64_t chunks, VerifyPart* __restrict__ parts) {
    constexpr int kN = Vec<T>::kN, kVecs = kPerThread / kN;
    __shared__ float tops[kWaves];
    __shared__ int bads[kWaves];
    __shared__ double sums[kWaves];
    const int64_t row = row0 + blockIdx.x / (uint32_t)chunks, chunk = blockIdx.x % (uint32_t)chunks;
    const int64_t targets = a.requests * (a.drafts + 1);
    const bool target = row < targets;
    const int64_t in = target ? row : row - targets;
    const int per = a.drafts + (target ? 1 : 0);
    const int64_t b = in / per;
    if ((int)(in - b * per) >= drafts_of(a, b) + (target ? 1 : 0)) return;  // behind the request's rows
    const T* z = row_of<T>(target ? a.target : a.draft, in) + chunk * kVerifyChunk;
    const int left = (int)(a.vocab - chunk * kVerifyChunk < kVerifyChunk ? a.vocab - chunk * kVerifyChunk
                                                                         : kVerifyChunk);
    float x[kPerThread];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int i = (v * kThreads + threadIdx.x) * kN;
        if (i + kN <= left) {
            const u32x4 w = *reinterpret_cast<const u32x4_u2*>(z + i);
#pragma unroll
            for (int e = 0; e < kN; ++e) x[v * kN + e] = Vec<T>::get(w, e);
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) x[v * kN + e] = i + e < left ? Vec<T>::one(z[i + e]) : -kInfF;
        }
    }
    float top = -kInfF;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
        top = fmaxf(top, x[e]);
        bad |= !(x[e] < kInfF);
    }
    top = wave_max(top);
    const int wave = threadIdx.x >> 6;
    const bool wave_bad = __ballot(bad) != 0;
    if ((threadIdx.x & 63) == 0) {
        tops[wave] = top;
        bads[wave] = wave_bad;
    }
    __syncthreads();
    bad = false;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        top = fmaxf(top, tops[i]);
        bad |= bads[i] != 0;
    }
    VerifyPart* part = parts + row * chunks + chunk;
    if (bad || top == -kInfF) {  // the same in the whole workgroup
        if (threadIdx.x == 0) *part = VerifyPart{bad ? __builtin_nan("") : -kInf, 0.0};
        return;
    }
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) sum += exp2_neg(((double)x[e] - (double)top) * per_logit);
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) sums[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = sums[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) sum += sums[i];
        *part = VerifyPart{(double)top, sum};
    }
}

// A row's largest logit and sum, from its chunks', by one wave.
__device__ __forceinline__ VerifyPart join(const VerifyPart* parts, int64_t chunks, double per_logit) {
    const int lane = threadIdx.x & 63;
    double top = -kInf;
    bool bad = false;
    for (int64_t c = lane; c < chunks; c += 64) {
        const double t = parts[c].top;
        bad |= !(t < kInf);
        top = fmax(top, t);
    }
    top = wave_max(top);
    if (__ballot(bad) != 0) return VerifyPart{__builtin_nan(""), 0.0};
    double sum = 0.0;
    if (top > -kInf)
        for (int64_t c = lane; c < chunks; c += 64) sum += parts[c].sum * exp2_neg((parts[c].top - top) * per_logit);
    return VerifyPart{top, wave_sum(sum)};
}

// ------------------------------------------------------------------ 2: what stands, and the rest

// Probability of logit z of a row.
__device__ __forceinline__ double prob(float z, const VerifyPart& r, double per_logit) {
    return r.sum > 0.0 ? exp2_neg(((double)z - r.top) * per_logit) / r.sum : 0.0;
}

// max(p - q, 0) of token j, or p alone.
template <typename T>
struct Rest {
    const T* p;
    const T* q;  // NULL: q is 1 at `token`, 0 elsewhere
    VerifyPart ps, qs;
    double per_logit;
    int kind;
    int64_t token;
    __device__ __forceinline__ double at(int64_t j) const {
        const double v = prob(Vec<T>::one(p[j]), ps, per_logit);
        if (kind == kDrawTarget) return v;
        if (!q) return j == token ? 0.0 : v;
        return fmax(v - prob(Vec<T>::one(q[j]), qs, per_logit), 0.0);
    }
};

// Workgroup (chunk, request). Every one of a request finds out by itself how
// many tokens stand; the first writes it down.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_verify_rest(VerifyArgs a, double per_logit, double inv_t,
                                                          int64_t request0, int64_t chunks,
                                                          const VerifyPart* __restrict__ parts,
                                                          double* __restrict__ totals,
                                                          VerifyPick* __restrict__ picks) {
    __shared__ VerifyPart stats[2 * ZS_VERIFY_MAX_DRAFTS + 1];  // target rows, then draft rows
    __shared__ int first_fallen;
    __shared__ double sums[kWaves];
    const int64_t b = request0 + blockIdx.x / (uint32_t)chunks, chunk = blockIdx.x % (uint32_t)chunks;
    const int k = a.drafts, n = drafts_of(a, b);
    int32_t* out = a.out + b * (k + 1);
    float* lps = a.logprobs ? a.logprobs + b * (k + 1) : nullptr;
    if (n < 0) {
        if (chunk == 0) {
            for (int i = threadIdx.x; i <= k; i += kThreads) {
                out[i] = -1;
                if (lps) lps[i] = 0.0f;
            }
            if (threadIdx.x == 0) {
                a.accepted[b] = 0;
                picks[b].kind = kDrawNothing;
            }
        }
        return;
    }
    const int64_t targets = a.requests * (k + 1);
    const int rows = n + 1 + (a.draft.p ? n : 0);
    for (int i = threadIdx.x >> 6; i < rows; i += kWaves) {
        const int64_t row = i <= n ? b * (k + 1) + i : targets + b * k + (i - n - 1);
        const VerifyPart s = join(parts + row * chunks, chunks, per_logit);
        if ((threadIdx.x & 63) == 0) stats[i] = s;
    }
    if (threadIdx.x == 0) first_fallen = n;
    __syncthreads();
    // thread i: whether token i stands (rows that cannot be used let it fall)
    double lp = 0.0;
    int x = -1;
    if ((int)threadIdx.x < n) {
        const int i = threadIdx.x;
        const VerifyPart ps = stats[i];
        x = a.tokens[b * k + i];
        const bool inside = x >= 0 && x < a.vocab;
        bool stands = inside && ps.top > -kInf;
        if (stands) {
            const float z = Vec<T>::one(row_of<T>(a.target, b * (k + 1) + i)[x]);
            double q = 1.0;
            if (a.draft.p) {
                const VerifyPart qs = stats[n + 1 + i];
                stands = !(qs.top != qs.top);
                q = prob(Vec<T>::one(row_of<T>(a.draft, b * k + i)[x]), qs, per_logit);
            }
            stands = stands && (double)a.uniforms[b * (k + 1) + i] * q < prob(z, ps, per_logit);
            lp = ((double)z - ps.top) * inv_t - log(ps.sum);
        }
        if (!stands) atomicMin(&first_fallen, i);  // shared memory; the least is the same in any order
    }
    __syncthreads();
    const int at = first_fallen;
    const VerifyPart ps = stats[at], qs = at < n && a.draft.p ? stats[n + 1 + at] : VerifyPart{0.0, 0.0};
    const bool dead = !(ps.top > -kInf) || qs.top != qs.top;
    const int kind = dead ? kDrawNothing : at < n ? kDrawRest : kDrawTarget;
    const int fallen = at < n ? a.tokens[b * k + at] : -1;
    if (chunk == 0) {
        if ((int)threadIdx.x < n && (int)threadIdx.x < at) {
            out[threadIdx.x] = x;
            if (lps) lps[threadIdx.x] = (float)lp;
        }
        for (int i = at + (int)threadIdx.x; i <= k; i += kThreads) {
            out[i] = -1;  // the token at `at` is drawn by the next launch
            if (lps) lps[i] = i == at && dead ? __builtin_nanf("") : 0.0f;
        }
        if (threadIdx.x == 0) {
            a.accepted[b] = at;
            picks[b] = VerifyPick{ps.top, ps.sum, qs.top, qs.sum, at, kind, fallen, 0};
        }
    }
    if (kind != kDrawRest) return;
    const Rest<T> rest{row_of<T>(a.target, b * (k + 1) + at), a.draft.p ? row_of<T>(a.draft, b * k + at) : nullptr,
                       ps, qs, per_logit, kind, fallen};
    const int64_t j0 = chunk * kVerifyChunk, j1 = j0 + kVerifyChunk < a.vocab ? j0 + kVerifyChunk : a.vocab;
    double sum = 0.0;
    for (int64_t j = j0 + threadIdx.x; j < j1; j += kThreads) sum += rest.at(j);
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = sums[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) sum += sums[i];
        totals[b * chunks + chunk] = sum;
    }
}

// ------------------------------------------------------------------ 3: the draw

// The running sum over a workgroup's threads before each one, and the sum of all.
__device__ __forceinline__ double before(double v, double& all, double (&shared)[kWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double run = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(run, d, 64);
        if (lane >= d) run += o;
    }
    __syncthreads();  // an earlier use of `shared` is over
    if (lane == 63) shared[wave] = run;
    __syncthreads();
    double base = 0.0;
    all = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
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
__device__ __forceinline__ int choose(double v, double run, double border, Choice& shared) {
    __syncthreads();
    if (threadIdx.x == 0) shared = Choice{kThreads, -1};
    __syncthreads();
    if (v > 0.0) {
        atomicMax(&shared.last, (int)threadIdx.x);
        if (!(run + v <= border)) atomicMin(&shared.first, (int)threadIdx.x);
    }
    __syncthreads();
    return shared.first < kThreads ? shared.first : shared.last;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_verify_draw(VerifyArgs a, double per_logit, double inv_t,
                                                          int64_t chunks, const VerifyPart* __restrict__ parts,
                                                          const double* __restrict__ totals,
                                                          const VerifyPick* __restrict__ picks) {
    __shared__ double scan[kWaves];
    __shared__ Choice choice;
    __shared__ int64_t chosen_chunk;
    __shared__ double chosen_before;
    const int64_t b = blockIdx.x;
    const VerifyPick pick = picks[b];
    if (pick.kind == kDrawNothing) return;
    const int k = a.drafts;
    const int64_t row = b * (k + 1) + pick.at;
    Rest<T> rest{row_of<T>(a.target, row), a.draft.p && pick.kind == kDrawRest ? row_of<T>(a.draft, b * k + pick.at)
                                                                             : nullptr,
                 VerifyPart{pick.p_top, pick.p_sum}, VerifyPart{pick.q_top, pick.q_sum}, per_logit, pick.kind,
                 pick.token};
    const double u = a.uniforms[b * (k + 1) + k];
    // the chunk: each thread has a run of them
    const int64_t per = (chunks + kThreads - 1) / kThreads;
    const int64_t c0 = threadIdx.x * per, c1 = c0 + per < chunks ? c0 + per : chunks;
    auto share = [&](int64_t c) {
        if (rest.kind == kDrawRest) return totals[b * chunks + c];
        const VerifyPart s = parts[row * chunks + c];
        return s.sum > 0.0 ? s.sum * exp2_neg((s.top - pick.p_top) * per_logit) / pick.p_sum : 0.0;
    };
    double mine = 0.0, all, run;
    for (int64_t c = c0; c < c1; ++c) mine += share(c);
    run = before(mine, all, scan);
    if (rest.kind == kDrawRest && !(all > 0.0)) {  // p nowhere exceeds q: drawn from p
        rest.kind = kDrawTarget;
        mine = 0.0;
        for (int64_t c = c0; c < c1; ++c) mine += share(c);
        run = before(mine, all, scan);
    }
    const double border = u * all;
    int owner = choose(mine, run, border, choice);
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
        chosen_chunk = found;
        chosen_before = found_before;
    }
    __syncthreads();
    // the token: each thread has a run of the chunk
    const int64_t j0 = chosen_chunk * kVerifyChunk + threadIdx.x * kPerThread;
    double v[kPerThread];
    mine = 0.0;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
        v[e] = j0 + e < a.vocab ? rest.at(j0 + e) : 0.0;
        mine += v[e];
    }
    run = chosen_before + before(mine, all, scan);
    owner = choose(mine, run, border, choice);
    if ((int)threadIdx.x == owner) {
        int64_t token = j0;
        bool done = false;
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
            if (!done && v[e] > 0.0) {
                token = j0 + e;
                done = !(run + v[e] <= border);
            }
            run += v[e];
        }
        a.out[row] = (int32_t)token;
        if (a.logprobs)
            a.logprobs[row] = (float)(((double)Vec<T>::one(rest.p[token]) - pick.p_top) * inv_t - log(pick.p_sum));
    }
}

template <typename T>
int verify(const VerifyArgs& a, double temperature, void* workspace, hipStream_t s) {
    const VerifyLayout l = verify_layout(a.requests, a.drafts, a.vocab);
    char* ws = static_cast<char*>(workspace);
    VerifyPart* parts = reinterpret_cast<VerifyPart*>(ws);
    double* totals = reinterpret_cast<double*>(ws + l.totals_off);
    VerifyPick* picks = reinterpret_cast<VerifyPick*>(ws + l.picks_off);
    const double inv_t = 1.0 / temperature, per_logit = 1.44269504088896340736 / temperature;
    // a launch covers at most 2^32 - 1 work-items
    const int64_t most = ((int64_t(1) << 32) - 1) / (l.chunks * kThreads);
    const int64_t rows = a.draft.p ? l.rows : a.requests * (a.drafts + 1);
    for (int64_t lo = 0; lo < rows; lo += most) {
        const int64_t n = rows - lo < most ? rows - lo : most;
        k_verify_rows<T><<<(unsigned)(n * l.chunks), kThreads, 0, s>>>(a, per_logit, lo, l.chunks, parts);
        if (hipError_t e = hipGetLastError()) return (int)e;
    }
    for (int64_t lo = 0; lo < a.requests; lo += most) {
        const int64_t n = a.requests - lo < most ? a.requests - lo : most;
        k_verify_rest<T><<<(unsigned)(n * l.chunks), kThreads, 0, s>>>(a, per_logit, inv_t, lo, l.chunks, parts,
                                                                       totals, picks);
        if (hipError_t e = hipGetLastError()) return (int)e;
    }
    k_verify_draw<T><<<(unsigned)a.requests, kThreads, 0, s>>>(a, per_logit, inv_t, l.chunks, parts, totals, picks);
    return (int)hipGetLastError();
}

}  // namespace

int launch_verify(const VerifyArgs& a, int dtype, double temperature, void* workspace, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == ZS_DTYPE_BF16 ? verify<uint16_t>(a, temperature, workspace, s)
                                  : verify<float>(a, temperature, workspace, s);
}

}  // namespace zs
