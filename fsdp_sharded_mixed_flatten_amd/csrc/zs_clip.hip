// Clipping of the multi-tensor step for CDNA4 (gfx950): the squared norm of the
// bf16 gradient over all bound pieces, and AdamW from the clipped gradient.
//
// Both are HBM streams over the chunks of the binding's table: 2 bytes an
// element for the norm, 28 to 32 for the step.
#include <hip/hip_runtime.h>

#include "zs_clip_internal.h"
#include "zs_device.h"

namespace zs {
namespace {

// ------------------------------------------------------------------ the norm

constexpr int kNormThreads = 256;
constexpr int kLanesPerChunk = kChunkElems / 8;  // 16-byte loads
constexpr int kRowChunks = kNormThreads / kLanesPerChunk;
constexpr int kNormRows = (int)kNormChunks / kRowChunks;
static_assert(kNormThreads % kLanesPerChunk == 0 && kNormChunks % kRowChunks == 0, "rows of whole chunks");

__device__ __forceinline__ double squares(const u32x4& v, double s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double a = (double)lo_bf16(v[i]), b = (double)hi_bf16(v[i]);
        s = fma(a, a, s);
        s = fma(b, b, s);
    }
    return s;
}

// Sum and flag of a workgroup of WAVES waves, in thread 0.
template <int WAVES>
__device__ __forceinline__ void group_sum(double& s, bool& bad) {
    __shared__ double sums[WAVES];
    __shared__ int bads[WAVES];
    s = wave_sum(s);
    const bool any = __ballot(bad) != 0;
    if ((threadIdx.x & 63) == 0) {
        sums[threadIdx.x >> 6] = s;
        bads[threadIdx.x >> 6] = any;
    }
    __syncthreads();
    s = 0.0;
    bad = false;
    for (int i = 0; i < WAVES; ++i) {
        s += sums[i];
        bad |= bads[i] != 0;
    }
}

// Workgroup g adds up chunks [g * kNormChunks, (g + 1) * kNormChunks). A square
// of a bf16 is finite in double, and so is any sum of them: a sum that is not
// comes from an element that is not. Bound by memory: a range inside one piece is
// streamed (842M elements 252 us, 6.7 TB/s); ranges of several pieces look theirs
// up first, all rows of the workgroup at once (434 pieces, 48M elements 19 us, 5.1
// TB/s). With a lookup a chunk before its load the calls took 1233 and 78 us.
__global__ __launch_bounds__(kNormThreads) void k_multi_norm(const MultiHeader* __restrict__ hdr, MultiOffsets moff,
                                                             int64_t unsummed, int64_t n_chunks,
                                                             double* __restrict__ part, int32_t* __restrict__ flags) {
    const char* ws = reinterpret_cast<const char*>(hdr);
    const int32_t* cpiece = reinterpret_cast<const int32_t*>(ws + moff.chunks);
    const PieceDev* pieces = reinterpret_cast<const PieceDev*>(ws + moff.pieces);
    const uint8_t* skip = unsummed ? reinterpret_cast<const uint8_t*>(ws + unsummed) : nullptr;
    double s = 0.0;
    bool bad = false;
    if (hdr->magic == kMultiMagic) {  // else not a bound table: nothing of it is followed
        const int64_t c0 = (int64_t)blockIdx.x * kNormChunks;
        const int64_t c1 = c0 + kNormChunks < n_chunks ? c0 + kNormChunks : n_chunks;
        const int32_t first = cpiece[c0], last = cpiece[c1 - 1];
        u32x4 v[kNormRows];
        if (first == last) {  // chunks follow their pieces' order: the whole range is of one
            const PieceDev pc = pieces[first];
            const int64_t at = (c0 - pc.first_chunk) * kChunkElems, end = (c1 - pc.first_chunk) * kChunkElems;
            const char* g = static_cast<const char*>(pc.grad) + 2 * at;
            const int n = (int)((end < pc.len ? end : pc.len) - at) / 8;  // lengths are multiples of 8
            if (n == kNormRows * kNormThreads) {
#pragma unroll
                for (int r = 0; r < kNormRows; ++r)
                    v[r] = ld_nt(reinterpret_cast<const u32x4*>(g) + r * kNormThreads + threadIdx.x);
            } else {
#pragma unroll
                for (int r = 0; r < kNormRows; ++r) {
                    const int i = r * kNormThreads + threadIdx.x;
                    v[r] = ld_nt(reinterpret_cast<const u32x4*>(g) + (i < n ? i : 0));
                    if (i >= n) v[r] = u32x4{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int r = 0; r < kNormRows; ++r) s = squares(v[r], s);
            bad = !__builtin_isfinite(s);
            if (skip && skip[first]) s = 0.0;
        } else {
            // every row's lookups, then every row's load, without a branch
            // between: a lane past its chunk's end reads the chunk's first vector
            int32_t chunk[kNormRows], piece[kNormRows];
            bool ok[kNormRows], counts[kNormRows];
            const u32x4* from[kNormRows];
            const int off = (threadIdx.x % kLanesPerChunk) * 8;
#pragma unroll
            for (int r = 0; r < kNormRows; ++r) {
                const int64_t c = c0 + r * kRowChunks + threadIdx.x / kLanesPerChunk;
                ok[r] = c < c1;
                chunk[r] = (int32_t)(ok[r] ? c : c0);
                piece[r] = ld_g(cpiece + chunk[r]);
            }
#pragma unroll
            for (int r = 0; r < kNormRows; ++r) {
                const PieceDev* pc = pieces + piece[r];
                const int64_t at = (int64_t)(chunk[r] - ld_g(&pc->first_chunk)) * kChunkElems;
                ok[r] = ok[r] && at + off < ld_g(&pc->len);
                counts[r] = !skip || !ld_g(skip + piece[r]);
                from[r] = reinterpret_cast<const u32x4*>(static_cast<const char*>(ld_g(&pc->grad)) +
                                                         2 * (at + (ok[r] ? off : 0)));
            }
#pragma unroll
            for (int r = 0; r < kNormRows; ++r) v[r] = ld_nt(from[r]);
#pragma unroll
            for (int r = 0; r < kNormRows; ++r) {
                const double t = ok[r] ? squares(v[r], 0.0) : 0.0;
                bad |= !__builtin_isfinite(t);
                if (counts[r]) s += t;
            }
        }
    }
    group_sum<kNormThreads / 64>(s, bad);
    if (threadIdx.x == 0) {
        part[blockIdx.x] = s;
        flags[blockIdx.x] = bad;
    }
}

// One workgroup: thread i adds up sums i, i + 1024, ... in order, eight loads at a
// time (51400 sums: 17 us one by one).
constexpr int kFinalThreads = 1024, kFinalHeld = 8;
__global__ __launch_bounds__(kFinalThreads) void k_multi_norm_final(const double* __restrict__ part,
                                                                    const int32_t* __restrict__ flags, int64_t n,
                                                                    double* __restrict__ sumsq_out,
                                                                    int32_t* __restrict__ nonfinite_out) {
    double s = 0.0;
    bool bad = false;
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += kFinalThreads * kFinalHeld) {
        double held[kFinalHeld];
        int32_t any[kFinalHeld];
#pragma unroll
        for (int k = 0; k < kFinalHeld; ++k) {
            const int64_t i = i0 + k * kFinalThreads;
            held[k] = part[i < n ? i : i0];
            any[k] = flags[i < n ? i : i0];
        }
#pragma unroll
        for (int k = 0; k < kFinalHeld; ++k) {
            if (i0 + k * kFinalThreads < n) s += held[k];
            bad |= any[k] != 0;
        }
    }
    group_sum<kFinalThreads / 64>(s, bad);
    if (threadIdx.x == 0) {
        *sumsq_out = s;
        *nonfinite_out = bad ? 1 : 0;
    }
}

// ------------------------------------------------------------------ the step

// One chunk (four elements a lane) a workgroup of one wave, as the unclipped
// multi-tensor step, with the same element arithmetic: without a factor the bits
// are the same. Bound by memory, 28 bytes an element: 193M elements 823 us,
// 6.6 TB/s.
constexpr unsigned kStepLds = 12u << 10;  // unused: fewer waves a compute unit keep fewer DRAM rows in play
__global__ __launch_bounds__(kBlockThreads) void k_multi_clip(CoefTable ct, const MultiHeader* __restrict__ hdr,
                                                              MultiOffsets off, const float* __restrict__ scale_p,
                                                              const int32_t* __restrict__ skip_p) {
    if (hdr->magic != kMultiMagic) return;
    if (skip_p && *skip_p) return;  // uniform: the whole grid skips the step
    const float scale = scale_p ? *scale_p : 1.0f;
    const char* ws = reinterpret_cast<const char*>(hdr);
    const int32_t piece = reinterpret_cast<const int32_t*>(ws + off.chunks)[blockIdx.x];
    const PieceDev pc = reinterpret_cast<const PieceDev*>(ws + off.pieces)[piece];
    const AdamCoef c = ct.c[pc.group];
    const int64_t start = (int64_t)((int32_t)blockIdx.x - pc.first_chunk) * kChunkElems;
    const int64_t u = (start >> 2) + threadIdx.x;
    if (u >= pc.len >> 2) return;
    const u32x2 g = ld_nt(reinterpret_cast<const u32x2*>(pc.grad) + u);
    f32x4 w = ld_nt(reinterpret_cast<const f32x4*>(pc.master) + u);
    f32x4 m = ld_nt(reinterpret_cast<const f32x4*>(pc.m) + u);
    f32x4 v = ld_nt(reinterpret_cast<const f32x4*>(pc.v) + u);
    const float ge[4] = {lo_bf16(g.x), hi_bf16(g.x), lo_bf16(g.y), hi_bf16(g.y)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float we = w[e], me = m[e], ve = v[e];
        adamw_elem(c, ge[e] * scale, we, me, ve);
        w[e] = we;
        m[e] = me;
        v[e] = ve;
    }
    st_lane(reinterpret_cast<f32x4*>(pc.master) + u, w);
    st_lane(reinterpret_cast<f32x4*>(pc.m) + u, m);
    st_lane(reinterpret_cast<f32x4*>(pc.v) + u, v);
    const u32x2 p = to_bf16x4(w);
    if (hdr->flags & kHasParam) st_lane(reinterpret_cast<u32x2*>(pc.param) + u, p);
    if (hdr->flags & kHasFull) st_lane(reinterpret_cast<u32x2*>(pc.full_own) + u, p);
}

}  // namespace

int launch_multi_norm(const void* workspace, const BoundTables& t, int64_t n_chunks, double* sumsq_out,
                      int32_t* nonfinite_out, void* stats_workspace, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t n = norm_groups(n_chunks);
    double* part = static_cast<double*>(stats_workspace);
    int32_t* flags = reinterpret_cast<int32_t*>(part + n);
    if (n > 0) {
        k_multi_norm<<<(unsigned)n, kNormThreads, 0, s>>>(static_cast<const MultiHeader*>(workspace), t.off,
                                                          t.unsummed, n_chunks, part, flags);
        if (hipError_t e = hipGetLastError()) return (int)e;
    }
    k_multi_norm_final<<<1, kFinalThreads, 0, s>>>(part, flags, n, sumsq_out, nonfinite_out);
    return (int)hipGetLastError();
}

int launch_multi_clip(const CoefTable& c, const void* workspace, const BoundTables& t, int64_t n_chunks,
                      const float* scale, const int32_t* skip, void* stream) {
    if (n_chunks == 0) return 0;
    k_multi_clip<<<(unsigned)n_chunks, kBlockThreads, kStepLds, static_cast<hipStream_t>(stream)>>>(
        c, static_cast<const MultiHeader*>(workspace), t.off, scale, skip);
    return (int)hipGetLastError();
}

}  // namespace zs
