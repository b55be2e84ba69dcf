// Drives the host part of the 4-bit format, the verification of drafted tokens
// and the clipped multi-tensor step (the kernel launchers are stand-ins that
// count their calls) through the largest extents that the calls accept, random
// arguments and concurrent callers, for address, undefined-behaviour and thread
// sanitizer builds. No address given here is ever read. Prints "more driver ok"
// and exits 0 when every check holds.
#include <zs_clip.h>
#include <zs_drafts.h>
#include <zs_mx4.h>

#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <string>
#include <thread>
#include <vector>

#include "../../fsdp_sharded_mixed_flatten_amd/csrc/zs_clip_internal.h"
#include "../../fsdp_sharded_mixed_flatten_amd/csrc/zs_drafts_internal.h"
#include "../../fsdp_sharded_mixed_flatten_amd/csrc/zs_mx4_internal.h"

#define CHECK(cond)                                                                                       \
    do {                                                                                                  \
        if (!(cond)) {                                                                                    \
            std::fprintf(stderr, "check failed at line %d: %s (%s)\n", __LINE__, #cond, zs_last_error()); \
            std::exit(1);                                                                                 \
        }                                                                                                 \
    } while (0)

namespace zs {
extern std::atomic<int> g_launches;
static thread_local BoundTables g_tables;

int launch_mx4_quantize(Rows, int, int64_t, int64_t, const Mx4&, void*) { return ++g_launches, 0; }
int launch_mx4_dequantize(const Mx4&, int64_t, int64_t, Rows, int, void*) { return ++g_launches, 0; }
int launch_mx4_matmul(const Mx4&, int64_t, const Mx4&, int64_t, int64_t, void*, int, int64_t, void*) {
    return ++g_launches, 0;
}
int launch_verify(const VerifyArgs&, int, double, void*, void*) { return ++g_launches, 0; }
int launch_multi_norm(const void*, const BoundTables& t, int64_t, double*, int32_t*, void*, void*) {
    return g_tables = t, ++g_launches, 0;
}
int launch_multi_clip(const CoefTable&, const void*, const BoundTables& t, int64_t, const float*, const int32_t*,
                      void*) {
    return g_tables = t, ++g_launches, 0;
}
// zs_lm_api.cpp is not part of this program; the file that is (zs_api.cpp) needs none of its launchers.
}  // namespace zs

namespace {

template <typename T = void>
T* at(uint64_t address) {
    return reinterpret_cast<T*>((uintptr_t)address);
}

void largest_extents() {
    const int64_t rows = int64_t(1) << 25, cols = int64_t(1) << 34;
    const uint64_t far = uint64_t(1) << 63;
    int before = zs::g_launches;
    // 2^25 rows of 2^34 elements: 2^59, an extent inside 2^60
    CHECK(zs_mx4_quantize(at(16), ZS_DTYPE_F32, rows, cols, cols, at(far), cols / 2, at(far + (far >> 1)), cols / 32,
                          nullptr) == ZS_OK);
    CHECK(zs_mx4_dequantize(at(far), cols / 2, at(far + (far >> 1)), cols / 32, rows, cols, at(16), ZS_DTYPE_F32, cols,
                            nullptr) == ZS_OK);
    CHECK(zs_mx4_quantize(at(16), ZS_DTYPE_F32, rows, cols, int64_t(1) << 36, at(far), cols / 2,
                          at(far + (far >> 1)), cols / 32, nullptr) == ZS_EINVAL);
    CHECK(zs_mx4_matmul(at(16), int64_t(1) << 28, at(uint64_t(1) << 54), int64_t(1) << 24, rows, at(uint64_t(1) << 55),
                        int64_t(1) << 28, at(uint64_t(1) << 56), int64_t(1) << 24, rows, int64_t(1) << 29, at(far),
                        ZS_DTYPE_F32, int64_t(1) << 34, nullptr) == ZS_OK);
    CHECK(zs::g_launches == before + 3);
    // the workspace of the largest call stays inside int64, and grows with every size
    const int64_t most = zs_verify_drafts_workspace_bytes(((int64_t(1) << 22) - 1) / 65, 64, int64_t(1) << 30);
    CHECK(most > 0 && most < int64_t(1) << 50);
    CHECK(zs_verify_drafts_workspace_bytes((int64_t(1) << 22) - 1, 0, int64_t(1) << 30) > 0);
    for (int64_t requests : {1, 3, 4096})
        for (int64_t v : {1, 512, 513, 2048, 2049, 151936}) {
            const zs::VerifyLayout l = zs::verify_layout(requests, 2, v);
            CHECK(l.rows == requests * 5 && (l.piece == zs::kVerifyPiece || l.piece == zs::kVerifySmallPiece));
            CHECK(l.pieces * l.piece >= v && (l.pieces - 1) * l.piece < v);
            CHECK(l.totals_off == l.rows * l.pieces * (int64_t)sizeof(zs::VerifyPart));
            CHECK(l.totals_off % 8 == 0 && l.picks_off % 8 == 0 && l.picks_off >= l.totals_off + requests * l.pieces * 8);
            CHECK(l.bytes == l.picks_off + requests * (int64_t)sizeof(zs::VerifyPick));
        }
    // a workspace serves the smaller calls
    for (int64_t requests = 1; requests < 30000; requests += 1 + requests / 5)
        for (int32_t drafts : {0, 1, 2, 5, 64})
            for (int64_t v = 1; v < 200000; v += 1 + v / 3) {
                const int64_t here = zs_verify_drafts_workspace_bytes(requests, drafts, v);
                CHECK(here <= zs_verify_drafts_workspace_bytes(requests + 1, drafts, v));
                CHECK(here <= zs_verify_drafts_workspace_bytes(requests, drafts + (drafts < 64), v));
                CHECK(here <= zs_verify_drafts_workspace_bytes(requests, drafts, v + 1));
                CHECK(here <= zs_verify_drafts_workspace_bytes(requests, drafts, v + v / 3));
            }
    before = zs::g_launches;
    const int64_t kRows = (int64_t(1) << 22) - 1, kStride = int64_t(1) << 38, kVocab = int64_t(1) << 30;
    const int64_t bytes = zs_verify_drafts_workspace_bytes(kRows, 0, kVocab);
    CHECK(zs_verify_drafts(at(16), ZS_DTYPE_F32, kRows, 0, kVocab, kStride, nullptr, 0, nullptr, nullptr,
                           at<float>(far), 1.0f, at<int32_t>(far + (1 << 26)), at<int32_t>(far + (2 << 26)), nullptr,
                           at(far + (uint64_t(1) << 40)), bytes, nullptr) == ZS_OK);
    CHECK(zs::g_launches == before + 1);
}

// Random arguments: whatever the call says, it launches exactly when it is ZS_OK and not empty.
void random_arguments(unsigned seed) {
    std::mt19937_64 rng(seed);
    auto pick = [&](std::initializer_list<int64_t> v) { return *(v.begin() + rng() % v.size()); };
    for (int i = 0; i < 20000; ++i) {
        const int64_t rows = pick({-1, 0, 1, 2, 77, int64_t(1) << 25, (int64_t(1) << 25) + 1});
        const int64_t cols = pick({-1, 0, 1, 31, 32, 33, 1531, int64_t(1) << 29, int64_t(1) << 34, INT64_MAX});
        const int64_t n = cols >= 0 && cols < INT64_MAX - 32 ? (cols + 31) / 32 : 1;
        const int64_t cs = pick({16 * n, 16 * n + 16, 16 * n - 16, 16 * n + 8, INT64_MIN, INT64_MAX});
        const int64_t ss = pick({n, n + 1, n - 1, 0, INT64_MAX});
        const int64_t xs = pick({cols, cols < INT64_MAX ? cols + 1 : cols, 0, -5, int64_t(1) << 38, INT64_MAX});
        auto a = [&]() { return at((rng() % 4 == 0) ? 0 : ((rng() % 8 + 1) << 60) + (rng() % 4 ? 0 : rng() % 64)); };
        const int32_t dtype = (int32_t)pick({0, 1, 2});
        const int before = zs::g_launches;
        zs_status st;
        switch (rng() % 3) {
            case 0: st = zs_mx4_quantize(a(), dtype, rows, cols, xs, a(), cs, a(), ss, nullptr); break;
            case 1: st = zs_mx4_dequantize(a(), cs, a(), ss, rows, cols, a(), dtype, xs, nullptr); break;
            default:
                st = zs_mx4_matmul(a(), cs, a(), ss, rows, a(), cs, a(), ss, pick({0, 1, 5, 1 << 25}), cols, a(),
                                   dtype, xs, nullptr);
        }
        CHECK(zs::g_launches - before <= (st == ZS_OK ? 1 : 0));
    }
    for (int i = 0; i < 20000; ++i) {
        const int64_t requests = pick({-1, 0, 1, 3, 1 << 16, (1 << 22) - 1, 1 << 22, INT64_MAX});
        const int32_t drafts = (int32_t)pick({-1, 0, 1, 4, 64, 65, INT32_MAX});
        const int64_t vocab = pick({-1, 0, 1, 100, 8193, 1 << 30, (1 << 30) + 1, INT64_MAX});
        const int64_t need = zs_verify_drafts_workspace_bytes(requests, drafts, vocab);
        auto a = [&]() { return at((rng() % 16 == 0) ? 0 : ((rng() % 15 + 1) << 60) + (rng() % 8 ? 0 : rng() % 64)); };
        const int before = zs::g_launches;
        const zs_status st = zs_verify_drafts(
            a(), (int32_t)pick({0, 1, 1, 3}), requests, drafts, vocab, pick({vocab, int64_t(1) << 38, 0, INT64_MAX}),
            a(), pick({vocab, int64_t(1) << 38, -1}), static_cast<int32_t*>(a()), static_cast<int32_t*>(a()),
            static_cast<float*>(a()), pick({1, 0, 2}), static_cast<int32_t*>(a()), static_cast<int32_t*>(a()),
            static_cast<float*>(a()), a(), pick({need, need - 1, INT64_MAX, 0}), nullptr);
        CHECK(need >= -1 && (need >= 0 || st != ZS_OK));
        CHECK(zs::g_launches - before <= (st == ZS_OK ? 1 : 0));
    }
}

// A binding's tables: marks of the pieces that are rank 0's to count.
void clip_tables() {
    const std::vector<int64_t> numels = {4096, 40, 100000, 8, 0};
    for (int32_t rank : {0, 3}) {
        for (int64_t below : {int64_t(0), int64_t(1000)}) {
            zs_plan_options o{ZS_LAYOUT_PER_TENSOR, 1, below, nullptr};
            zs_plan* p = nullptr;
            CHECK(zs_shard_plan_ex(numels.data(), (int32_t)numels.size(), 4, rank, &o, &p) == ZS_OK);
            const int64_t need = zs_multi_workspace_bytes(p, 0);
            std::vector<char> ws((size_t)need + 32);
            char* w = ws.data() + (16 - reinterpret_cast<uintptr_t>(ws.data()) % 16) % 16;
            std::vector<zs_piece_ptrs> pieces(numels.size());
            for (size_t i = 0; i < numels.size(); ++i)
                pieces[i] = zs_piece_ptrs{at((i + 1) << 32), at<float>((i + 10) << 32), at<float>((i + 20) << 32),
                                          at<float>((i + 30) << 32), nullptr, nullptr};
            CHECK(zs_multi_bind(p, pieces.data(), nullptr, 0, w, need - 1, nullptr) == ZS_ENOMEM);
            CHECK(zs_multi_bind(p, pieces.data(), nullptr, 0, w, need, nullptr) == ZS_OK);
            const int64_t sb = zs_grad_stats_multi_workspace_bytes(p);
            double* sum = at<double>(uint64_t(1) << 50);
            int32_t* flag = at<int32_t>((uint64_t(1) << 50) + 8);
            void* stats = at(uint64_t(1) << 51);
            CHECK(zs_grad_stats_multi(p, w, sum, flag, stats, sb, nullptr) == ZS_OK);
            const int64_t marks = zs::g_tables.unsummed;
            CHECK((marks != 0) == (rank != 0 && below != 0));
            if (marks) {
                CHECK(marks + (int64_t)numels.size() <= need);
                for (size_t i = 0; i < numels.size(); ++i) CHECK(w[marks + (int64_t)i] == (numels[i] < below));
            }
            CHECK(zs_grad_stats_multi(p, w, sum, flag, stats, sb - 1, nullptr) == ZS_ENOMEM);
            CHECK(zs_grad_stats_multi(p, w, at<double>(4), flag, stats, sb, nullptr) == ZS_EALIGN);
            CHECK(zs_grad_stats_multi(p, w, sum, at<int32_t>(uint64_t(1) << 50), stats, sb, nullptr) == ZS_EINVAL);
            CHECK(zs_grad_stats_multi(p, w, at<double>(uint64_t(1) << 51), flag, stats, sb, nullptr) == ZS_EINVAL);
            CHECK(zs_grad_stats_multi(p, w, sum, flag, nullptr, sb, nullptr) == ZS_EINVAL);
            CHECK(zs_grad_stats_multi(p, w, reinterpret_cast<double*>(w + need - 8), flag, stats, sb, nullptr) == ZS_EINVAL);
            CHECK(zs_grad_stats_multi(p, w, sum, reinterpret_cast<int32_t*>(w), stats, sb, nullptr) == ZS_EINVAL);
            CHECK(zs_grad_stats_multi(p, w, sum, flag, w, sb, nullptr) == ZS_EINVAL);
            zs_adamw_hparams hp{1e-4, 0.9, 0.95, 1e-8, 0.1, 1};
            const float* scale = at<float>(uint64_t(1) << 52);
            CHECK(zs_adamw_shard_step_multi_clip(p, &hp, 1, scale, nullptr, w, nullptr) == ZS_OK);
            CHECK(zs_adamw_shard_step_multi_clip(p, &hp, 0, scale, nullptr, w, nullptr) == ZS_EINVAL);
            CHECK(zs_adamw_shard_step_multi_clip(p, nullptr, 1, scale, nullptr, w, nullptr) == ZS_EINVAL);
            CHECK(zs_adamw_shard_step_multi_clip(p, &hp, 1, at<float>(2), nullptr, w, nullptr) == ZS_EALIGN);
            CHECK(zs_adamw_shard_step_multi_clip(p, &hp, 1, nullptr, at<int32_t>(2), w, nullptr) == ZS_EALIGN);
            for (auto& pc : pieces) pc.grad = nullptr;
            CHECK(zs_multi_bind(p, pieces.data(), nullptr, 0, w, need, nullptr) == ZS_OK);
            CHECK(zs_grad_stats_multi(p, w, sum, flag, stats, sb, nullptr) == ZS_EINVAL);
            CHECK(zs_multi_unbind(w, nullptr) == ZS_OK);
            CHECK(zs_adamw_shard_step_multi_clip(p, &hp, 1, scale, nullptr, w, nullptr) == ZS_EINVAL);
            zs_plan_destroy(p);
        }
    }
}

void everything(unsigned seed) {
    random_arguments(seed);
    clip_tables();
}

}  // namespace

int main(int argc, char** argv) {
    const std::string mode = argc > 1 ? argv[1] : "all";
    if (mode == "threads") {
        std::vector<std::thread> pool;
        for (unsigned t = 0; t < 4; ++t) pool.emplace_back([] { clip_tables(); });
        for (auto& t : pool) t.join();
    } else {
        largest_extents();
        everything(1);
    }
    std::printf("more driver ok (%s)\n", mode.c_str());
    return 0;
}
