// Drives the host part of the language-model operators (zs_lm_api.cpp; the
// kernel launchers are stand-ins that count their calls) through the largest
// extents that the calls accept, every way in which two buffers can touch,
// random arguments and concurrent callers, for address, undefined-behaviour
// and thread sanitizer builds. No address given here is ever read. Prints
// "lm driver ok" and exits 0 when every check holds.
#include <zs_lm.h>

#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <string>
#include <thread>
#include <vector>

#include "../../fsdp_sharded_mixed_flatten_amd/csrc/zs_lm_internal.h"

#define CHECK(cond)                                                              \
    do {                                                                         \
        if (!(cond)) {                                                           \
            std::fprintf(stderr, "check failed at line %d: %s (%s)\n", __LINE__, #cond, zs_last_error()); \
            std::exit(1);                                                        \
        }                                                                        \
    } while (0)

namespace zs {
extern std::atomic<int> g_launches;

int launch_quant_matvec(const QuantWeight&, Rows, int, void*, int, int64_t, void*) { return ++g_launches, 0; }
int launch_logprobs(Rows, int, int64_t, int64_t, const int32_t*, double, const LogprobsOut&, void*) {
    return ++g_launches, 0;
}
int launch_logprobs_grad(Rows, int, int64_t, int64_t, double, const LogprobsGradIn&, void*, int64_t, void*) {
    return ++g_launches, 0;
}
int launch_distill(Rows, int, int64_t, int64_t, const Teacher&, double, float*, void*, int64_t, void*) {
    return ++g_launches, 0;
}
}  // namespace zs

namespace {

constexpr int64_t kRows = (int64_t(1) << 22) - 1, kStride = int64_t(1) << 38, kVocab = int64_t(1) << 30;

template <typename T = void>
T* at(uint64_t address) {
    return reinterpret_cast<T*>((uintptr_t)address);
}

struct PlanOf {
    zs_plan* p = nullptr;
    PlanOf(std::vector<int64_t> numels, int32_t world, int32_t align) {
        CHECK(zs_shard_plan(numels.data(), (int32_t)numels.size(), world, 0, align, ZS_LAYOUT_FLAT, &p) == ZS_OK);
    }
    ~PlanOf() { zs_plan_destroy(p); }
};

// Matrices of 2^62 bytes: every row and column, the widest stride, fp32.
void largest_extents() {
    const uint64_t z = 16, end = z + 4 * ((kRows - 1) * kStride + kVocab);
    const uint64_t g = end, small = uint64_t(1) << 63;
    auto* f = at<float>(small);
    auto* tokens = at<int32_t>(small - (uint64_t(1) << 40));
    const int before = zs::g_launches;
    CHECK(zs_token_logprobs(at(z), ZS_DTYPE_F32, kRows, kVocab, kStride, tokens, 1.0f, f, f + kRows, f + 2 * kRows,
                            ZS_LOGPROBS_MAX_TOP, at<int32_t>(small + (uint64_t(1) << 40)),
                            at<float>(small + (uint64_t(1) << 41)), nullptr) == ZS_OK);
    CHECK(zs_token_logprobs(at(z), ZS_DTYPE_F32, kRows, kVocab, kStride, tokens, 1.0f, at<float>(end - 4), nullptr,
                            nullptr, 0, nullptr, nullptr, nullptr) == ZS_EINVAL);
    CHECK(zs_token_logprobs_backward(at(z), ZS_DTYPE_F32, kRows, kVocab, kStride, tokens, 1.0f, f, f, f, f, at(g),
                                     kStride, nullptr) == ZS_OK);
    CHECK(zs_token_logprobs_backward(at(z), ZS_DTYPE_F32, kRows, kVocab, kStride, tokens, 1.0f, f, f, f, f, at(z),
                                     kStride, nullptr) == ZS_OK);
    CHECK(zs_token_logprobs_backward(at(z), ZS_DTYPE_F32, kRows, kVocab, kStride, tokens, 1.0f, f, f, f, f,
                                     at(end - 4), kStride, nullptr) == ZS_EINVAL);
    CHECK(zs_distill_topk(at(z), ZS_DTYPE_F32, kRows, kVocab, kStride, tokens, f, ZS_DISTILL_MAX_K, 1.0f, nullptr,
                          at<float>(small + (uint64_t(1) << 41)), at(g), kStride, nullptr) == ZS_OK);
    CHECK(zs::g_launches == before + 4);
}

// The largest matrix, in the last place of the largest buffer a plan takes
// (2^60 elements, of more ranks than anyone has).
void largest_products() {
    const int64_t out = int64_t(1) << 25, in = int64_t(1) << 29;
    const PlanOf plan({(int64_t(1) << 60) - out * in, out * in}, 1 << 27, 1);
    CHECK(zs_plan_padded_numel(plan.p) == int64_t(1) << 60 && zs_plan_shard_numel(plan.p) == int64_t(1) << 33);
    const uint64_t x = 16, y = uint64_t(1) << 48, codes = uint64_t(1) << 60, scales = uint64_t(1) << 62;
    const int before = zs::g_launches;
    for (int bits : {4, 8}) {
        CHECK(zs_quant_matvec(plan.p, 1, out, in, bits, 8, at(codes), at<float>(scales), at(x), kStride, 64, at(y),
                              ZS_DTYPE_F32, kStride, nullptr) == ZS_OK);
        // y in the codes' last bytes
        const uint64_t last = codes + (uint64_t(1) << 60) * (unsigned)bits / 8 - 16;
        CHECK(zs_quant_matvec(plan.p, 1, out, in, bits, 8, at(codes), at<float>(scales), at(x), kStride, 64, at(last),
                              ZS_DTYPE_F32, kStride, nullptr) == ZS_EINVAL);
    }
    CHECK(zs::g_launches == before + 2);
}

// Buffers that share an address range and no element are accepted (columns side
// by side in one matrix, an array between two rows), buffers that share one
// byte are not. Rows of 100 elements, 4 of them.
void neighbours() {
    const uint64_t a = uint64_t(1) << 40, far = uint64_t(1) << 50;
    auto* tok = at<int32_t>(far);
    auto* f = at<float>(far + (1 << 20));
    auto grad = [&](uint64_t z, int64_t zs, uint64_t g, int64_t gs, int dtype, int64_t rows = 4) {
        return zs_token_logprobs_backward(at(z), dtype, rows, 100, zs, tok, 1.0f, f, nullptr, f, nullptr, at(g), gs,
                                          nullptr);
    };
    for (int dtype : {ZS_DTYPE_BF16, ZS_DTYPE_F32}) {
        const uint64_t e = dtype == ZS_DTYPE_BF16 ? 2 : 4;
        CHECK(grad(a, 200, a + 100 * e, 200, dtype) == ZS_OK);          // right half
        CHECK(grad(a + 100 * e, 200, a, 200, dtype) == ZS_OK);          // left half
        CHECK(grad(a, 203, a + 103 * e, 203, dtype) == ZS_OK);
        CHECK(grad(a, 200, a + 99 * e, 200, dtype) == ZS_EINVAL);       // an element too far left
        CHECK(grad(a, 200, a + 101 * e, 200, dtype) == ZS_EINVAL);      // an element too far right
        CHECK(grad(a, 200, a + (3 * 200 + 100) * e, 200, dtype) == ZS_OK);
        CHECK(grad(a, 200, a + (2 * 200 + 100) * e, 200, dtype) == ZS_OK);
        CHECK(grad(a, 200, a + 2 * 200 * e, 200, dtype) == ZS_EINVAL);  // two rows further on
        CHECK(grad(a, 200, a + 100 * e, 201, dtype) == ZS_EINVAL);      // halves that drift into each other
        CHECK(grad(a, 300, a + 100 * e, 500, dtype, 1) == ZS_OK);       // one row: its stride says nothing
        CHECK(grad(a, 300, a + 99 * e, 500, dtype, 1) == ZS_EINVAL);
        // distillation: loss and entries between the rows of a gradient
        auto distill = [&](uint64_t loss, uint64_t ids) {
            return zs_distill_topk(at(a + 100 * e), dtype, 4, 100, 300, at<int32_t>(ids), f, 2, 1.0f, nullptr,
                                   at<float>(loss), at(a), 300, nullptr);
        };
        CHECK(distill(a + 200 * e, a + (300 + 200) * e) == ZS_OK);
        CHECK(distill(a + 300 * e - 16, far) == ZS_OK);
        CHECK(distill(a + 300 * e - 12, far) == ZS_EINVAL);
        CHECK(distill(a + 200 * e - 4, far) == ZS_EINVAL);
        CHECK(distill(far + (1 << 24), a + 300 * e - 32) == ZS_OK);
        CHECK(distill(far + (1 << 24), a + 300 * e - 28) == ZS_EINVAL);
        CHECK(distill(a + 200 * e, a + 200 * e + 12) == ZS_EINVAL);  // and between themselves
    }
    // log-probabilities: tokens and outputs behind the logits of each row
    auto scored = [&](uint64_t lp, uint64_t st) {
        return zs_token_logprobs(at(a), ZS_DTYPE_F32, 4, 100, 164, tok, 1.0f, at<float>(lp), nullptr, at<float>(st), 0,
                                 nullptr, nullptr, nullptr);
    };
    CHECK(scored(a + 400, a + 416) == ZS_OK);
    CHECK(scored(a + 400, a + 412) == ZS_EINVAL);
    CHECK(scored(a + 396, far + 4096) == ZS_EINVAL);
    CHECK(scored(a + 656 - 16, a + 656 - 48) == ZS_OK);
    CHECK(scored(a + 656 - 12, far + 4096) == ZS_EINVAL);
    // products: x and y columns of one matrix, in bf16 and with fp32 results
    const PlanOf plan({24 * 48}, 2, 8);
    auto product = [&](uint64_t x, int64_t xs, uint64_t y, int64_t ys, int dtype) {
        return zs_quant_matvec(plan.p, 0, 24, 48, 4, 8, at(far), at<float>(far + (1 << 20)), at(x), xs, 5, at(y), dtype,
                               ys, nullptr);
    };
    CHECK(product(a, 72, a + 96, 72, ZS_DTYPE_BF16) == ZS_OK);
    CHECK(product(a + 48, 72, a, 72, ZS_DTYPE_BF16) == ZS_OK);
    CHECK(product(a, 72, a + 94, 72, ZS_DTYPE_BF16) == ZS_EINVAL);
    CHECK(product(a, 96, a + 96, 48, ZS_DTYPE_F32) == ZS_OK);
    CHECK(product(a, 96, a + 100, 48, ZS_DTYPE_F32) == ZS_EINVAL);
    CHECK(product(a, 96, a + 96, 96, ZS_DTYPE_F32) == ZS_EINVAL);  // rows of other lengths in bytes
}

// x and y of a product at random places and strides against their bytes one by
// one: nothing that overlaps is accepted, and at one distance of rows nothing
// else is refused.
void neighbours_at_random(std::mt19937_64& rng) {
    const int64_t out = 3, in = 5;
    const PlanOf plan({out * in}, 1, 1);
    const uint64_t far = uint64_t(1) << 50, base = uint64_t(1) << 40;
    int accepted = 0, refused = 0;
    for (int i = 0; i < 100000; ++i) {
        const int32_t rows = 1 + (int32_t)(rng() % 4), dtype = (int32_t)(rng() % 2);
        const int64_t e = dtype == ZS_DTYPE_BF16 ? 2 : 4, xs = in + (int64_t)(rng() % 8);
        const int64_t ys = rng() % 2 && (xs * 2) % e == 0 && xs * 2 / e >= out ? xs * 2 / e : out + (int64_t)(rng() % 8);
        const uint64_t x = base + 2 * (rng() % 64), y = base + (uint64_t)e * (rng() % 32);
        bool touch = false;
        for (int64_t r = 0; r < rows; ++r)
            for (int64_t q = 0; q < rows; ++q) {
                const uint64_t xr = x + (uint64_t)(r * xs * 2), yr = y + (uint64_t)(q * ys * e);
                touch = touch || (xr < yr + (uint64_t)(out * e) && yr < xr + (uint64_t)(in * 2));
            }
        const zs_status st = zs_quant_matvec(plan.p, 0, out, in, 4, 8, at(far), at<float>(far + 4096), at(x), xs, rows,
                                             at(y), dtype, ys, nullptr);
        CHECK(st == ZS_OK || st == ZS_EINVAL);
        CHECK(!touch || st == ZS_EINVAL);
        if (xs * 2 == ys * e || rows == 1) CHECK(touch == (st == ZS_EINVAL));
        ++(st == ZS_OK ? accepted : refused);
    }
    CHECK(accepted > 1000 && refused > 1000);
}

// Random arguments around the limits: a call that is accepted launches once or
// has nothing to do, any other leaves a text.
void random_calls(std::mt19937_64& rng, int count, const zs_plan* plan) {
    auto pick = [&](std::vector<int64_t> v) { return v[rng() % v.size()]; };
    auto ptr = [&] { return at((rng() % 8 == 0 ? 0 : (rng() % 32) << 36) + (rng() % 4 == 0 ? rng() % 64 : 0)); };
    for (int i = 0; i < count; ++i) {
        const int64_t rows = pick({-1, 0, 1, 2, 5, kRows, kRows + 1}), vocab = pick({0, 1, 7, 1000, kVocab, kVocab + 1});
        const int64_t stride = pick({vocab, vocab + 3, kStride, kStride + 1, -1, INT64_MAX, INT64_MIN});
        const int32_t dtype = (int32_t)pick({0, 1, 1, 2});
        const float t = rng() % 8 ? 1.0f : 0.0f;
        auto* tok = static_cast<int32_t*>(ptr());
        float* f[5];
        for (auto& p : f) p = static_cast<float*>(ptr());
        zs_status st = ZS_OK;
        switch (rng() % 4) {
            case 0:
                st = zs_token_logprobs(ptr(), dtype, rows, vocab, stride, tok, t, f[0], f[1], f[2],
                                       (int32_t)pick({-1, 0, 1, 32, 33, INT32_MAX}), static_cast<int32_t*>(ptr()), f[3],
                                       nullptr);
                break;
            case 1:
                st = zs_token_logprobs_backward(ptr(), dtype, rows, vocab, stride, tok, t, f[0], f[1], f[2], f[3],
                                                ptr(), stride + (int64_t)(rng() % 2 ? 0 : stride < 0), nullptr);
                break;
            case 2:
                st = zs_distill_topk(ptr(), dtype, rows, vocab, stride, tok, f[0],
                                     (int32_t)pick({0, 1, 64, 1024, 1025, INT32_MIN}), t, f[1], f[2], ptr(), stride,
                                     nullptr);
                break;
            default:
                st = zs_quant_matvec(plan, (int32_t)pick({-1, 0, 1, 2}), pick({-6, 0, 6, 12, int64_t(1) << 62}),
                                     pick({-4, 0, 4, 8, INT64_MAX}), (int32_t)pick({4, 8, 5}),
                                     (int32_t)pick({8, 32, 256, 7, 0, INT32_MIN}), ptr(), f[0], ptr(), stride,
                                     (int32_t)pick({-1, 0, 1, 64, 65, INT32_MAX}), ptr(), dtype,
                                     pick({6, 12, kStride, INT64_MAX, -1}), nullptr);
        }
        if (st != ZS_OK) CHECK(std::strlen(zs_last_error()) > 0);
    }
}

// Several threads at once, each of which reads its own error text.
void concurrent_callers() {
    const PlanOf plan({24, 48}, 2, 8);
    std::vector<std::thread> th;
    std::atomic<int> failures{0};
    for (int i = 0; i < 8; ++i)
        th.emplace_back([i, &failures, &plan] {
            std::mt19937_64 rng(100 + (uint64_t)i);
            for (int rep = 0; rep < 200; ++rep) {
                const int k = 2000 + 1000 * i + rep;
                if (zs_distill_topk(at(16), ZS_DTYPE_F32, 1, 8, 8, nullptr, nullptr, k, 1.0f, nullptr, nullptr, nullptr,
                                    8, nullptr) != ZS_EINVAL ||
                    std::string(zs_last_error()).find("k = " + std::to_string(k)) == std::string::npos)
                    ++failures;
                random_calls(rng, 20, plan.p);
            }
        });
    for (auto& t : th) t.join();
    CHECK(failures.load() == 0);
}

}  // namespace

int main(int argc, char** argv) {
    const std::string mode = argc > 1 ? argv[1] : "all";
    if (mode == "all") {
        largest_extents();
        largest_products();
        neighbours();
        const PlanOf plan({24, 48}, 2, 8);
        std::mt19937_64 rng(1);
        neighbours_at_random(rng);
        random_calls(rng, 200000, plan.p);
    }
    concurrent_callers();
    std::printf("lm driver ok (%s)\n", mode.c_str());
    return 0;
}
