// Internal declarations of the language-model operators (zs_lm.h): what their
// host side shares with the step's (zs_api.cpp) and the kernel launchers. Not
// part of the public ABI.
#pragma once

#include <cstdint>

#include "../../include/zs_lm.h"
#include "zs_internal.h"

namespace zs {

// zs_api.cpp: records a thread's error text and returns st; turns a launcher's
// hipError_t value into a status; writes the ZS_LOG line of a call.
zs_status report(zs_status st, const char* fmt, ...);
zs_status report_hip(int err, const char* what);
void trace_call(const char* op, const zs_plan* p, int32_t n_contribs, int64_t off, int64_t len, const void* stream);

// A row-major matrix in device memory: rows start `stride` elements apart.
struct Rows {
    const void* p;
    int64_t stride;
};

// Where a tensor's codes and scales lie in the gathered payload. Codes are
// contiguous over all ranks (every shard is a whole number of code bytes):
// element j of the flat buffer is code j. Its scale is number
// (j / shard) * n_scales + (j % shard) / block.
struct QuantWeight {
    const void* codes;
    const float* scales;
    int64_t off;       // the tensor's first element in the flat buffer
    int64_t n_out, n_in;
    int64_t shard;     // S
    int64_t n_scales;  // scales a rank
    int32_t world;     // N
    int32_t bits;
    int32_t block_shift;  // log2(block)
};

// Launchers; they return a hipError_t value cast to int.
int launch_quant_matvec(const QuantWeight& w, Rows x, int rows, void* y, int y_dtype, int64_t y_stride, void* stream);

struct LogprobsOut {
    float* logprob;
    float* entropy;
    float* stats;
    int32_t* top_ids;
    float* top_logprobs;
    int32_t top;
};
int launch_logprobs(Rows logits, int dtype, int64_t rows, int64_t vocab, const int32_t* tokens, double temperature,
                    const LogprobsOut& out, void* stream);

struct LogprobsGradIn {
    const int32_t* tokens;
    const float* stats;
    const float* entropy;
    const float* grad_logprob;
    const float* grad_entropy;
};
int launch_logprobs_grad(Rows logits, int dtype, int64_t rows, int64_t vocab, double temperature,
                         const LogprobsGradIn& in, void* grad, int64_t grad_stride, void* stream);

struct Teacher {
    const int32_t* ids;
    const float* logits;
    int32_t k;
    const float* row_weight;
};
int launch_distill(Rows logits, int dtype, int64_t rows, int64_t vocab, const Teacher& t, double temperature,
                   float* loss, void* grad, int64_t grad_stride, void* stream);

}  // namespace zs
