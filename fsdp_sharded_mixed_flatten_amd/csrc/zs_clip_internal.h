// What the clipping of the multi-tensor step (zs_clip.h) shares with the step's
// host side (zs_api.cpp), and its kernel launchers. Not part of the public ABI.
#pragma once

#include <cstdint>

#include "../../include/zs_clip.h"
#include "zs_internal.h"

namespace zs {

// The tables of a bound workspace. unsummed: byte offset of one byte a piece, 1
// where its squares are another rank's to count; 0: this rank counts all. bytes:
// of the whole binding.
struct BoundTables {
    MultiOffsets off;
    int64_t unsummed, bytes;
};

// zs_api.cpp: the tables of the binding in a workspace, after checking that it
// is of this plan and, unless the plan has no element, has the fields of `need`
// (MultiFlags); the coefficients of each group's hyperparameters.
zs_status bound_tables(const zs_plan* plan, const void* workspace, int32_t need, BoundTables* out);
zs_status group_coefs(const zs_plan* plan, const zs_adamw_hparams* hps, int32_t n_groups, CoefTable* ct);

// Chunks (kChunkElems elements each) that one workgroup of the norm adds up, and
// the bytes of the workgroups' sums and flags (of a plan without elements: some,
// so that a workspace has an address).
constexpr int64_t kNormChunks = 64;
inline int64_t norm_groups(int64_t n_chunks) { return (n_chunks + kNormChunks - 1) / kNormChunks; }
inline int64_t norm_bytes(int64_t n_chunks) {
    const int64_t n = norm_groups(n_chunks);
    return ((n > 0 ? n : 1) * 12 + 255) / 256 * 256;
}

// Launchers; they return a hipError_t value cast to int.
int launch_multi_norm(const void* workspace, const BoundTables& t, int64_t n_chunks, double* sumsq_out,
                      int32_t* nonfinite_out, void* stats_workspace, void* stream);
int launch_multi_clip(const CoefTable& c, const void* workspace, const BoundTables& t, int64_t n_chunks,
                      const float* scale, const int32_t* skip, void* stream);

}  // namespace zs
