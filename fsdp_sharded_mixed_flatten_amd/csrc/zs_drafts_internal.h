// Kernel launcher of the verification of drafted tokens (zs_drafts.h) and its
// workspace. Not part of the public ABI.
#pragma once

#include <cstdint>

#include "../../include/zs_drafts.h"
#include "zs_lm_internal.h"

namespace zs {

// Logits of a row that one wave sums: large pieces where there are many of them,
// small ones where waves are few and each one's time counts, and for short rows.
// us of a call with 4 drafts in bf16 in a graph, large and small pieces:
//   1 x 32000    24  14     1 x 151936   23  18    256 x 32000    95 113
//   8 x 32000    30  17     4 x 151936   28  24    16 x 100000    39  33
//   64 x 32000   44  36     8 x 151936   32  31    32 x 65536     37  37
//   128 x 32000  61  63     16 x 151936  43  47    64 x 151936   101 144
// Without drafts 1 x 32000 16 and 11, 64 x 151936 23 and 37; 300 x 500 (2 drafts)
// has a piece a row either way. The rule errs most at 64 x 32000, whose 11520 pieces
// are large, and at 64 x 151936 without drafts, whose 4800 are not.
constexpr int32_t kVerifyPiece = 2048, kVerifySmallPiece = 512;
constexpr int64_t kVerifyManyPieces = 8192;

// Largest logit of a piece (NaN: there is a NaN or +infinity in it) and the sum of
// its exponentials relative to that logit, in 64 bits.
struct VerifyPart {
    double top, sum;
};

// What the first workgroup of a request leaves for the draw.
struct VerifyPick {
    double p_top, p_sum, q_top, q_sum;
    int32_t at;     // the place the token is drawn for
    int32_t kind;   // VerifyKind
    int32_t token;  // the drafted token that fell
    int32_t unused;
};
enum VerifyKind : int32_t { kDrawNothing = 0, kDrawTarget = 1, kDrawRest = 2 };

// The workspace: parts [rows, pieces], the target's rows before the drafts';
// totals [requests, pieces]; picks [requests].
struct VerifyLayout {
    int32_t piece;
    int64_t pieces, rows, totals_off, picks_off, bytes;
};
inline VerifyLayout verify_layout(int64_t requests, int32_t drafts, int64_t vocab) {
    VerifyLayout l;
    l.rows = requests * (2 * (int64_t)drafts + 1);
    const int64_t large = (vocab + kVerifyPiece - 1) / kVerifyPiece;
    l.piece = vocab >= kVerifyPiece && l.rows * large >= kVerifyManyPieces ? kVerifyPiece : kVerifySmallPiece;
    l.pieces = (vocab + l.piece - 1) / l.piece;
    l.totals_off = l.rows * l.pieces * (int64_t)sizeof(VerifyPart);
    l.picks_off = l.totals_off + requests * l.pieces * 8;
    // a workspace serves every smaller call, the ones of small pieces too
    const int64_t small = (l.rows > kVerifyManyPieces ? l.rows : kVerifyManyPieces) *
                          (kVerifyPiece / kVerifySmallPiece) * (int64_t)(sizeof(VerifyPart) + 8);
    if (l.piece == kVerifyPiece && l.picks_off < small) l.picks_off = small;
    l.bytes = l.picks_off + requests * (int64_t)sizeof(VerifyPick);
    return l;
}

struct VerifyArgs {
    Rows target, draft;  // draft.p may be NULL
    int64_t requests, vocab;
    int32_t drafts;
    const int32_t* tokens;
    const int32_t* lens;  // may be NULL
    const float* uniforms;
    int32_t* accepted;
    int32_t* out;
    float* logprobs;  // may be NULL
};

// Returns a hipError_t value cast to int.
int launch_verify(const VerifyArgs& a, int dtype, double temperature, void* workspace, void* stream);

}  // namespace zs
