// args_beam.h -- launch interface of the beam selection (between the C ABI layer, api_beam.cu, and the
// kernel translation unit).  Internal to libsinkattn.
#pragma once
#include "args_common.h"

namespace sinkattn {

constexpr int kDtF32 = 0, kDtBf16 = 1, kDtF16 = 2;  // sinkattn_dtype_t
constexpr int kBeamMaxBeams = 32;    // K
constexpr int kBeamMaxSelect = 64;   // M
constexpr int kBeamMaxPart = 262144;  // tokens of one row that one CTA reads at most

constexpr int kBeamMaxCands = 4096;  // K x shares of a row x M: candidates that meet in the merge

// One CTA's share of a row: its largest logit m and its sum of exponentials, hi + lo = sum 2^(x L - r2) with L the
// float log2(e), or, where r2 is +inf (|m| above 2^20), sum e^(x - m).
struct BeamPart {
    float r2, m, hi, lo;
};
struct BeamArgs {
    const void* logits;         // [N * K rows, V], rows row_stride elements apart
    const float* scores;        // [N * K]
    const uint8_t* finished;    // [N * K] or null
    float* out_scores;          // [N, M]
    int32_t* out_parents;       // [N, M]
    int32_t* out_tokens;        // [N, M]
    BeamPart* part;             // [N * K, parts]
    unsigned long long* best;   // [N * K, parts, M] (order of the logit, ~token), descending, 0 = none
    unsigned* err;
    long long row_stride;
    int N, K, V, M, pad_token, dtype;
    int parts, part_len;        // CTAs per row, tokens of each (a multiple of 32; the last may have fewer)
};
struct BeamPlan {
    int parts, part_len;
    size_t best_offset, ws_bytes;
};
cudaError_t beam_plan(int N, int K, int V, int M, BeamPlan* plan);
cudaError_t beam_select_launch(const BeamArgs& args, cudaStream_t stream);

}  // namespace sinkattn
