// Internal layout shared by the C-ABI layer of the scores of logits (scores_api.hip)
// and their kernels (scores.hip).
#pragma once

#include "losses.h"

namespace mpk {

struct ScoreArgs {
    LogitsView x;
    const int64_t* targets;       // NULL: no log-probabilities, and every row counts
    float* logp;                  // each output may be NULL
    float* lse;
    float* entropy;
    int64_t* top_ids;             // rows x top; NULL with top = 0
    float* top_logp;
    float* top_values;
    void* workspace;              // MP_SCORE_WORKSPACE_BYTES, or NULL
    int32_t top;
};

struct ScoreGradArgs {
    LogitsView x;
    GradView g;
    const int64_t* targets;       // NULL with dlogp
    const float* lse;
    const float* entropy;         // NULL with dentropy
    const float* dlogp;
    const float* dentropy;
};

hipError_t launch_scores(const ScoreArgs& a, int dtype, hipStream_t s);
hipError_t launch_score_grad(const ScoreGradArgs& a, int dtype, hipStream_t s);

}  // namespace mpk
