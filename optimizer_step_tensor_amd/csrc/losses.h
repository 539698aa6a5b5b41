// Internal layout shared by the C-ABI layer of the losses (losses_api.hip) and
// their kernels (losses.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mpstep.h"

namespace mpk {

// The row formula of a fused loss pass.
enum LossKind : int32_t { kLogprob, kXent, kPolicy, kDistill };

// The logits of one call, as the kernels take them.
struct LogitsView {
    const void* x;
    int64_t stride;       // elements
    int32_t rows;
    int32_t vocab;
    int32_t stream;       // set by the launch: read past the infinity cache
    float k_hi, k_lo;     // log2(e) / T as a sum of two positive floats, k_hi the larger
    double inv_t;         // 1 / T
};

// Where the gradient goes (dx NULL: nowhere) and what multiplies it.
struct GradView {
    void* dx;
    int64_t stride;
    const float* dev_scale;
    const int64_t* dev_count;
    double scale;         // scale / T
};

struct LossArgs {
    LogitsView x;
    GradView g;
    void* workspace;              // MP_LOSS_WORKSPACE_BYTES, or NULL
    int32_t kind;
    int32_t k;                    // teacher's entries per row
    const int64_t* targets;       // NULL for distillation
    const float* weights;         // NULL: all 1
    float* loss;                  // NULL where the call has none
    float* logp;
    float* lse;
    float* kl;
    const float* old_logp;
    const float* ref_logp;
    const float* advantage;
    float clip_low, clip_high, kl_coef;
    int32_t teacher_dtype;
    const void* teacher_values;
    const int64_t* teacher_ids;
    const float* teacher_lse;
};

struct PairArgs {
    const int64_t* targets;
    const int64_t* seq_start;
    const float* ref_logp;
    const float* logp;
    float* loss;
    float* seq_logp;
    float* dlogp;
    int64_t n_pairs;
    int32_t rows;
    int32_t kind;
    int32_t length_mean;
    double beta, label_smoothing, margin;
};

hipError_t launch_target_count(int64_t n, const int64_t* targets, int64_t* count, hipStream_t s);
// The statistics of every row, its loss and (g.dx set) its gradient.
hipError_t launch_rows(const LossArgs& a, int dtype, hipStream_t s);
// dx = factor * dlogp * (onehot(target) - exp(z - lse))
hipError_t launch_logprob_grad(const LogitsView& x, const int64_t* targets, const float* lse,
                               const float* dlogp, const GradView& g, int dtype, hipStream_t s);
hipError_t launch_pairs(const PairArgs& a, hipStream_t s);

// api.hip: record the detail of an error (printf-style) and return its status; clear it.
mp_status set_error(mp_status st, const char* fmt, ...);
mp_status set_ok();

}  // namespace mpk
