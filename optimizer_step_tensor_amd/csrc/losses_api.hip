// C-ABI layer of the losses over vocabulary logits: argument checks and kernel
// launches.  Every entry point is declared and documented in include/mpstep.h.
#include "checks.h"

using namespace mpk;

namespace {

mp_status run_rows(const mp_logits* x, const mp_logits_grad* g, LossArgs& a, mp_stream stream)
{
    if (x->rows == 0) return set_ok();
    mp_status st = check_place(x->data, "logits", stream);
    if (st != MP_OK) return st;
    a.x = view_of(x);
    a.g = view_of(x, g);
    a.workspace = x->workspace;
    hipError_t e = mpk::launch_rows(a, x->dtype, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "loss launch: %s", hipGetErrorString(e));
    return set_ok();
}

}  // namespace

extern "C" {

mp_status mp_target_count(int64_t n, const int64_t* targets, int64_t* count, mp_stream stream)
{
    if (n < 0) return set_error(MP_ERR_INVALID, "n must be >= 0");
    Arrays arrays;
    mp_status st = arrays.in(targets, 8, n, true, "targets");
    if (st == MP_OK) st = arrays.out(count, 8, 1, true, "count");
    if (st == MP_OK) st = check_place(count, "count", stream);
    if (st != MP_OK) return st;
    hipError_t e = mpk::launch_target_count(n, targets, count, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "target count launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_token_logprob(const mp_logits* x, const int64_t* targets, float* logp, float* lse,
                           mp_stream stream)
{
    mp_status st = check_logits(x);
    Arrays arrays;
    if (st == MP_OK) st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.out(logp, 4, x->rows, true, "logp");
    if (st == MP_OK) st = arrays.out(lse, 4, x->rows, false, "lse");
    if (st == MP_OK) st = arrays.disjoint(x, nullptr);
    if (st != MP_OK) return st;
    LossArgs a{};
    a.kind = mpk::kLogprob;
    a.targets = targets;
    a.logp = logp;
    a.lse = lse;
    return run_rows(x, nullptr, a, stream);
}

mp_status mp_token_logprob_grad(const mp_logits* x, const int64_t* targets, const float* lse,
                                const float* dlogp, const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK && grad == nullptr) st = set_error(MP_ERR_INVALID, "grad is NULL");
    if (st == MP_OK) st = check_grad(x, grad);
    Arrays arrays;
    if (st == MP_OK) st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.in(lse, 4, x->rows, true, "lse");
    if (st == MP_OK) st = arrays.in(dlogp, 4, x->rows, true, "dlogp");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st != MP_OK) return st;
    if (x->rows == 0) return set_ok();
    st = check_place(x->data, "logits", stream);
    if (st != MP_OK) return st;
    hipError_t e = mpk::launch_logprob_grad(view_of(x), targets, lse, dlogp, view_of(x, grad), x->dtype,
                                            static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "gradient launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_cross_entropy(const mp_logits* x, const int64_t* targets, const float* weights,
                           float* loss, const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK) st = check_grad(x, grad);
    Arrays arrays;
    if (st == MP_OK) st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.in(weights, 4, x->rows, false, "weights");
    if (st == MP_OK) st = arrays.out(loss, 4, x->rows, true, "loss");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st != MP_OK) return st;
    LossArgs a{};
    a.kind = mpk::kXent;
    a.targets = targets;
    a.weights = weights;
    a.loss = loss;
    return run_rows(x, grad, a, stream);
}

mp_status mp_policy_loss(const mp_logits* x, const int64_t* targets, const float* old_logp,
                         const float* ref_logp, const float* advantage, const float* weights,
                         const mp_policy_cfg* cfg, float* loss, float* logp, float* kl,
                         const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK) st = check_grad(x, grad);
    if (st != MP_OK) return st;
    if (cfg == nullptr) return set_error(MP_ERR_INVALID, "cfg is NULL");
    if (!(cfg->clip_low >= 0.0f && cfg->clip_low <= 1.0f))
        return set_error(MP_ERR_INVALID, "clip_low must be in [0, 1]");
    if (!(cfg->clip_high >= 0.0f) || !std::isfinite(cfg->clip_high))
        return set_error(MP_ERR_INVALID, "clip_high must be finite and >= 0");
    if (!(cfg->kl_coef >= 0.0f) || !std::isfinite(cfg->kl_coef))
        return set_error(MP_ERR_INVALID, "kl_coef must be finite and >= 0");
    if (x->rows > 0 && ref_logp == nullptr && (cfg->kl_coef != 0.0f || kl != nullptr))
        return set_error(MP_ERR_INVALID, "a KL term needs ref_logp");
    Arrays arrays;
    st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.in(old_logp, 4, x->rows, true, "old_logp");
    if (st == MP_OK) st = arrays.in(ref_logp, 4, x->rows, false, "ref_logp");
    if (st == MP_OK) st = arrays.in(advantage, 4, x->rows, true, "advantage");
    if (st == MP_OK) st = arrays.in(weights, 4, x->rows, false, "weights");
    if (st == MP_OK) st = arrays.out(loss, 4, x->rows, true, "loss");
    if (st == MP_OK) st = arrays.out(logp, 4, x->rows, false, "logp");
    if (st == MP_OK) st = arrays.out(kl, 4, x->rows, false, "kl");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st != MP_OK) return st;
    LossArgs a{};
    a.kind = mpk::kPolicy;
    a.targets = targets;
    a.weights = weights;
    a.loss = loss;
    a.logp = logp;
    a.kl = kl;
    a.old_logp = old_logp;
    a.ref_logp = ref_logp;
    a.advantage = advantage;
    a.clip_low = cfg->clip_low;
    a.clip_high = cfg->clip_high;
    a.kl_coef = cfg->kl_coef;
    return run_rows(x, grad, a, stream);
}

mp_status mp_preference_loss(const mp_logits* x, const int64_t* targets, int64_t n_pairs,
                             const int64_t* seq_start, const float* ref_logp,
                             const mp_preference_cfg* cfg, float* loss, float* seq_logp,
                             float* logp, float* lse, float* dlogp, const mp_logits_grad* grad,
                             mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK) st = check_grad(x, grad);
    if (st != MP_OK) return st;
    if (cfg == nullptr) return set_error(MP_ERR_INVALID, "cfg is NULL");
    if (cfg->kind != MP_PREF_SIGMOID && cfg->kind != MP_PREF_SQUARED)
        return set_error(MP_ERR_INVALID, "kind must be MP_PREF_SIGMOID or MP_PREF_SQUARED");
    if (!(cfg->beta > 0.0f) || !std::isfinite(cfg->beta))
        return set_error(MP_ERR_INVALID, "beta must be finite and > 0");
    if (!(cfg->label_smoothing >= 0.0f && cfg->label_smoothing <= 0.5f))
        return set_error(MP_ERR_INVALID, "label_smoothing must be in [0, 0.5]");
    if (!std::isfinite(cfg->margin)) return set_error(MP_ERR_INVALID, "margin must be finite");
    if (n_pairs < 1 || n_pairs > kMaxRows)
        return set_error(MP_ERR_INVALID, "n_pairs must be 1 to 2^22 - 1");
    Arrays arrays;
    st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.in(seq_start, 8, 2 * n_pairs + 1, true, "seq_start");
    if (st == MP_OK) st = arrays.in(ref_logp, 4, 2 * n_pairs, false, "ref_logp");
    if (st == MP_OK) st = arrays.out(loss, 4, n_pairs, true, "loss");
    if (st == MP_OK) st = arrays.out(seq_logp, 4, 2 * n_pairs, true, "seq_logp");
    if (st == MP_OK) st = arrays.out(logp, 4, x->rows, true, "logp");
    if (st == MP_OK) st = arrays.out(lse, 4, x->rows, true, "lse");
    if (st == MP_OK) st = arrays.out(dlogp, 4, x->rows, true, "dlogp");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st == MP_OK) st = check_place(x->rows > 0 ? x->data : seq_start,
                                      x->rows > 0 ? "logits" : "seq_start", stream);
    if (st != MP_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    LossArgs a{};
    a.kind = mpk::kLogprob;
    a.x = view_of(x);
    a.workspace = x->workspace;
    a.targets = targets;
    a.logp = logp;
    a.lse = lse;
    mpk::PairArgs p{};
    p.targets = targets;
    p.seq_start = seq_start;
    p.ref_logp = ref_logp;
    p.logp = logp;
    p.loss = loss;
    p.seq_logp = seq_logp;
    p.dlogp = dlogp;
    p.n_pairs = n_pairs;
    p.rows = static_cast<int32_t>(x->rows);
    p.kind = cfg->kind;
    p.length_mean = cfg->length_mean != 0;
    p.beta = static_cast<double>(cfg->beta);
    p.label_smoothing = static_cast<double>(cfg->label_smoothing);
    p.margin = static_cast<double>(cfg->margin);
    hipError_t e = x->rows > 0 ? mpk::launch_rows(a, x->dtype, s) : hipSuccess;
    if (e == hipSuccess) e = mpk::launch_pairs(p, s);
    if (e == hipSuccess && grad != nullptr && x->rows > 0)
        e = mpk::launch_logprob_grad(a.x, targets, lse, dlogp, view_of(x, grad), x->dtype, s);
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "preference launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_distill_loss(const mp_logits* x, const mp_teacher* teacher, const float* weights,
                          float* loss, const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK) st = check_grad(x, grad);
    if (st != MP_OK) return st;
    if (teacher == nullptr) return set_error(MP_ERR_INVALID, "teacher is NULL");
    if (teacher->k < 1 || teacher->k > MP_DISTILL_MAX_K)
        return set_error(MP_ERR_INVALID, "teacher: k must be 1 to %d", MP_DISTILL_MAX_K);
    if (!known_dtype(teacher->dtype)) return set_error(MP_ERR_INVALID, "teacher: unknown dtype");
    Arrays arrays;
    const int64_t entries = x->rows * teacher->k;
    st = arrays.in(teacher->values, elem_bytes(teacher->dtype), entries, true, "teacher values");
    if (st == MP_OK) st = arrays.in(teacher->ids, 8, entries, true, "teacher ids");
    if (st == MP_OK) st = arrays.in(teacher->lse, 4, x->rows, false, "teacher lse");
    if (st == MP_OK) st = arrays.in(weights, 4, x->rows, false, "weights");
    if (st == MP_OK) st = arrays.out(loss, 4, x->rows, true, "loss");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st != MP_OK) return st;
    LossArgs a{};
    a.kind = mpk::kDistill;
    a.weights = weights;
    a.loss = loss;
    a.k = teacher->k;
    a.teacher_dtype = teacher->dtype;
    a.teacher_values = teacher->values;
    a.teacher_ids = teacher->ids;
    a.teacher_lse = teacher->lse;
    return run_rows(x, grad, a, stream);
}

}  // extern "C"
