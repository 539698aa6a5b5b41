// C-ABI layer of the scores of logits: argument checks and kernel launches.  Every entry
// point is declared and documented in include/mpstep.h.
#include "checks.h"
#include "scores.h"

using namespace mpk;

extern "C" {

mp_status mp_token_score(const mp_logits* x, const int64_t* targets, const mp_score* out,
                         mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st != MP_OK) return st;
    if (out == nullptr) return set_error(MP_ERR_INVALID, "score is NULL");
    if (out->top < 0 || out->top > MP_SCORE_MAX_TOP)
        return set_error(MP_ERR_INVALID, "top must be 0 to %d", MP_SCORE_MAX_TOP);
    if (out->top == 0 &&
        (out->top_ids != nullptr || out->top_logp != nullptr || out->top_values != nullptr))
        return set_error(MP_ERR_INVALID, "top = 0 takes no lists");
    if (out->logp != nullptr && targets == nullptr)
        return set_error(MP_ERR_INVALID, "logp needs targets");
    if (out->top == 0 && out->logp == nullptr && out->lse == nullptr && out->entropy == nullptr)
        return set_error(MP_ERR_INVALID, "the score has no output");
    const int64_t lists = x->rows * out->top;
    Arrays arrays;
    st = arrays.in(targets, 8, x->rows, false, "targets");
    if (st == MP_OK) st = arrays.out(out->logp, 4, x->rows, false, "logp");
    if (st == MP_OK) st = arrays.out(out->lse, 4, x->rows, false, "lse");
    if (st == MP_OK) st = arrays.out(out->entropy, 4, x->rows, false, "entropy");
    if (st == MP_OK) st = arrays.out(out->top_ids, 8, lists, out->top > 0, "top_ids");
    if (st == MP_OK) st = arrays.out(out->top_logp, 4, lists, false, "top_logp");
    if (st == MP_OK) st = arrays.out(out->top_values, 4, lists, false, "top_values");
    if (st == MP_OK) st = arrays.scratch(out->workspace, MP_SCORE_WORKSPACE_BYTES, x->rows);
    mp_logits alone = *x;           // the losses' workspace is not used here
    alone.workspace = nullptr;
    if (st == MP_OK) st = arrays.disjoint(&alone, nullptr);
    if (st != MP_OK) return st;
    if (x->rows == 0) return set_ok();
    st = check_place(x->data, "logits", stream);
    if (st != MP_OK) return st;
    ScoreArgs a{};
    a.x = view_of(x);
    a.targets = targets;
    a.logp = out->logp;
    a.lse = out->lse;
    a.entropy = out->entropy;
    a.top_ids = out->top_ids;
    a.top_logp = out->top_logp;
    a.top_values = out->top_values;
    a.workspace = out->workspace;
    a.top = out->top;
    hipError_t e = launch_scores(a, x->dtype, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "score launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_token_score_grad(const mp_logits* x, const int64_t* targets, const float* lse,
                              const float* entropy, const float* dlogp, const float* dentropy,
                              const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK && grad == nullptr) st = set_error(MP_ERR_INVALID, "grad is NULL");
    if (st == MP_OK) st = check_grad(x, grad);
    if (st == MP_OK && dlogp == nullptr && dentropy == nullptr)
        st = set_error(MP_ERR_INVALID, "dlogp or dentropy is required");
    if (st == MP_OK && dlogp != nullptr && targets == nullptr)
        st = set_error(MP_ERR_INVALID, "dlogp needs targets");
    if (st == MP_OK && dentropy != nullptr && entropy == nullptr)
        st = set_error(MP_ERR_INVALID, "dentropy needs the entropy");
    if (st != MP_OK) return st;
    Arrays arrays;
    st = arrays.in(targets, 8, x->rows, false, "targets");
    if (st == MP_OK) st = arrays.in(lse, 4, x->rows, true, "lse");
    if (st == MP_OK) st = arrays.in(entropy, 4, x->rows, false, "entropy");
    if (st == MP_OK) st = arrays.in(dlogp, 4, x->rows, false, "dlogp");
    if (st == MP_OK) st = arrays.in(dentropy, 4, x->rows, false, "dentropy");
    mp_logits alone = *x;
    alone.workspace = nullptr;
    if (st == MP_OK) st = arrays.disjoint(&alone, grad);
    if (st != MP_OK) return st;
    if (x->rows == 0) return set_ok();
    st = check_place(x->data, "logits", stream);
    if (st != MP_OK) return st;
    ScoreGradArgs a{};
    a.x = view_of(x);
    a.g = view_of(x, grad);
    a.targets = targets;
    a.lse = lse;
    a.entropy = entropy;
    a.dlogp = dlogp;
    a.dentropy = dentropy;
    hipError_t e = launch_score_grad(a, x->dtype, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "gradient launch: %s", hipGetErrorString(e));
    return set_ok();
}

}  // extern "C"
