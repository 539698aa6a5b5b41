// C-ABI layer of the routing to experts: argument checks and kernel launches.  Every entry
// point is declared and documented in include/mpstep.h.
#include "checks.h"
#include "routing.h"

using namespace mpk;

namespace {

mp_status check_router(const mp_logits* x, const mp_route_cfg* cfg)
{
    mp_status st = check_logits(x);
    if (st != MP_OK) return st;
    if (x->vocab > MP_ROUTE_MAX_EXPERTS)
        return set_error(MP_ERR_INVALID, "a router has at most %d experts", MP_ROUTE_MAX_EXPERTS);
    if (x->temperature != 1.0f) return set_error(MP_ERR_INVALID, "a router's temperature must be 1");
    if (cfg == nullptr) return set_error(MP_ERR_INVALID, "cfg is NULL");
    if (cfg->score != MP_ROUTE_SOFTMAX && cfg->score != MP_ROUTE_SIGMOID)
        return set_error(MP_ERR_INVALID, "cfg: unknown score");
    if (cfg->groups < 1 || cfg->groups > MP_ROUTE_MAX_GROUPS || x->vocab % cfg->groups != 0)
        return set_error(MP_ERR_INVALID, "cfg: groups must be 1 to %d and divide the experts",
                         MP_ROUTE_MAX_GROUPS);
    if (cfg->top_groups < 1 || cfg->top_groups > cfg->groups)
        return set_error(MP_ERR_INVALID, "cfg: top_groups must be 1 to groups");
    if (cfg->group_best != 1 && cfg->group_best != 2)
        return set_error(MP_ERR_INVALID, "cfg: group_best must be 1 or 2");
    if (cfg->top < 1 || cfg->top > MP_ROUTE_MAX_TOP ||
        cfg->top > x->vocab / cfg->groups * cfg->top_groups)
        return set_error(MP_ERR_INVALID, "cfg: top must be 1 to %d, and no more than the experts of "
                                         "top_groups groups", MP_ROUTE_MAX_TOP);
    if (!std::isfinite(cfg->scale)) return set_error(MP_ERR_INVALID, "cfg: scale must be finite");
    return MP_OK;
}

}  // namespace

extern "C" {

mp_status mp_route(const mp_logits* x, const float* bias, const uint8_t* mask, const mp_route_cfg* cfg,
                   const mp_routed* out, mp_stream stream)
{
    mp_status st = check_router(x, cfg);
    if (st != MP_OK) return st;
    if (out == nullptr) return set_error(MP_ERR_INVALID, "routed is NULL");
    if (out->load == nullptr && (out->share != nullptr || out->aux != nullptr))
        return set_error(MP_ERR_INVALID, "share and aux need the load");
    if (out->aux != nullptr && out->share == nullptr)
        return set_error(MP_ERR_INVALID, "aux needs the share");
    if (out->load != nullptr && out->workspace == nullptr)
        return set_error(MP_ERR_INVALID, "the load needs a workspace");
    const int64_t lists = x->rows * cfg->top;
    const int64_t sums = out->load != nullptr ? 1 : 0;
    Arrays arrays;
    st = arrays.in(bias, 4, x->vocab, false, "bias");
    if (st == MP_OK) st = arrays.in(mask, 1, x->rows, false, "mask");
    if (st == MP_OK) st = arrays.out(out->weights, 4, lists, true, "weights");
    if (st == MP_OK) st = arrays.out(out->ids, 8, lists, true, "ids");
    if (st == MP_OK) st = arrays.out(out->load, 8, x->vocab + 1, false, "load");
    if (st == MP_OK) st = arrays.out(out->share, 4, x->vocab, false, "share");
    if (st == MP_OK) st = arrays.out(out->aux, 4, 2, false, "aux");
    if (st == MP_OK) st = arrays.scratch(out->workspace, MP_ROUTE_WORKSPACE_BYTES, sums);
    mp_logits alone = *x;           // the losses' workspace is not used here
    alone.workspace = nullptr;
    if (st == MP_OK) st = arrays.disjoint(&alone, nullptr);
    if (st != MP_OK) return st;
    if (x->rows == 0 && sums == 0) return set_ok();
    st = check_place(x->rows > 0 ? x->data : out->load, x->rows > 0 ? "logits" : "load", stream);
    if (st != MP_OK) return st;
    RouteArgs a{};
    a.x = view_of(x);
    a.bias = bias;
    a.mask = mask;
    a.sigmoid = cfg->score == MP_ROUTE_SIGMOID;
    a.top = cfg->top;
    a.groups = cfg->groups;
    a.top_groups = cfg->top_groups;
    a.group_best = cfg->group_best;
    a.renormalise = cfg->renormalise != 0;
    a.scale = cfg->scale;
    a.weights = out->weights;
    a.ids = out->ids;
    a.load = out->load;
    a.share = out->share;
    a.aux = out->aux;
    a.workspace = out->workspace;
    hipError_t e = launch_route(a, x->dtype, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "route launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_route_grad(const mp_logits* x, const uint8_t* mask, const mp_route_cfg* cfg,
                        const int64_t* ids, const float* dweights, const int64_t* load,
                        float balance_coef, float z_coef, const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_router(x, cfg);
    if (st == MP_OK && grad == nullptr) st = set_error(MP_ERR_INVALID, "grad is NULL");
    if (st == MP_OK) st = check_grad(x, grad);
    if (st != MP_OK) return st;
    if (!std::isfinite(balance_coef) || !std::isfinite(z_coef))
        return set_error(MP_ERR_INVALID, "the losses' coefficients must be finite");
    if (cfg->score == MP_ROUTE_SIGMOID && z_coef != 0.0f)
        return set_error(MP_ERR_INVALID, "z_coef is of a softmax's logits");
    const bool aux = balance_coef != 0.0f || z_coef != 0.0f;
    if (aux && load == nullptr) return set_error(MP_ERR_INVALID, "the auxiliary losses need the load");
    if (!aux && dweights == nullptr) return set_error(MP_ERR_INVALID, "dweights or a loss is required");
    const int64_t lists = x->rows * cfg->top;
    Arrays arrays;
    st = arrays.in(mask, 1, x->rows, false, "mask");
    if (st == MP_OK) st = arrays.in(ids, 8, lists, true, "ids");
    if (st == MP_OK) st = arrays.in(dweights, 4, lists, false, "dweights");
    if (st == MP_OK) st = arrays.in(load, 8, x->vocab + 1, false, "load");
    mp_logits alone = *x;
    alone.workspace = nullptr;
    if (st == MP_OK) st = arrays.disjoint(&alone, grad);
    if (st != MP_OK) return st;
    if (x->rows == 0) return set_ok();
    st = check_place(x->data, "logits", stream);
    if (st != MP_OK) return st;
    RouteGradArgs a{};
    a.x = view_of(x);
    a.g = view_of(x, grad);
    a.mask = mask;
    a.sigmoid = cfg->score == MP_ROUTE_SIGMOID;
    a.top = cfg->top;
    a.renormalise = cfg->renormalise != 0;
    a.scale = cfg->scale;
    a.ids = ids;
    a.dweights = dweights;
    a.load = aux ? load : nullptr;
    a.balance = balance_coef;
    a.large = z_coef;
    hipError_t e = launch_route_grad(a, x->dtype, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "gradient launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_route_bias_update(int32_t layers, int32_t experts, const float* bias, int32_t n_loads,
                               const int64_t* load, float speed, float* out, const mp_state* state,
                               mp_stream stream)
{
    if (layers < 0 || layers > (1 << 20)) return set_error(MP_ERR_INVALID, "layers must be 0 to 2^20");
    if (experts < 1 || experts > MP_ROUTE_MAX_EXPERTS)
        return set_error(MP_ERR_INVALID, "experts must be 1 to %d", MP_ROUTE_MAX_EXPERTS);
    if (n_loads < 1 || n_loads > (1 << 20)) return set_error(MP_ERR_INVALID, "n_loads must be 1 to 2^20");
    if (!std::isfinite(speed)) return set_error(MP_ERR_INVALID, "speed must be finite");
    const int64_t n = int64_t(layers) * experts;
    mp_logits none{};
    Arrays arrays;
    mp_status st = arrays.in(load, 8, int64_t(n_loads) * layers * (experts + 1), true, "load");
    if (st == MP_OK) st = arrays.out(out, 4, n, true, "out");
    // each element is read and then written by one lane: the bias may be replaced
    if (st == MP_OK && bias == nullptr && n > 0) st = set_error(MP_ERR_INVALID, "bias is NULL");
    if (st == MP_OK && bias != out) st = arrays.in(bias, 4, n, true, "bias");
    if (st == MP_OK) st = arrays.disjoint(&none, nullptr);
    if (st != MP_OK) return st;
    if (layers == 0) return set_ok();
    st = check_place(out, "out", stream);
    RouteBiasArgs a{};
    if (st == MP_OK && state != nullptr) st = state_found_inf(state, &a.skipped);
    if (st != MP_OK) return st;
    a.layers = layers;
    a.experts = experts;
    a.n_loads = n_loads;
    a.bias = bias;
    a.load = load;
    a.speed = speed;
    a.out = out;
    hipError_t e = launch_route_bias(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "bias update launch: %s", hipGetErrorString(e));
    return set_ok();
}

}  // extern "C"
