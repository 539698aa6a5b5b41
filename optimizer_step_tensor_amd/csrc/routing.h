// Internal layout shared by the C-ABI layer of the routing to experts (routing_api.hip)
// and its kernels (routing.hip).
#pragma once

#include "losses.h"

namespace mpk {

struct RouteArgs {
    LogitsView x;                 // vocab: the experts
    const float* bias;            // NULL: none
    const uint8_t* mask;          // NULL: every token is routed
    int32_t sigmoid;
    int32_t top, groups, top_groups, group_best, renormalise;
    float scale;
    float* weights;
    int64_t* ids;
    int64_t* load;                // NULL: no sums over the tokens
    float* share;                 // NULL with load NULL, or not wanted
    float* aux;                   // the same
    void* workspace;              // MP_ROUTE_WORKSPACE_BYTES with load
};

struct RouteGradArgs {
    LogitsView x;
    GradView g;                   // its factor is of the auxiliary losses
    const uint8_t* mask;
    int32_t sigmoid;
    int32_t top, renormalise;
    float scale;
    const int64_t* ids;           // NULL with dweights
    const float* dweights;
    const int64_t* load;          // NULL without auxiliary losses
    float balance, large;
};

struct RouteBiasArgs {
    int32_t layers, experts, n_loads;
    const float* bias;
    const int64_t* load;
    float speed;
    float* out;
    const int32_t* skipped;       // NULL, or nonzero there: the bias stays
};

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s);
hipError_t launch_route_grad(const RouteGradArgs& a, int dtype, hipStream_t s);
hipError_t launch_route_bias(const RouteBiasArgs& a, hipStream_t s);

// api.hip: the overflow flag of a state's last check, in device memory; refused where the state
// is another device's.
mp_status state_found_inf(const mp_state* state, const int32_t** flag);

}  // namespace mpk
