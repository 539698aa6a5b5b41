// HIP kernels of the routing to experts: the choice and the weights of each token, the sums over the
// tokens that balance the experts, the gradient of all of it, and the balancing bias's step.
//
// Experts are chosen by c_e = s_e + b_e, s = softmax(x) or sigmoid(x).  Two of a token's c are closer
// than 2^-24 about once in 10^5 tokens, and fp32 arithmetic would then choose by its rounding
// errors: c is formed in binary64, which runs at fp32's rate here.  A choice is made on c rounded to
// 42 bits, with the expert's number in the last ten (`expert_key`), so that one maximum finds the
// largest c and, of equal ones, the lowest number.
#include <float.h>

#include "rows.h"
#include "routing.h"

namespace mpk {
namespace {

// 2^y for -1100 <= y <= 1000: y's fraction by the exponential series (14 digits), its whole part as the
// exponent.  (No table and no double-word steps: the library's exp takes twice the operations.)
__device__ __forceinline__ double exp2_series(double y)
{
    const double whole = __builtin_rint(y);
    const double t = (y - whole) * 0.69314718055994531;        // |t| < 0.3466
    double p = 1.0 / 39916800.0;                               // t^12 / 12! < 7e-15
    p = __builtin_fma(p, t, 1.0 / 3628800.0);
    p = __builtin_fma(p, t, 1.0 / 362880.0);
    p = __builtin_fma(p, t, 1.0 / 40320.0);
    p = __builtin_fma(p, t, 1.0 / 5040.0);
    p = __builtin_fma(p, t, 1.0 / 720.0);
    p = __builtin_fma(p, t, 1.0 / 120.0);
    p = __builtin_fma(p, t, 1.0 / 24.0);
    p = __builtin_fma(p, t, 1.0 / 6.0);
    p = __builtin_fma(p, t, 0.5);
    p = __builtin_fma(p, t, 1.0);
    p = __builtin_fma(p, t, 1.0);
    return __builtin_ldexp(p, static_cast<int>(whole));
}

// 1 / d for 1 <= d <= 2^1000 or so: the instruction's 2^-26 and two of Newton's steps.
__device__ __forceinline__ double reciprocal(double d)
{
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

constexpr double kLog2E = 1.4426950408889634;

__device__ __forceinline__ double clamp_exponent(double y)
{
    return __builtin_fmin(__builtin_fmax(y, -1100.0), 1000.0);
}

__device__ __forceinline__ double sigmoid_of(float z)
{
    const double y = static_cast<double>(z) * -kLog2E;
    return y > 1000.0 ? 0.0 : reciprocal(1.0 + exp2_series(clamp_exponent(y)));
}

// exp(z - m), z <= m.
__device__ __forceinline__ double share_to(float z, float m)
{
    return exp2_series(clamp_exponent((static_cast<double>(z) - static_cast<double>(m)) * kLog2E));
}

constexpr int kIdBits = 10;                              // MP_ROUTE_MAX_EXPERTS is 2^10
constexpr uint64_t kIdMask = (1 << kIdBits) - 1;
constexpr double kNoKey = -__builtin_inf();

// c (finite) as far as it counts: what is equal but for the rounding of sums is equal then.
__device__ __forceinline__ uint64_t rounded(double c)
{
    return (__builtin_bit_cast(uint64_t, c + 0.0) + (kIdMask + 1) / 2) & ~kIdMask;       // -0 is 0
}

// A number that orders experts by c and then by lowest number.  Of a negative c the larger last bits
// are the smaller number.
__device__ __forceinline__ double expert_key(double c, int e)
{
    const uint64_t u = rounded(c);
    return __builtin_bit_cast(double, u | (u >> 63 ? uint64_t(e) : kIdMask - uint64_t(e)));
}

__device__ __forceinline__ int key_expert(double key)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    const int last = static_cast<int>(u & kIdMask);
    return u >> 63 ? last : static_cast<int>(kIdMask) - last;
}

__device__ __forceinline__ double max_of(double a, double b) { return a > b ? a : b; }

template <int WIDTH, int D = 1>
__device__ __forceinline__ double lanes_max_key(double v)
{
    if constexpr (D < WIDTH) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        uint32_t a0, b0, a1, b1;
        across<D>(static_cast<uint32_t>(u), a0, b0);
        across<D>(static_cast<uint32_t>(u >> 32), a1, b1);
        return lanes_max_key<WIDTH, 2 * D>(max_of(__builtin_bit_cast(double, uint64_t(a1) << 32 | a0),
                                                  __builtin_bit_cast(double, uint64_t(b1) << 32 | b0)));
    }
    return v;
}

// A bound that no c reaches, so that a key has ten bits to spare of any.
constexpr double kMost = 1e300;

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr double kTiny = 1e-20;

// What a workgroup leaves of its tokens: experts + 1 sums of shares (the last: of squared lse), then as
// many counts (the last: tokens routed).
struct RouteSums {
    double* share;
    int32_t* load;
    int groups;         // workgroups
};

// One wave per token, P experts a lane (expert lane + 64 i).
template <int DT, int P, bool SIGMOID>
__global__ __launch_bounds__(kRouteThreads) void k_route(RouteArgs a, RouteSums w)
{
    using T = typename Fmt<DT>::T;
    __shared__ double sum[kRouteWaves][MP_ROUTE_MAX_GROUPS];
    __shared__ double c_of[kRouteWaves][P * kWave];
    __shared__ int32_t count[P * kWave];
    __shared__ double square[kRouteWaves];
    __shared__ int32_t routed[kRouteWaves];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int n = a.x.vocab;
    const int width = n / a.groups;
    const bool sums = w.share != nullptr;
    double total[P] = {};
    double squares = 0.0;
    int tokens = 0;
    float bias[P] = {};
    if (sums) {
        for (int e = threadIdx.x; e < P * kWave; e += kRouteThreads) count[e] = 0;
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (a.bias != nullptr && lane + i * kWave < n) bias[i] = a.bias[lane + i * kWave];
    for (int64_t row = int64_t(blockIdx.x) * kRouteWaves + wave; row < a.x.rows;
         row += int64_t(gridDim.x) * kRouteWaves) {
        const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
        float* weights = a.weights + row * a.top;
        int64_t* ids = a.ids + row * a.top;
        if (a.mask != nullptr && a.mask[row] == 0) {
            if (lane < a.top) {
                weights[lane] = 0.0f;
                ids[lane] = -1;
            }
            continue;
        }
        float z[P];
        bool bad = false;
        float m = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = lane + i * kWave;
            z[i] = e < n ? widen<DT>(x[e]) : -__builtin_inff();
            bad |= z[i] != z[i] || (!SIGMOID && z[i] == __builtin_inff());
            m = __builtin_fmaxf(m, z[i]);
        }
        m = lanes_max<kWave>(m);
        double s[P];
        double all = 0.0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            // -inf: no expert there, a share of 0
            s[i] = z[i] == -__builtin_inff() ? 0.0 : SIGMOID ? sigmoid_of(z[i]) : share_to(z[i], m);
            all += s[i];
        }
        all = lanes_sum<kWave>(all);
        if (__builtin_amdgcn_ballot_w64(bad) != 0 || (!SIGMOID && !(all > 0.0))) {
            if (lane < a.top) {                      // no distribution
                weights[lane] = __builtin_nanf("");
                ids[lane] = -1;
            }
            continue;
        }
        const double part = all > 0.0 ? 1.0 / all : 0.0;
        double key[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (!SIGMOID) s[i] *= part;
            double c = s[i] + static_cast<double>(bias[i]);
            const bool in = z[i] > -__builtin_inff() && c > -__builtin_inf();
            c = __builtin_fmin(c, kMost);
            key[i] = in ? expert_key(c, lane + i * kWave) : kNoKey;
            if (a.groups > 1) c_of[wave][lane + i * kWave] = in ? c : -__builtin_inf();
        }
        if (a.groups > 1) {
            // a wave's accesses to its own shared memory are in order
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            double mine = -__builtin_inf();
            if (lane < a.groups) {
                double first = -__builtin_inf(), second = -__builtin_inf();
                for (int i = 0; i < width; ++i) {
                    const double c = c_of[wave][lane * width + i];
                    second = max_of(second, c < first ? c : first);
                    first = max_of(first, c);
                }
                if (first > -__builtin_inf())
                    mine = __builtin_bit_cast(
                        double, rounded(first + (a.group_best == 2 && second > -__builtin_inf() ? second : 0.0)));
                sum[wave][lane] = mine;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            int before = 0;
            if (lane < a.groups)
                for (int g = 0; g < a.groups; ++g) {
                    const double o = sum[wave][g];
                    before += o > mine || (o == mine && g < lane);
                }
            const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && before < a.top_groups);
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (!(kept >> ((lane + i * kWave) / width % 64) & 1)) key[i] = kNoKey;
        }
        double chosen = kNoKey;          // lane i: the i-th expert
        for (int i = 0; i < a.top; ++i) {
            double best = key[0];
#pragma unroll
            for (int j = 1; j < P; ++j) best = max_of(best, key[j]);
            best = lanes_max_key<kWave>(best);
            if (lane == i) chosen = best;
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (key[j] == best) key[j] = kNoKey;
        }
        const bool there = chosen > kNoKey;
        const int e = there ? key_expert(chosen) : 0;
        double ws = 0.0;
        if (there) {
            const float ze = widen<DT>(x[e]);
            ws = SIGMOID ? sigmoid_of(ze) : share_to(ze, m) * part;
        }
        const double d = lanes_sum<kWave>(ws) + kTiny;
        if (lane < a.top) {
            weights[lane] = static_cast<float>((a.renormalise ? ws / d : ws) * static_cast<double>(a.scale));
            ids[lane] = there ? e : -1;
            if (sums && there) atomicAdd(&count[e], 1);
        }
        if (sums && __builtin_amdgcn_ballot_w64(there) != 0) {
            ++tokens;
#pragma unroll
            for (int i = 0; i < P; ++i) total[i] += SIGMOID ? s[i] * part : s[i];
            if (!SIGMOID) {
                const double lse = static_cast<double>(m) + log_sum(all);
                squares += lse * lse;
            }
        }
    }
    if (!sums) return;
#pragma unroll
    for (int i = 0; i < P; ++i) c_of[wave][lane + i * kWave] = total[i];
    if (lane == 0) {
        square[wave] = squares;
        routed[wave] = tokens;
    }
    __syncthreads();
    double* share = w.share + int64_t(blockIdx.x) * (n + 1);
    int32_t* load = w.load + int64_t(blockIdx.x) * (n + 1);
    for (int e = threadIdx.x; e <= n; e += kRouteThreads) {
        double s = 0.0;
        int32_t c = e < n ? count[e] : 0;
#pragma unroll
        for (int i = 0; i < kRouteWaves; ++i) {
            s += e < n ? c_of[i][e] : square[i];
            if (e == n) c += routed[i];
        }
        share[e] = s;
        load[e] = c;
    }
}

// The workgroups' sums joined in a fixed order, 8 experts a workgroup.
constexpr int kFinishThreads = 256;
constexpr int kFinishExperts = 8;

__global__ __launch_bounds__(kFinishThreads) void k_route_finish(RouteArgs a, RouteSums w)
{
    constexpr int SLICES = kFinishThreads / kFinishExperts;
    __shared__ double s_part[SLICES][kFinishExperts];
    __shared__ int64_t c_part[SLICES][kFinishExperts];
    __shared__ int64_t n_part[SLICES][kFinishExperts];
    const int n = a.x.vocab;
    const int col = threadIdx.x % kFinishExperts, slice = threadIdx.x / kFinishExperts;
    const int e = static_cast<int>(blockIdx.x) * kFinishExperts + col;
    double s = 0.0;
    int64_t c = 0, t = 0;
    for (int g = slice; g < w.groups; g += SLICES) {
        if (e <= n) {
            s += w.share[int64_t(g) * (n + 1) + e];
            c += w.load[int64_t(g) * (n + 1) + e];
        }
        t += w.load[int64_t(g) * (n + 1) + n];
    }
    s_part[slice][col] = s;
    c_part[slice][col] = c;
    n_part[slice][col] = t;
    __syncthreads();
    if (slice != 0 || e > n) return;
    s = 0.0;
    c = t = 0;
    for (int i = 0; i < SLICES; ++i) {
        s += s_part[i][col];
        c += c_part[i][col];
        t += n_part[i][col];
    }
    a.load[e] = c;
    const double mean = t > 0 ? s / static_cast<double>(t) : 0.0;
    if (e < n && a.share != nullptr) a.share[e] = static_cast<float>(mean);
    if (e == n && a.aux != nullptr) a.aux[1] = static_cast<float>(mean);
}

__global__ __launch_bounds__(kFinishThreads) void k_route_aux(RouteArgs a)
{
    __shared__ double part[kFinishThreads / kWave];
    const int n = a.x.vocab;
    double s = 0.0;
    for (int e = threadIdx.x; e < n; e += kFinishThreads)
        s += static_cast<double>(a.load[e]) * static_cast<double>(a.share[e]);
    s = lanes_sum<kWave>(s);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = s;
    __syncthreads();
    if (threadIdx.x != 0) return;
    s = 0.0;
    for (int i = 0; i < kFinishThreads / kWave; ++i) s += part[i];
    const double tokens = static_cast<double>(a.load[n]);
    a.aux[0] = tokens > 0.0 ? static_cast<float>(s * n / (a.top * tokens)) : 0.0f;
}

// One wave per token.  With F the factor over the tokens routed, pull_e = F balance E load_e / (k N)
// and ds the gradient of the chosen experts' scores,
//   softmax  dx_e = s_e (pull_e + ds_e - sum_j s_j (pull_j + ds_j) + 2 F z lse)
//   sigmoid  dx_e = s_e (1 - s_e) ((pull_e - sum_j p_j pull_j) / sum s + ds_e),    p = s / sum s.
template <int DT, int P, bool SIGMOID>
__global__ __launch_bounds__(kRouteThreads) void k_route_grad(RouteGradArgs a)
{
    using T = typename Fmt<DT>::T;
    __shared__ float extra[kRouteWaves][P * kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int n = a.x.vocab;
    double factor = 0.0;
    float pull[P] = {};
    if (a.load != nullptr) {
        const int64_t tokens = read_table(a.load + n);
        factor = tokens > 0 ? grad_factor(a.g) / static_cast<double>(tokens) : 0.0;
        const double unit = factor * static_cast<double>(a.balance) * n / a.top /
                            static_cast<double>(tokens > 0 ? tokens : 1);
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (lane + i * kWave < n)
                pull[i] = static_cast<float>(unit * static_cast<double>(a.load[lane + i * kWave]));
    }
    const double large = 2.0 * factor * static_cast<double>(a.large);
    for (int64_t row = int64_t(blockIdx.x) * kRouteWaves + wave; row < a.x.rows;
         row += int64_t(gridDim.x) * kRouteWaves) {
        const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
        T* dx = static_cast<T*>(a.g.dx) + row * a.g.stride;
        float z[P];
        const bool live = a.mask == nullptr || a.mask[row] != 0;
        bool bad = false;
        float m = -FLT_MAX;
        if (live) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int e = lane + i * kWave;
                z[i] = e < n ? widen<DT>(x[e]) : -__builtin_inff();
                bad |= z[i] != z[i] || (!SIGMOID && z[i] == __builtin_inff());
                m = __builtin_fmaxf(m, z[i]);
            }
        }
        int64_t id = -1;
        float dw = 0.0f;
        if (live && lane < a.top) {
            id = a.ids[row * a.top + lane];
            if (a.dweights != nullptr && id >= 0)
                dw = a.dweights[row * a.top + lane] * a.scale;
        }
        const bool past = id >= n;
        if (past) id = -1;
        m = lanes_max<kWave>(m);
        float s[P], slope[P];            // slope: ds_e / dx_e of a sigmoid
        double all = 0.0;
        if (live) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (SIGMOID) {
                    const float u = exp2_hw(-__builtin_fabsf(z[i]) * static_cast<float>(kLog2E));
                    const float r = 1.0f / (1.0f + u);
                    s[i] = z[i] >= 0.0f ? r : u * r;
                    slope[i] = u * r * r;
                } else {
                    s[i] = exp2_hw((z[i] - m) * static_cast<float>(kLog2E));
                }
                all += static_cast<double>(s[i]);
            }
        }
        all = lanes_sum<kWave>(all);
        const bool nan = __builtin_amdgcn_ballot_w64(bad || past) != 0 || (live && !SIGMOID && !(all > 0.0));
        const bool any = __builtin_amdgcn_ballot_w64(id >= 0) != 0;
        if (!live || nan || !any) {
            const float v = live && nan ? __builtin_nanf("") : 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (lane + i * kWave < n) store_one<DT>(dx + lane + i * kWave, v);
            continue;
        }
        const float part = all > 0.0 ? static_cast<float>(1.0 / all) : 0.0f;
        // the chosen experts' scores and their gradient
        float ws = 0.0f;
        if (id >= 0) {
            const float ze = widen<DT>(x[id]);
            if (SIGMOID) {
                const float u = exp2_hw(-__builtin_fabsf(ze) * static_cast<float>(kLog2E));
                ws = (ze >= 0.0f ? 1.0f : u) / (1.0f + u);
            } else {
                ws = exp2_hw((ze - m) * static_cast<float>(kLog2E)) * part;
            }
        }
        double ds = static_cast<double>(dw);
        if (a.renormalise) {
            const double d = lanes_sum<kWave>(static_cast<double>(ws)) + kTiny;
            const double mean = lanes_sum<kWave>(static_cast<double>(dw) * static_cast<double>(ws)) / d;
            ds = id >= 0 ? (static_cast<double>(dw) - mean) / d : 0.0;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) extra[wave][lane + i * kWave] = 0.0f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // the same expert twice: its parts add up, in the list's order
        double same = 0.0;
        for (int i = 0; i < a.top; ++i) {
            const int64_t other = __shfl(id, i);
            const double part_of = __shfl(ds, i);
            if (other == id) same += part_of;
        }
        if (id >= 0) extra[wave][id] = static_cast<float>(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        double dot = 0.0;
        float to[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            to[i] = extra[wave][lane + i * kWave];
            if (!SIGMOID) {
                s[i] *= part;
                to[i] += pull[i];
                dot += static_cast<double>(s[i]) * static_cast<double>(to[i]);
            } else {
                dot += static_cast<double>(s[i]) * static_cast<double>(pull[i]);
            }
        }
        dot = lanes_sum<kWave>(dot);
        float base;
        if (SIGMOID) base = all > 0.0 ? static_cast<float>(dot / all) : 0.0f;
        else base = static_cast<float>(large * (static_cast<double>(m) + log_sum(all)) - dot);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = lane + i * kWave;
            const float v = SIGMOID ? slope[i] * ((pull[i] - base) * part + to[i]) : s[i] * (to[i] + base);
            if (e < n) store_one<DT>(dx + e, v);
        }
    }
}

// out = bias + speed sign(mean load - load), one workgroup a layer; a skipped step leaves the bias.
__global__ __launch_bounds__(kFinishThreads) void k_route_bias(RouteBiasArgs a)
{
    __shared__ int64_t part[kFinishThreads / kWave];
    const int64_t layer = blockIdx.x;
    const int n = a.experts;
    const bool skip = a.skipped != nullptr && *a.skipped != 0;
    auto load_of = [&](int e) {
        int64_t c = 0;
        for (int i = 0; i < a.n_loads; ++i) c += a.load[(int64_t(i) * a.layers + layer) * (n + 1) + e];
        return c;
    };
    int64_t all = 0;
    for (int e = threadIdx.x; e < n; e += kFinishThreads) all += load_of(e);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) all += __shfl_xor(all, d);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = all;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int i = 0; i < kFinishThreads / kWave; ++i) all += part[i];
    for (int e = threadIdx.x; e < n; e += kFinishThreads) {
        const int64_t off = all - load_of(e) * n;
        const float step = skip || off == 0 ? 0.0f : off > 0 ? a.speed : -a.speed;
        a.out[layer * n + e] = a.bias[layer * n + e] + step;
    }
}

template <int DT, int P>
void route_p(const RouteArgs& a, const RouteSums& w, unsigned grid, hipStream_t s)
{
    if (a.sigmoid) k_route<DT, P, true><<<grid, kRouteThreads, 0, s>>>(a, w);
    else k_route<DT, P, false><<<grid, kRouteThreads, 0, s>>>(a, w);
}

template <int DT>
void route_dt(const RouteArgs& a, const RouteSums& w, unsigned grid, hipStream_t s)
{
    if (a.x.vocab <= 64) route_p<DT, 1>(a, w, grid, s);
    else if (a.x.vocab <= 256) route_p<DT, 4>(a, w, grid, s);
    else route_p<DT, 16>(a, w, grid, s);
}

template <int DT, int P>
void grad_p(const RouteGradArgs& a, unsigned grid, hipStream_t s)
{
    if (a.sigmoid) k_route_grad<DT, P, true><<<grid, kRouteThreads, 0, s>>>(a);
    else k_route_grad<DT, P, false><<<grid, kRouteThreads, 0, s>>>(a);
}

template <int DT>
void grad_dt(const RouteGradArgs& a, unsigned grid, hipStream_t s)
{
    if (a.x.vocab <= 64) grad_p<DT, 1>(a, grid, s);
    else if (a.x.vocab <= 256) grad_p<DT, 4>(a, grid, s);
    else grad_p<DT, 16>(a, grid, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s)
{
    const int64_t per = 12 * (int64_t(a.x.vocab) + 1);
    int64_t most = a.load != nullptr ? MP_ROUTE_WORKSPACE_BYTES / per : 1 << 16;
    if (a.load != nullptr && most > 1024) most = 1024;
    int64_t grid = (int64_t(a.x.rows) + kRouteWaves - 1) / kRouteWaves;
    if (grid > most) grid = most;
    RouteSums w{};
    if (a.load != nullptr) {
        w.groups = static_cast<int>(grid);
        w.share = static_cast<double*>(a.workspace);
        w.load = reinterpret_cast<int32_t*>(w.share + grid * (a.x.vocab + 1));
    }
    if (grid > 0) {
        const unsigned g = static_cast<unsigned>(grid);
        if (dtype == kBF16) route_dt<kBF16>(a, w, g, s);
        else if (dtype == kFP16) route_dt<kFP16>(a, w, g, s);
        else route_dt<kFP32>(a, w, g, s);
    }
    if (a.load != nullptr) {
        const unsigned cols = (static_cast<unsigned>(a.x.vocab) + kFinishExperts) / kFinishExperts;
        k_route_finish<<<cols, kFinishThreads, 0, s>>>(a, w);
        if (a.aux != nullptr) k_route_aux<<<1, kFinishThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, int dtype, hipStream_t s)
{
    int64_t grid = (int64_t(a.x.rows) + kRouteWaves - 1) / kRouteWaves;
    if (grid > 4096) grid = 4096;
    const unsigned g = static_cast<unsigned>(grid);
    if (dtype == kBF16) grad_dt<kBF16>(a, g, s);
    else if (dtype == kFP16) grad_dt<kFP16>(a, g, s);
    else grad_dt<kFP32>(a, g, s);
    return hipGetLastError();
}

hipError_t launch_route_bias(const RouteBiasArgs& a, hipStream_t s)
{
    k_route_bias<<<static_cast<unsigned>(a.layers), kFinishThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace mpk
