// HIP kernels of the scores of logits: log-probability, entropy and the likeliest
// entries of a row, and the gradient of the first two.
//
// With k = log2(e) / T as the nearest float kf plus a rest and a lane's reference
// R = fl(m kf), m its maximum, one fma gives y_j = x_j kf - R, and a lane sums
//   s = sum_j 2^y_j,   c = sum_j y_j 2^y_j,
// both rescaled when m grows.  R's rounding and kf's are the same for all of a row's
// elements, so they drop out of the shares q_j but for a factor near 1 of known
// logarithm: with d = R - m kf,
//   log2 S = log2 s + d + (rest / kf) (c / s + d)     (S = sum_j 2^((x_j - m) k)),
//   lse = m / T + ln S,   lp = (x_t - m) / T - ln S,   H = ln S - (c / s + d) / (kf T).
// That saves two operations a logit against differences x_j - m; a row whose largest
// logit reaches 2^24 / kf, where R's steps are no longer small, is summed again from
// differences.
#include <float.h>

#include "rows.h"
#include "scores.h"

namespace mpk {
namespace {

struct RowScale {
    float k;               // the float nearest to log2(e) / T
    double rest;           // log2(e) / T - k
    double inv_t;
};

__device__ __forceinline__ RowScale scale_of(const LogitsView& x)
{
    const double whole = static_cast<double>(x.k_hi) + static_cast<double>(x.k_lo);
    RowScale r;
    r.k = static_cast<float>(whole);
    r.rest = whole - static_cast<double>(r.k);
    r.inv_t = x.inv_t;
    return r;
}

constexpr float kRefMost = 0x1p26f;      // a lane's reference; a row's is below 2^24 or not used
constexpr float kRowMost = 0x1p24f;
constexpr float kGone = -200.0f;         // an exponent whose power of two is 0

// A lane's sums.  m starts at the lowest finite value: -inf never enters a difference.
struct Share {
    float m = -FLT_MAX;
    float ref = 0.0f;
    float s = 0.0f, c = 0.0f;
};

template <int N>
__device__ __forceinline__ void add(Share& a, const float (&f)[N], float k)
{
    float g = a.m;
#pragma unroll
    for (int i = 0; i < N; ++i) g = __builtin_fmaxf(g, f[i]);
    if (g > a.m) {
        // an unlikely row's references may be limited; none is infinite, so nothing here is NaN
        const float r = __builtin_amdgcn_fmed3f(g * k, -kRefMost, kRefMost);
        const float d = __builtin_amdgcn_fmed3f(a.ref - r, kGone, 0.0f);
        const float down = exp2_hw(d);
        a.c = __builtin_fmaf(a.s, d, a.c) * down;
        a.s *= down;
        a.ref = r;
        a.m = g;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = __builtin_fmaf(f[i], k, -a.ref);
        const float e = exp2_hw(y);                    // NaN stays NaN
        a.s += e;
        a.c = __builtin_fmaf(e, __builtin_fmaxf(y, kGone), a.c);      // 0, not 0 * -inf
    }
}

// The same from differences to the row's maximum.
template <int N>
__device__ __forceinline__ void add_to(Share& a, const float (&f)[N], float k)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = (f[i] - a.m) * k;
        const float e = exp2_hw(y);
        a.s += e;
        a.c = __builtin_fmaf(e, __builtin_fmaxf(y, kGone), a.c);
    }
}

// A row's statistics, in all lanes.
struct RowStat {
    float m;
    double ln_s;          // of the sum relative to m
    double lse, entropy;
};

// Sums relative to the largest reference among groups of WIDTH lanes.
template <int WIDTH>
__device__ __forceinline__ void join_lanes(float& m, float& ref, double& s, double& c)
{
    m = lanes_max<WIDTH>(m);
    const float own = ref;
    ref = lanes_max<WIDTH>(own);
    const float d = own - ref;
    const double down = static_cast<double>(exp2_hw(d));
    c = lanes_sum<WIDTH>((c + s * static_cast<double>(d)) * down);
    s = lanes_sum<WIDTH>(s * down);
}

template <int THREADS>
struct JoinSpace {
    float m[THREADS / kWave], ref[THREADS / kWave];
    double s[THREADS / kWave], c[THREADS / kWave];
};

// All lanes' shares, valid in all lanes.
template <int THREADS>
__device__ __forceinline__ void join(const Share& a, JoinSpace<THREADS>& l, float& m, float& ref, double& s,
                                     double& c)
{
    constexpr int W = THREADS / kWave;
    m = a.m;
    // a lane without any element in reach has no say in the reference
    ref = a.s != 0.0f ? a.ref : -kRefMost;
    s = static_cast<double>(a.s);
    c = static_cast<double>(a.c);
    join_lanes<kWave>(m, ref, s, c);
    if constexpr (W > 1) {
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        __syncthreads();                  // the space may still be read from an earlier join
        if (lane == 0) {
            l.m[wave] = m;
            l.ref[wave] = ref;
            l.s[wave] = s;
            l.c[wave] = c;
        }
        __syncthreads();
        m = l.m[lane % W];
        ref = l.ref[lane % W];
        s = l.s[lane % W];
        c = l.c[lane % W];
        join_lanes<W>(m, ref, s, c);
    }
}

__device__ __forceinline__ RowStat stat_of(float m, double ref, double s, double c, const RowScale& k)
{
    const double kf = static_cast<double>(k.k);
    const double d = ref - static_cast<double>(m) * kf;
    const double mean = c / s + d;                             // of (x - m) kf
    RowStat r;
    r.m = m;
    r.ln_s = log_sum(s) + 0.69314718055994531 * (d + k.rest / kf * mean);
    r.lse = static_cast<double>(m) * k.inv_t + r.ln_s;
    const double h = r.ln_s - mean * (k.inv_t / kf);
    r.entropy = h < 0.0 ? 0.0 : h;                             // NaN stays
    if (!(s > 0.0) || __builtin_isinf(s)) r.ln_s = r.lse = r.entropy = __builtin_nan("");
    return r;
}

// Entries in their order -- the larger logit first, of equal ones (-0 and 0) the lower id -- as whole
// numbers, the first the largest.  0 comes after every entry.
__device__ __forceinline__ uint64_t entry_key(float v, int id)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    const uint32_t up = u & 0x80000000u ? ~u : u | 0x80000000u;
    return uint64_t(up) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t up = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(up & 0x80000000u ? up & 0x7FFFFFFFu : ~up);
}

__device__ __forceinline__ int key_id(uint64_t key)
{
    return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}

// Calls f(value, id) for every element of a row, each in one lane.
template <int DT, int THREADS, class F>
__device__ __forceinline__ void each_element(const typename Fmt<DT>::T* x, const Span<DT>& sp, F f)
{
    constexpr int E = Fmt<DT>::E;
    for (int i = threadIdx.x; i < sp.nvec; i += THREADS) {
        const int at = sp.head + i * E;
        float v[E];
        unpack<DT>(load_vec<DT, false>(x + at), v);
#pragma unroll
        for (int j = 0; j < E; ++j) f(v[j], at + j);
    }
    const int one = sp.single(threadIdx.x);
    if (one >= 0) f(widen<DT>(x[one]), one);
}

template <int THREADS>
__device__ __forceinline__ uint64_t block_max(uint64_t v)
{
    __shared__ uint64_t part[THREADS / kWave];
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint64_t o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    __syncthreads();
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < THREADS / kWave; ++i) v = part[i] > v ? part[i] : v;
    return v;
}

__device__ __forceinline__ void write_entry(const ScoreArgs& a, int64_t at, uint64_t key, const RowStat& r)
{
    const bool there = key != 0;
    const float v = there ? key_value(key) : -__builtin_inff();
    a.top_ids[at] = there ? key_id(key) : -1;
    if (a.top_values != nullptr) a.top_values[at] = v;
    if (a.top_logp != nullptr)
        a.top_logp[at] =
            there ? static_cast<float>((static_cast<double>(v) - static_cast<double>(r.m)) * a.x.inv_t - r.ln_s) : v;
}

__device__ __forceinline__ void write_row(const ScoreArgs& a, int64_t row, int64_t target, float xt,
                                          const RowStat& r)
{
    if (a.lse != nullptr) a.lse[row] = static_cast<float>(r.lse);
    if (a.entropy != nullptr) a.entropy[row] = static_cast<float>(r.entropy);
    if (a.logp != nullptr)
        a.logp[row] =
            target >= a.x.vocab
                ? __builtin_nanf("")
                : static_cast<float>((static_cast<double>(xt) - static_cast<double>(r.m)) * a.x.inv_t - r.ln_s);
}

// A switched-off row: nothing of it is read.
__device__ __forceinline__ void write_off(const ScoreArgs& a, int64_t row)
{
    if (threadIdx.x == 0) {
        if (a.logp != nullptr) a.logp[row] = 0.0f;
        if (a.lse != nullptr) a.lse[row] = 0.0f;
        if (a.entropy != nullptr) a.entropy[row] = 0.0f;
    }
    for (int e = threadIdx.x; e < a.top; e += blockDim.x) write_entry(a, row * a.top + e, 0, RowStat{});
}

// One row per workgroup, in one pass for the sums, then one for each entry.
template <int DT, int THREADS>
__global__ __launch_bounds__(THREADS) void k_scores(ScoreArgs a)
{
    using T = typename Fmt<DT>::T;
    __shared__ JoinSpace<THREADS> space;
    const int64_t row = blockIdx.x;
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    const int64_t target = a.targets != nullptr ? read_table(a.targets + row) : 0;
    if (target < 0) return write_off(a, row);
    const RowScale k = scale_of(a.x);
    const Span<DT> sp(x, n);
    Share share;
    each_element<DT, THREADS>(x, sp, [&](float v, int) {
        const float f[1] = {v};
        add(share, f, k.k);
    });
    float m, ref;
    double s, c;
    join<THREADS>(share, space, m, ref, s, c);
    double exact_ref = static_cast<double>(ref);
    if (!(__builtin_fabsf(m * k.k) < kRowMost)) {
        share = Share{};
        share.m = m;
        each_element<DT, THREADS>(x, sp, [&](float v, int) {
            const float f[1] = {v};
            add_to(share, f, k.k);
        });
        join<THREADS>(share, space, m, ref, s, c);
        exact_ref = static_cast<double>(m) * static_cast<double>(k.k);
    }
    const RowStat r = stat_of(m, exact_ref, s, c, k);
    if (threadIdx.x == 0) write_row(a, row, target, target < n ? widen<DT>(x[target]) : 0.0f, r);
    uint64_t last = ~uint64_t(0);
    for (int e = 0; e < a.top; ++e) {
        uint64_t best = 0;
        if (last != 0 && r.ln_s == r.ln_s)
            each_element<DT, THREADS>(x, sp, [&](float v, int id) {
                const uint64_t key = entry_key(v, id);
                if (v > -__builtin_inff() && key < last && key > best) best = key;
            });
        last = block_max<THREADS>(best);
        if (threadIdx.x == 0) write_entry(a, row * a.top + e, last, r);
    }
}

// The gradient of sum_r (g lp + h H): with y = log2 q = x k - lse log2(e) in two floats,
//   dx_j = f (g (1[j = t] - q_j) - h q_j (ln q_j + H)) = q_j (y_j (-h f ln 2) - f (g + h H)),
// the target's element apart, from expm1 of its log-probability, stored over the dense one by
// the lane that has its vector.  Two roundings of y as in the gradient of log-probabilities.
// Bound by HBM: 2 bytes read and written per 16-bit logit against about 10 VALU operations.
template <int DT>
__global__ __launch_bounds__(kGradThreads) void k_score_grad(ScoreGradArgs a, int chunks, int chunk_vecs)
{
    using T = typename Fmt<DT>::T;
    constexpr int E = Fmt<DT>::E;
    const unsigned block = xcd_chunk(blockIdx.x, gridDim.x);
    const int64_t row = block / static_cast<unsigned>(chunks);
    const int chunk = static_cast<int>(block % static_cast<unsigned>(chunks));
    const int tid = threadIdx.x;
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    T* dx = static_cast<T*>(a.g.dx) + row * a.g.stride;
    const Span<DT> sp(dx, n);
    const int lo = chunk * chunk_vecs;
    const int hi = min(lo + chunk_vecs, sp.nvec);
    const int one = chunk == 0 ? sp.single(tid) : -1;
    const int64_t target = a.targets != nullptr ? read_table(a.targets + row) : 0;
    const float dl = a.dlogp != nullptr ? read_table(a.dlogp + row) : 0.0f;
    const float dh = a.dentropy != nullptr ? read_table(a.dentropy + row) : 0.0f;
    if (target < 0 || (dl == 0.0f && dh == 0.0f)) {
        const u32x4 z = {0u, 0u, 0u, 0u};
        for (int i = lo + tid; i < hi; i += kGradThreads) store_vec<DT>(dx + sp.head + int64_t(i) * E, z);
        if (one >= 0) store_one<DT>(dx + one, 0.0f);
        return;
    }
    const double factor = grad_factor(a.g);
    const double g = factor * static_cast<double>(dl), h = factor * static_cast<double>(dh);
    const double lse = static_cast<double>(read_table(a.lse + row));
    const double entropy = dh != 0.0f ? static_cast<double>(read_table(a.entropy + row)) : 0.0;
    const float slope = static_cast<float>(h * -0.69314718055994531);
    const float rest = target < n ? static_cast<float>(-(g + h * entropy)) : __builtin_nanf("");
    const double l2 = lse * 1.4426950408889634;
    const float l_hi = static_cast<float>(l2);
    const float l_lo = __builtin_isinf(l_hi) ? 0.0f : static_cast<float>(l2 - static_cast<double>(l_hi));
    const float k_hi = a.x.k_hi, k_lo = a.x.k_lo;
    auto one_of = [&](float f) {
        float y = __builtin_fmaf(f, k_hi, -l_hi);
        if constexpr (DT == kFP32) y += __builtin_fmaf(f, k_lo, -l_lo);
        // no probability: 0 and not 0 * -inf
        return exp2_hw(y) * __builtin_fmaf(__builtin_fmaxf(y, kGone), slope, rest);
    };
    const int te = a.dlogp != nullptr && target < n ? static_cast<int>(target) : -1;
    bool mine = false;
    float xt = 0.0f;
    if (te >= 0) {
        const int tv = te < sp.head ? -1 : (te - sp.head) / E;
        mine = tv >= 0 && tv < sp.nvec ? (tv >= lo && tv < hi && (tv - lo) % kGradThreads == tid)
                                       : one == te;
        if (mine) xt = widen<DT>(x[te]);
    }
    const float single = one >= 0 ? widen<DT>(x[one]) : 0.0f;
    auto vec = [&](u32x4 raw, int i) {
        float f[E];
        unpack<DT>(raw, f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = one_of(f[j]);
        store_vec<DT>(dx + sp.head + int64_t(i) * E, pack<DT>(f));
    };
    if (a.x.stream) {
        for (int i = lo + tid; i < hi; i += kGradThreads)
            vec(load_vec<DT, true>(x + sp.head + int64_t(i) * E), i);
    } else {
        for (int i = lo + tid; i < hi; i += kGradThreads)
            vec(load_vec<DT, false>(x + sp.head + int64_t(i) * E), i);
    }
    if (one >= 0) store_one<DT>(dx + one, one_of(single));
    if (mine) {
        const double lp = static_cast<double>(xt) * a.x.inv_t - lse;
        const double q = exp_of(lp);
        const double bonus = dh != 0.0f && q > 0.0 ? h * q * (lp + entropy) : 0.0;
        store_one<DT>(dx + te, static_cast<float>(-g * expm1_of(lp) - bonus));
    }
}

template <int DT>
void scores_dt(const ScoreArgs& a, hipStream_t s)
{
    k_scores<DT, 256><<<static_cast<unsigned>(a.x.rows), 256, 0, s>>>(a);
}

template <int DT>
void score_grad_dt(ScoreGradArgs a, hipStream_t s)
{
    // read past the cache, cut into chunks and dealt to the XCDs as the gradient of
    // log-probabilities: the same bytes in the same order
    a.x.stream = logits_bytes<DT>(a.x) > kCacheBytes / 2;
    const int nvec = a.x.vocab / Fmt<DT>::E + 1;
    int per = 2 * kGradThreads;
    while (static_cast<int64_t>((nvec + per - 1) / per) * a.x.rows > (int64_t(1) << 23)) per *= 2;
    const int chunks = (nvec + per - 1) / per;
    k_score_grad<DT><<<static_cast<unsigned>(chunks) * static_cast<unsigned>(a.x.rows), kGradThreads, 0, s>>>(
        a, chunks, per);
}

}  // namespace

hipError_t launch_scores(const ScoreArgs& a, int dtype, hipStream_t s)
{
    if (dtype == kBF16) scores_dt<kBF16>(a, s);
    else if (dtype == kFP16) scores_dt<kFP16>(a, s);
    else scores_dt<kFP32>(a, s);
    return hipGetLastError();
}

hipError_t launch_score_grad(const ScoreGradArgs& a, int dtype, hipStream_t s)
{
    if (dtype == kBF16) score_grad_dt<kBF16>(a, s);
    else if (dtype == kFP16) score_grad_dt<kFP16>(a, s);
    else score_grad_dt<kFP32>(a, s);
    return hipGetLastError();
}

}  // namespace mpk
