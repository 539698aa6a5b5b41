// HIP kernels of the scores of logits: log-probability, entropy and the likeliest
// entries of a row, and the gradient of the first two.
//
// With k = log2(e) / T as the nearest float kf plus a rest, and a lane's reference R near its
// largest logit's exponent, one fma gives y_j = x_j kf - R, and a lane sums
//   s = sum_j 2^y_j,   c = sum_j y_j 2^y_j.
// Both are scaled down, and R raised, only where a logit exceeds R by kSlack: the sums need not
// be relative to the maximum, but near it.  What R and kf are off is the same for all of a row's
// elements, so it drops out of the shares q_j but for a factor near 1 of known logarithm:
// with m the row's maximum and d = R - m kf,
//   log2 S = log2 s + d + (rest / kf) (c / s + d)     (S = sum_j 2^((x_j - m) k)),
//   lse = m / T + ln S,   lp = (x_t - m) / T - ln S,   H = ln S - (c / s + d) / (kf T).
// That takes fewer operations a logit than differences x_j - m do; a row whose largest
// logit reaches 2^24 / kf, where R's steps are no longer small, is summed again from
// differences.
//
// The passes are bound by HBM and the vector units alike: 6.5 TB/s of 16-bit logits leave 12 lane
// operations a logit, and its exponential counts for four of them.
#include <float.h>

#include <algorithm>

#include "rows.h"
#include "scores.h"

namespace mpk {
namespace {

constexpr float kSlack = 8.0f;           // of an exponent over its reference

struct RowScale {
    float k;               // the float nearest to log2(e) / T
    float slack;           // kSlack of an exponent as a difference of logits
    double rest;           // log2(e) / T - k
    double inv_t;
};

__device__ __forceinline__ RowScale scale_of(const LogitsView& x)
{
    const double whole = static_cast<double>(x.k_hi) + static_cast<double>(x.k_lo);
    RowScale r;
    r.k = static_cast<float>(whole);
    r.slack = static_cast<float>(static_cast<double>(kSlack) / whole);
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
    float most = -FLT_MAX;               // the logit that raises the reference
    float ref = 0.0f;
    float s = 0.0f, c = 0.0f;
};

// The reference raised where a maximum g asks for it.
__device__ __forceinline__ void raise(Share& a, float g, float k, float slack)
{
    a.m = __builtin_fmaxf(a.m, g);
    if (g > a.most) {
        // an unlikely row's references may be limited; none is infinite, so nothing here is NaN
        const float r = __builtin_amdgcn_fmed3f(g * k, -kRefMost, kRefMost);
        const float d = __builtin_amdgcn_fmed3f(a.ref - r, kGone, 0.0f);
        const float down = exp2_hw(d);
        a.c = __builtin_fmaf(a.s, d, a.c) * down;
        a.s *= down;
        a.ref = r;
        a.most = g + slack;
    }
}

template <int N>
__device__ __forceinline__ void add_shares(Share& a, const float (&f)[N], float k)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = __builtin_fmaf(f[i], k, -a.ref);
        const float e = exp2_hw(y);                    // NaN stays NaN
        a.s += e;
        a.c = __builtin_fmaf(e, y, a.c);
    }
}

// c again where it met 0 * -inf, of a mask or of an overflow downwards: these add 0.
template <int N>
__device__ __forceinline__ float add_masked(const Share& a, float c, const float (&f)[N], float k)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = __builtin_fmaf(f[i], k, -a.ref);
        c = __builtin_fmaf(exp2_hw(y), __builtin_fmaxf(y, kGone), c);
    }
    return c;
}

__device__ __forceinline__ void add_one(Share& a, float f, float k, float slack)
{
    const float one[1] = {f};
    raise(a, f, k, slack);
    const float before = a.c;
    add_shares(a, one, k);
    if (a.c != a.c) a.c = add_masked(a, before, one, k);
}

// The largest of two vectors' elements.  fp16 ones are compared two at a time: the sums then take
// them as they are (v_fma_mix_f32), and none is widened.
template <int DT>
__device__ __forceinline__ float max_of(u32x4 a, u32x4 b)
{
    if constexpr (DT == kFP16) {
        f16x2 h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = a[i], v = b[i];
            h[i] = __builtin_bit_cast(f16x2, u);
            h[4 + i] = __builtin_bit_cast(f16x2, v);
        }
#pragma unroll
        for (int i = 1; i < 8; ++i) h[0] = __builtin_elementwise_max(h[0], h[i]);
        return __builtin_fmaxf(static_cast<float>(h[0].x), static_cast<float>(h[0].y));
    } else {
        constexpr int E = Fmt<DT>::E;
        float f[E], g[E];
        unpack<DT>(a, f);
        unpack<DT>(b, g);
        float m = __builtin_fmaxf(f[0], g[0]);
#pragma unroll
        for (int i = 1; i < E; ++i) m = __builtin_fmaxf(__builtin_fmaxf(m, f[i]), g[i]);
        return m;
    }
}

// Two vectors; returns their maximum.
template <int DT>
__device__ __forceinline__ float add_pair(Share& s, u32x4 a, u32x4 b, const RowScale& k)
{
    constexpr int E = Fmt<DT>::E;
    const float g = max_of<DT>(a, b);
    raise(s, g, k.k, k.slack);
    const float before = s.c;
    float f[E];
    unpack<DT>(a, f);
    add_shares(s, f, k.k);
    unpack<DT>(b, f);
    add_shares(s, f, k.k);
    if (s.c != s.c) {
        asm volatile("" : "+v"(a), "+v"(b));           // unpacked again, not kept for this
        unpack<DT>(a, f);
        s.c = add_masked(s, before, f, k.k);
        unpack<DT>(b, f);
        s.c = add_masked(s, s.c, f, k.k);
    }
    return g;
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

// A row's statistics.
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

// All lanes' shares joined: m valid in all lanes, the sums in the first wave's.
template <int THREADS>
__device__ __forceinline__ void join(const Share& a, float k, JoinSpace<THREADS>& l, float& m, float& ref, double& s,
                                     double& c)
{
    constexpr int W = THREADS / kWave;
    m = a.m;
    // a lane without any element in reach has no say in the reference
    ref = a.s != 0.0f ? a.ref : -kRefMost;
    s = static_cast<double>(a.s);
    c = static_cast<double>(a.c);
    // A reference is its logit's exponent rounded to fp32, and the logit counts as 2^y with y that rounding: what the
    // exponential's own rounding near 1 adds, 2^-24 or so, may be all of a confident row's entropy.  Put right here, of
    // the lane's largest logit (2^y to 1e-14).  Where a lane's reference is another's, that one has at least 2^-kSlack
    // of the largest's share, and the entropy is large beside it.
    const float y = __builtin_fmaf(a.m, k, -a.ref);
    if (__builtin_fabsf(y) < 0x1p-10f) {
        const double t = static_cast<double>(y) * 0.69314718055994531;
        const double off = 1.0 + t * (1.0 + t * (0.5 + t * (1.0 / 6.0))) - static_cast<double>(exp2_hw(y));
        s += off;
        c += off * static_cast<double>(y);
    }
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
        if (wave == 0) {
            ref = l.ref[lane % W];
            s = l.s[lane % W];
            c = l.c[lane % W];
            join_lanes<W>(m, ref, s, c);
        } else {
            m = lanes_max<W>(m);
        }
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

// Floats in their order as whole numbers, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Entries in their order -- the larger logit first, of equal ones the lower id (below 2^30) -- as whole
// numbers of 62 bits, the first the largest.  0 comes after every entry.
constexpr int kIdBits = 30;
constexpr uint32_t kIdMost = (1u << kIdBits) - 1;

__device__ __forceinline__ uint64_t entry_key(float v, int id)
{
    return uint64_t(order_of(v)) << kIdBits | (kIdMost - static_cast<uint32_t>(id));
}

__device__ __forceinline__ float order_value(uint32_t up)
{
    return __uint_as_float(up & 0x80000000u ? up & 0x7FFFFFFFu : ~up);
}

__device__ __forceinline__ float key_value(uint64_t key)
{
    return order_value(static_cast<uint32_t>(key >> kIdBits));
}

__device__ __forceinline__ int key_id(uint64_t key)
{
    return static_cast<int>(kIdMost - (static_cast<uint32_t>(key) & kIdMost));
}

// What a workgroup goes over: the vectors [lo, hi) of a row, and the elements that lanes take singly.
template <int DT>
struct Piece {
    const typename Fmt<DT>::T* x;      // the row
    int head, lo, hi;
    int one;                           // this lane's single element, or -1
    float single;

    __device__ __forceinline__ const typename Fmt<DT>::T* at(int vec) const
    {
        return x + head + int64_t(vec) * Fmt<DT>::E;
    }
    // Calls f(value, id) for every element, each in one lane.
    template <int THREADS, class F>
    __device__ __forceinline__ void each(F f) const
    {
        constexpr int E = Fmt<DT>::E;
        for (int i = lo + static_cast<int>(threadIdx.x); i < hi; i += THREADS) {
            float v[E];
            unpack<DT>(load_vec<DT, false>(at(i)), v);
#pragma unroll
            for (int j = 0; j < E; ++j) f(v[j], head + i * E + j);
        }
        if (one >= 0) f(single, one);
    }
};

// The choice of the k largest of a piece.  While the sums are formed every lane leaves the maximum of
// each pair of its vectors in a slot (the first 16 bits of its order: a bound that a comparison
// may only find too high; several pairs share a slot in long rows).  The k-th largest of the lanes' own
// maxima is a bound that at least k elements reach, and few more: k elements fall into different
// lanes mostly.  So the slots that reach it name the few vectors that are read again, and what of them
// reaches it is ranked by counting, as (logit, id) in one whole number.
template <int THREADS>
struct Lists {
    static constexpr int kKeys = THREADS < 256 ? 8 * THREADS : 2048, kHits = kKeys / 2;
    static constexpr int kSlots = 4 * kKeys / THREADS;           // of a lane
    union {
        uint16_t slot[kSlots * THREADS];
        uint64_t key[kKeys];
    };
    union {
        uint16_t hit[kHits];
        uint32_t count[256];
    };
    uint32_t lane_max[THREADS];
    uint16_t lane[THREADS];              // the lanes that reach the bound
    uint32_t bound;
    int lanes, hits, keys, above, bin;
};

template <int THREADS>
__device__ __forceinline__ void put_key(Lists<THREADS>& l, uint64_t key)
{
    const int i = atomicAdd(&l.keys, 1);
    if (i < Lists<THREADS>::kKeys) l.key[i] = key;
}

// -inf in 32 bits of a vector.
template <int DT>
constexpr uint32_t kGoneBits = DT == kBF16 ? 0xFF80FF80u : DT == kFP16 ? 0xFC00FC00u : 0xFF800000u;

// Shares of a piece's vectors, and with TOP the slots; `per` pairs to a slot.
template <int DT, int THREADS, bool TOP, bool NT>
__device__ __forceinline__ void piece_sums(Share& share, const Piece<DT>& p, const RowScale& k,
                                           Lists<THREADS>& l, int per)
{
    constexpr int U = 4;
    const int tid = threadIdx.x;
    int slot = tid, left = per;
    auto pair = [&](u32x4 a, u32x4 b) {
        const float g = add_pair<DT>(share, a, b, k);
        if constexpr (TOP) {
            uint16_t o = static_cast<uint16_t>(order_of(g) >> 16);
            if (left != per) o = max(o, l.slot[slot]);
            l.slot[slot] = o;
            if (--left == 0) {
                left = per;
                slot += THREADS;
            }
        }
    };
    int base = p.lo;
    for (; base + U * THREADS <= p.hi; base += U * THREADS) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load_vec<DT, NT>(p.at(base + u * THREADS + tid));
#pragma unroll
        for (int u = 0; u < U; u += 2) pair(v[u], v[u + 1]);
    }
    for (; base < p.hi; base += 2 * THREADS) {
        const int i = base + tid, j = i + THREADS;
        u32x4 a = load_vec<DT, NT>(p.at(min(i, p.hi - 1)));
        u32x4 b = load_vec<DT, NT>(p.at(min(j, p.hi - 1)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i >= p.hi) a[e] = kGoneBits<DT>;
            if (j >= p.hi) b[e] = kGoneBits<DT>;
        }
        pair(a, b);
    }
}

// The largest of a wave's.
template <class N, int D = 1>
__device__ __forceinline__ N lanes_largest(N v)
{
    if constexpr (D < kWave) {
        uint32_t a0, b0, a1 = 0, b1 = 0;
        N a, b;
        if constexpr (sizeof(N) == 8) {
            const uint64_t u = __builtin_bit_cast(uint64_t, v);
            across<D>(static_cast<uint32_t>(u), a0, b0);
            across<D>(static_cast<uint32_t>(u >> 32), a1, b1);
            a = __builtin_bit_cast(N, uint64_t(a1) << 32 | a0);
            b = __builtin_bit_cast(N, uint64_t(b1) << 32 | b0);
        } else {
            across<D>(__builtin_bit_cast(uint32_t, v), a0, b0);
            a = __builtin_bit_cast(N, a0);
            b = __builtin_bit_cast(N, b0);
        }
        return lanes_largest<N, 2 * D>(a > b ? a : b);
    }
    return v;
}

// A bound on the order that at least k of the workgroup's lane maxima reach and not many more: found
// bit by bit, by one wave.
template <int THREADS>
__device__ __forceinline__ uint32_t lane_bound(const Lists<THREADS>& l, int k)
{
    constexpr int N = THREADS / kWave;
    uint32_t v[N], lo = ~0u, hi = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = l.lane_max[i * kWave + threadIdx.x % kWave];
        lo = min(lo, v[i]);
        hi = max(hi, v[i]);
    }
    lo = ~__builtin_amdgcn_readfirstlane(lanes_largest(~lo));
    hi = __builtin_amdgcn_readfirstlane(lanes_largest(hi));
    int bit = 31 - __builtin_clz((lo ^ hi) | 1);
    uint32_t bound = hi >> bit >> 1 << bit << 1;              // what all have in common
    for (; bit >= 0; --bit) {
        const uint32_t trial = bound | 1u << bit;
        int c = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(v[i] >= trial));
        if (c < k) continue;
        bound = trial;
        if (c <= k + k / 16 + 1) break;
    }
    return max(bound, 0x00800000u);                           // -inf is no entry
}

// Where the bound leaves too many (nearly equal rows, and rows made for it): the exact bound of the k
// largest keys, eight bits at a time from histograms, each a pass over the piece, until few enough
// reach it.
template <int DT, int THREADS>
__device__ __forceinline__ void choose_by_passes(const Piece<DT>& p, int k, Lists<THREADS>& l)
{
    uint32_t* const count = l.count;
    uint64_t prefix = 0, bound;
    int before = 0;
    for (int shift = 56;; shift -= 8) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += THREADS) count[i] = 0;
        __syncthreads();
        p.template each<THREADS>([&](float v, int id) {
            const uint64_t key = entry_key(v, id);
            const bool in = v > -__builtin_inff() && (shift == 56 || key >> shift >> 8 == prefix);
            const int bin = in ? static_cast<int>(key >> shift & 255) : -1;
            // all of a wave in one bin is the common case here
            const int first = __builtin_amdgcn_readfirstlane(bin);
            const uint64_t alike = __builtin_amdgcn_ballot_w64(bin == first);
            if (bin == first) {
                if (in && threadIdx.x % kWave == __builtin_ctzll(alike))
                    atomicAdd(&count[bin], static_cast<uint32_t>(__builtin_popcountll(alike)));
            } else if (in) {
                atomicAdd(&count[bin], 1u);
            }
        });
        __syncthreads();
        if (threadIdx.x == 0) {
            int c = before, b = 255;
            for (; b > 0; --b) {
                if (c + static_cast<int>(count[b]) >= k) break;
                c += static_cast<int>(count[b]);
            }
            l.above = c;
            l.bin = b;
        }
        __syncthreads();
        before = l.above;
        prefix = prefix << 8 | static_cast<uint64_t>(l.bin);
        if (shift == 0 || before + static_cast<int>(count[l.bin]) <= Lists<THREADS>::kKeys) {
            bound = prefix << shift;
            break;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) l.keys = 0;
    __syncthreads();
    p.template each<THREADS>([&](float v, int id) {
        const uint64_t key = entry_key(v, id);
        if (v > -__builtin_inff() && key >= bound) put_key(l, key);
    });
    __syncthreads();
}

// Calls emit(rank, key) for the k largest of l.key[0 .. n), the largest first, and emit(rank, 0) for
// the ranks that are left.
template <int THREADS, class F>
__device__ __forceinline__ void emit_ranked(const Lists<THREADS>& l, int n, int k, F emit)
{
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const uint64_t own = l.key[i];
        // 62 bits are a positive finite binary64 number, whose comparison is the faster one
        const double o = __builtin_bit_cast(double, own);
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank += __builtin_bit_cast(double, l.key[j]) > o;
        if (rank < k) emit(rank, own);
    }
    for (int i = n + static_cast<int>(threadIdx.x); i < k; i += THREADS) emit(i, uint64_t(0));
}

// The k largest of a piece: collect(bound) puts all keys that reach the bound and ends with a barrier;
// false where there are too many.
template <int DT, int THREADS, class C, class F>
__device__ __forceinline__ void choose(const Piece<DT>& p, float lane_max, int k, Lists<THREADS>& l, C collect,
                                       F emit)
{
    const int tid = threadIdx.x;
    l.lane_max[tid] = order_of(lane_max);
    if (tid == 0) l.lanes = l.hits = l.keys = 0;
    __syncthreads();
    if (tid < kWave) {
        const uint32_t b = lane_bound(l, k);
        if (tid == 0) l.bound = b;
    }
    __syncthreads();
    const bool fits = collect(l.bound);
    if (!fits || l.keys > Lists<THREADS>::kKeys) choose_by_passes(p, k, l);
    emit_ranked(l, l.keys, k, emit);
}

// The keys of a piece whose slots say where they are.
template <int DT, int THREADS>
__device__ __forceinline__ bool collect_by_slots(const Piece<DT>& p, uint32_t bound, int per, Lists<THREADS>& l)
{
    constexpr int E = Fmt<DT>::E;
    const int tid = threadIdx.x;
    if (l.lane_max[tid] >= bound) l.lane[atomicAdd(&l.lanes, 1)] = static_cast<uint16_t>(tid);
    __syncthreads();
    const int pairs = (p.hi - p.lo + 2 * THREADS - 1) / (2 * THREADS);
    const int slots = (pairs + per - 1) / per;
    const int lanes = l.lanes;
    for (int i = tid / 16; i < lanes; i += THREADS / 16)
        for (int q = tid % 16; q < slots; q += 16) {
            const int at = q * THREADS + l.lane[i];
            if (l.slot[at] >= bound >> 16) {
                const int h = atomicAdd(&l.hits, 1);
                if (h < Lists<THREADS>::kHits) l.hit[h] = static_cast<uint16_t>(at);
            }
        }
    __syncthreads();                          // from here on keys take the slots' place
    const int hits = l.hits;
    if (hits > Lists<THREADS>::kHits) return false;
    const float least = order_value(bound);
    const int each = 2 * per;
    for (int i = tid; i < hits * each; i += THREADS) {
        const int h = l.hit[i / each];
        const int vec = p.lo + (h / THREADS * each + i % each) * THREADS + h % THREADS;
        if (vec >= p.hi) continue;
        float v[E];
        unpack<DT>(load_vec<DT, false>(p.at(vec)), v);
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (v[j] >= least) put_key(l, entry_key(v[j], p.head + vec * E + j));
    }
    if (p.one >= 0 && p.single >= least) put_key(l, entry_key(p.single, p.one));
    __syncthreads();
    return true;
}

// The sums of a piece, relative to 2^ref (in the first wave; m in all lanes).
struct PieceStat {
    double ref, s, c;
    float m;
};

// From the lanes' shares of a piece's vectors.
template <int DT, int THREADS>
__device__ __forceinline__ PieceStat piece_stat(Share share, const Piece<DT>& p, const RowScale& k,
                                                JoinSpace<THREADS>& space, float& lane_max)
{
    if (p.one >= 0) add_one(share, p.single, k.k, k.slack);
    lane_max = share.m;
    PieceStat r;
    float ref;
    join<THREADS>(share, k.k, space, r.m, ref, r.s, r.c);
    r.ref = static_cast<double>(ref);
    if (!(__builtin_fabsf(r.m * k.k) < kRowMost)) {
        share = Share{};
        share.m = r.m;
        p.template each<THREADS>([&](float v, int) {
            const float f[1] = {v};
            add_to(share, f, k.k);
        });
        join<THREADS>(share, k.k, space, r.m, ref, r.s, r.c);
        r.ref = static_cast<double>(r.m) * static_cast<double>(k.k);
    }
    return r;
}

__device__ __forceinline__ void write_entry(const ScoreArgs& a, int64_t at, uint64_t key, const RowStat& r)
{
    const bool there = key != 0 && r.ln_s == r.ln_s;
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

// One row per workgroup.  Bound by HBM and the vector units alike, which are at work two thirds of the
// time: 8192 x 128256 bf16, 0.1 off, 20 entries, 310 us, 6.1 TB/s of the logits that count; without lists
// 2048 x 128256, 0.3 off, 70 us, 5.3 TB/s.  64 entries cost 4096 x 50304 fp16 a second read of a
// seventh of its row (86 us, 4.8 TB/s); 1531 x 32001 fp32, six rows a compute unit, is over before
// the reads are evenly dealt (35 us, 4.5 TB/s).
template <int DT, int THREADS, bool TOP>
__global__ __launch_bounds__(THREADS, 8) void k_scores(ScoreArgs a, int per)
{
    using T = typename Fmt<DT>::T;
    __shared__ JoinSpace<THREADS> space;
    __shared__ Lists<TOP ? THREADS : 1> lists;
    const int64_t row = blockIdx.x;
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    const int64_t target = a.targets != nullptr ? read_table(a.targets + row) : 0;
    if (target < 0) return write_off(a, row);
    const RowScale k = scale_of(a.x);
    const Span<DT> sp(x, n);
    Piece<DT> p;
    p.x = x;
    p.head = sp.head;
    p.lo = 0;
    p.hi = sp.nvec;
    p.one = sp.single(threadIdx.x);
    p.single = p.one >= 0 ? widen<DT>(x[p.one]) : 0.0f;
    const float xt = target < n ? widen<DT>(x[target]) : 0.0f;
    float lane_max;
    auto& l = reinterpret_cast<Lists<THREADS>&>(lists);
    Share share;
    if (a.x.stream) piece_sums<DT, THREADS, TOP, true>(share, p, k, l, per);
    else piece_sums<DT, THREADS, TOP, false>(share, p, k, l, per);
    const PieceStat st = piece_stat<DT, THREADS>(share, p, k, space, lane_max);
    __shared__ RowStat whole;
    if (threadIdx.x < kWave) {
        const RowStat r = stat_of(st.m, st.ref, st.s, st.c, k);
        if (threadIdx.x == 0) {
            write_row(a, row, target, xt, r);
            whole = r;                       // the choice has barriers before anything is emitted
        }
    }
    if constexpr (TOP)
        choose<DT, THREADS>(
            p, lane_max, a.top, l, [&](uint32_t bound) { return collect_by_slots(p, bound, per, l); },
            [&](int rank, uint64_t key) { write_entry(a, row * a.top + rank, key, whole); });
}

// Few rows, less than the chip has room for: a row is cut into parts, one workgroup each, that leave
// their sums and their own k largest in the workspace; then one workgroup a row joins them.  A lane
// holds its vectors of a part, up to kPartHeld: the choice needs no slots and no second read then.
// Bound by latency: 1 x 128256 bf16 takes 4.0 us and 2.5 us without lists, two launches and the dependent steps of a
// row's sums; the choice of 20 entries, a bound found bit by bit and barriers, adds as much again (7.8 and 5.1 us).  48
// rows with 8 entries 10 us and 4.5 us, where the reads alone take 0.04 and 1.9 us.
constexpr int kPartThreads = 256;
constexpr int kPartHeld = 4;
constexpr int kMaxParts = kWave;

struct ScoreParts {
    PieceStat* stat;         // rows x parts
    uint64_t* key;           // rows x parts x top
    int parts, vecs;         // per row; vectors of a part
};

template <int DT, bool TOP, bool HELD>
__global__ __launch_bounds__(kPartThreads) void k_score_parts(ScoreArgs a, ScoreParts w, int per)
{
    using T = typename Fmt<DT>::T;
    __shared__ JoinSpace<kPartThreads> space;
    __shared__ Lists<TOP ? kPartThreads : 1> lists;
    const unsigned parts = static_cast<unsigned>(w.parts);
    const int64_t row = blockIdx.x / parts;
    const int part = static_cast<int>(blockIdx.x % parts);
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    if (a.targets != nullptr && read_table(a.targets + row) < 0) return;
    const RowScale k = scale_of(a.x);
    const Span<DT> sp(x, a.x.vocab);
    Piece<DT> p;
    p.x = x;
    p.head = sp.head;
    p.lo = min(part * w.vecs, sp.nvec);
    p.hi = min(p.lo + w.vecs, sp.nvec);
    p.one = part == 0 ? sp.single(threadIdx.x) : -1;
    p.single = p.one >= 0 ? widen<DT>(x[p.one]) : 0.0f;
    float lane_max;
    auto& l = reinterpret_cast<Lists<kPartThreads>&>(lists);
    Share share;
    u32x4 v[kPartHeld];
    if constexpr (HELD) {
#pragma unroll
        for (int u = 0; u < kPartHeld; ++u)
            v[u] = load_vec<DT, false>(p.at(max(min(p.lo + u * kPartThreads + static_cast<int>(threadIdx.x), p.hi - 1), 0)));
#pragma unroll
        for (int u = 0; u < kPartHeld; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (p.lo + u * kPartThreads + static_cast<int>(threadIdx.x) >= p.hi) v[u][e] = kGoneBits<DT>;
#pragma unroll
        for (int u = 0; u < kPartHeld; u += 2) add_pair<DT>(share, v[u], v[u + 1], k);
    } else {
        piece_sums<DT, kPartThreads, TOP, false>(share, p, k, l, per);
    }
    const PieceStat st = piece_stat<DT, kPartThreads>(share, p, k, space, lane_max);
    if (threadIdx.x == 0) w.stat[blockIdx.x] = st;
    if constexpr (TOP)
        choose<DT, kPartThreads>(
            p, lane_max, a.top, l,
            [&](uint32_t bound) {
                if constexpr (!HELD) return collect_by_slots(p, bound, per, l);
                constexpr int E = Fmt<DT>::E;
                const float least = order_value(bound);
                if (lane_max >= least) {
#pragma unroll
                    for (int u = 0; u < kPartHeld; ++u) {
                        float f[E];
                        unpack<DT>(v[u], f);
#pragma unroll
                        for (int j = 0; j < E; ++j)
                            if (f[j] >= least)
                                put_key(l, entry_key(f[j], p.head + (p.lo + u * kPartThreads + static_cast<int>(threadIdx.x)) * E + j));
                    }
                    if (p.one >= 0 && p.single >= least) put_key(l, entry_key(p.single, p.one));
                }
                __syncthreads();
                return true;
            },
            [&](int rank, uint64_t key) { w.key[int64_t(blockIdx.x) * a.top + rank] = key; });
}

template <int DT, bool TOP>
__global__ __launch_bounds__(kPartThreads) void k_score_join(ScoreArgs a, ScoreParts w)
{
    using T = typename Fmt<DT>::T;
    __shared__ Lists<TOP ? kPartThreads : 1> lists;
    const int64_t row = blockIdx.x;
    const int n = a.x.vocab, tid = threadIdx.x, lane = tid % kWave;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    const int64_t target = a.targets != nullptr ? read_table(a.targets + row) : 0;
    if (target < 0) return write_off(a, row);
    const RowScale k = scale_of(a.x);
    const float xt = target < n ? widen<DT>(x[target]) : 0.0f;
    // all loads before anything waits for one: the parts' sums, the lists and their deep entries
    PieceStat st{-__builtin_inf(), 0.0, 0.0, -FLT_MAX};
    if (lane < w.parts) st = w.stat[row * w.parts + lane];
    constexpr int kEach = Lists<kPartThreads>::kKeys / kPartThreads;
    const int entries = w.parts * a.top;                   // at most kKeys
    uint64_t key[TOP ? kEach : 1], bound = 0;
    if constexpr (TOP) {
        const uint64_t* list = w.key + row * entries;
        // of P sorted lists the entries d + 1 deep, d + 1 = k / P rounded up: at least k entries reach the
        // j-th largest of these, j = k / (d + 1) rounded up
        const int deep = (a.top + w.parts - 1) / w.parts - 1;
        if (lane < w.parts) bound = list[lane * a.top + deep];
#pragma unroll
        for (int i = 0; i < kEach; ++i) key[i] = i * kPartThreads + tid < entries ? list[i * kPartThreads + tid] : 0;
    }
    const float m = lanes_max<kWave>(st.m);
    // a part without any element in reach has no say in the reference; a NaN's is kept
    const double own = st.ref;
    const double ref = lanes_largest(st.s != 0.0 ? own : -__builtin_inf());
    const double d = st.s != 0.0 ? own - ref : 0.0;
    const double down = static_cast<double>(exp2_hw(static_cast<float>(d)));
    const double c = lanes_sum<kWave>(down == 0.0 ? 0.0 : (st.c + st.s * d) * down);
    const double s = lanes_sum<kWave>(st.s * down);
    const RowStat r = stat_of(m, ref, s, c, k);
    if (tid == 0) write_row(a, row, target, xt, r);
    if constexpr (TOP) {
        auto& l = reinterpret_cast<Lists<kPartThreads>&>(lists);
        const int deep = (a.top + w.parts - 1) / w.parts, nth = (a.top + deep - 1) / deep;
        const double b = __builtin_bit_cast(double, bound);       // a positive number, as in emit_ranked
        auto of_lane = [&](int i) {
            const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(bound), i);
            const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(bound >> 32), i);
            return uint64_t(hi) << 32 | lo;
        };
        int before = 0;
        for (int i = 0; i < w.parts; ++i) before += __builtin_bit_cast(double, of_lane(i)) > b;
        // of keys none is alike; where the j-th is an empty place, all keys are taken
        const uint64_t nth_lane = __builtin_amdgcn_ballot_w64(lane < w.parts && before == nth - 1 && bound != 0);
        bound = nth_lane != 0 ? of_lane(__builtin_ctzll(nth_lane)) : 1;
        if (tid == 0) l.keys = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (key[i] >= bound) put_key(l, key[i]);
        __syncthreads();
        emit_ranked(l, l.keys, a.top,
                    [&](int rank, uint64_t v) { write_entry(a, row * a.top + rank, v, r); });
    }
}

// The gradient of sum_r (g lp + h H): with y = log2 q = x k - lse log2(e) in two floats,
//   dx_j = f (g (1[j = t] - q_j) - h q_j (ln q_j + H)) = q_j (y_j (-h f ln 2) - f (g + h H)),
// the target's element apart, from expm1 of its log-probability, stored over the dense one by
// the lane that has its vector.  Two roundings of y as in the gradient of log-probabilities.
// Bound by HBM: 2 bytes read and written per 16-bit logit against about 10 VALU operations.
// 2048 x 128256 bf16, 0.3 off: 144 us, 6.2 TB/s read and written.
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

// Pairs that share a slot where `vecs` vectors are dealt to `threads` lanes.
template <int THREADS>
int pairs_per_slot(int vecs)
{
    constexpr int slots = Lists<THREADS>::kSlots;
    const int pairs = (vecs + 2 * THREADS - 1) / (2 * THREADS);
    const int per = (pairs + slots - 1) / slots;
    return per > 0 ? per : 1;
}

// Without lists, at 7 to 8 rows a compute unit: only five workgroups of 256 lanes fit on one, by shared memory that
// nothing uses.  With eight, all rows are there at once, and where some are switched off a unit may have eight live ones
// and another three.  bf16, five against eight: 2048 x 128256 all live 82 us against 85, 0.3 off 67 against 71;
// 1920 x 50304 34.4 against 36.3 and 28.0 against 30.4.  With fewer rows the rest of a second turn costs more (1281 x
// 128256 63 against 56; 1664 70 against 70), and with more, eight take turns too (2300 x 128256 100 against 98,
// 4096 x 32001 fp32 84 against 81).
constexpr unsigned kReserved = 32000;
constexpr int kComputeUnits = 256;

template <int DT, int THREADS>
void whole_rows(const ScoreArgs& a, hipStream_t s)
{
    const unsigned rows = static_cast<unsigned>(a.x.rows);
    const int per = pairs_per_slot<THREADS>(a.x.vocab / Fmt<DT>::E);
    const bool apart = THREADS == 256 && a.x.rows > 7 * kComputeUnits && a.x.rows <= 8 * kComputeUnits;
    if (a.top > 0) k_scores<DT, THREADS, true><<<rows, THREADS, 0, s>>>(a, per);
    else k_scores<DT, THREADS, false><<<rows, THREADS, apart ? kReserved : 0, s>>>(a, per);
}

// Rows of at least kSplitVecs vectors, up to kSplitRows of them.  A call, 20 entries, split against whole:
// 128256 bf16 logits (16032 vectors), 1 row 12.9 us against 18.3, 64 rows 15.7 against 19.1, 128 rows 21.0
// against 21.7, 160 rows 23.3 against 23.2, 200 rows 26.5 against 23.9; 60000 fp32 logits (15000), 1 row 11.5 against
// 15.3, 128 rows 16.8 against 19.1, 200 rows 21.0 against 24.0, 256 rows 23.7 against 24.4; 262144 bf16 logits, 128 rows 30.5
// against 37.5, 160 rows 35.0 against 38.2, 200 rows 40.9 against 38.5; 50304 bf16 logits (6288), 1 row 11.5 against 11.3.
// (Between 128 and 200 rows the shortest of these gain nothing.)
constexpr int kSplitRows = 128;
constexpr int kSplitVecs = 10000;

// Split the rows over several workgroups?  Fills `w` in the workspace if so.
template <int DT>
bool split(const ScoreArgs& a, ScoreParts* w)
{
    const int nvec = a.x.vocab / Fmt<DT>::E;
    if (a.workspace == nullptr || a.x.rows > kSplitRows || nvec < kSplitVecs) return false;
    const int entry = static_cast<int>(sizeof(PieceStat)) + 8 * a.top;
    // what the joining workgroup and the workspace have room for
    int most = a.top > 0 ? std::min(kMaxParts, Lists<kPartThreads>::kKeys / a.top) : kMaxParts;
    most = static_cast<int>(std::min<int64_t>(most, MP_SCORE_WORKSPACE_BYTES / (int64_t(entry) * a.x.rows)));
    // two workgroups for each compute unit, parts of two vectors a lane at least, and such as lanes can
    // hold if possible
    int parts = std::min(512 / a.x.rows, (nvec + 2 * kPartThreads - 1) / (2 * kPartThreads));
    parts = std::min(std::max(parts, (nvec + kPartHeld * kPartThreads - 1) / (kPartHeld * kPartThreads)), most);
    if (parts < 2) return false;
    w->vecs = (nvec + parts - 1) / parts;
    w->parts = (nvec + w->vecs - 1) / w->vecs;
    w->stat = static_cast<PieceStat*>(a.workspace);
    w->key = reinterpret_cast<uint64_t*>(w->stat + int64_t(a.x.rows) * w->parts);
    return true;
}

template <int DT>
void scores_dt(ScoreArgs a, hipStream_t s)
{
    a.x.stream = logits_bytes<DT>(a.x) > kCacheBytes;
    ScoreParts w;
    if (split<DT>(a, &w)) {
        const unsigned rows = static_cast<unsigned>(a.x.rows), all = rows * static_cast<unsigned>(w.parts);
        const int per = pairs_per_slot<kPartThreads>(w.vecs);
        const bool held = w.vecs <= kPartHeld * kPartThreads;
        if (a.top > 0) {
            if (held) k_score_parts<DT, true, true><<<all, kPartThreads, 0, s>>>(a, w, per);
            else k_score_parts<DT, true, false><<<all, kPartThreads, 0, s>>>(a, w, per);
            k_score_join<DT, true><<<rows, kPartThreads, 0, s>>>(a, w);
        } else {
            if (held) k_score_parts<DT, false, true><<<all, kPartThreads, 0, s>>>(a, w, per);
            else k_score_parts<DT, false, false><<<all, kPartThreads, 0, s>>>(a, w, per);
            k_score_join<DT, false><<<rows, kPartThreads, 0, s>>>(a, w);
        }
        return;
    }
    // Workgroups of 256 lanes; of fewer for short rows, whose joins and barriers would cost more than
    // their logits, and for somewhat longer ones where there are enough of them to fill the chip.  bf16, 20
    // entries, 64, 128 and 256 lanes: 8192 x 2000 23, 25 and 40 us, 8192 x 8192 38, 38 and 45, 8192 x 16000
    // 68, 61 and 66, 8192 x 64000 197, 181 and 179; 512 x 8192 11.0, 9.6 and 9.8, 512 x 32000 24, 18 and 14.
    // At 1024 rows the forms are alike (1024 x 8192 11.1, 10.6 and 11.4, 1024 x 16000 15.6, 13.8 and 14.0), and from there
    // fewer lanes gain (2048 x 8192 13.7, 13.6 and 15.6, 2048 x 16000 19.0, 19.1 and 20.4).
    // (A bound from 64 lanes' maxima is one for at most 64 entries.)
    const int nvec = a.x.vocab / Fmt<DT>::E;
    const bool many = a.x.rows >= 2048;
    if (nvec <= (many ? 1024 : 512) && a.top <= 64) whole_rows<DT, 64>(a, s);
    else if (nvec <= (many ? 4096 : 512)) whole_rows<DT, 128>(a, s);
    else whole_rows<DT, 256>(a, s);
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
