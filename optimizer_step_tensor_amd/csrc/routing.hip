// HIP kernels of the routing to experts: the choice and the weights of each token, the sums over the
// tokens that balance the experts, the gradient of all of it, and the balancing bias's step.
//
// Experts are chosen by c_e = s_e + b_e, s = softmax(x) or sigmoid(x).  Two of a token's c are closer
// than 2^-24 about once in 10^5 tokens, and fp32 arithmetic would then choose by its rounding
// errors: c is formed in binary64, which runs at fp32's rate here, and rounded to 42 bits.  Without a bias
// (and without sums of two scores) the order of c is that of the logits: no score is formed for the
// choice then.
//
// A choice is made on keys, numbers that hold c (or the logit) and the expert, the lower the larger,
// so that equal c fall to the lowest number and one maximum or minimum instruction is a whole step of
// a sorting network: binary64 with the expert in the last ten bits, or, for 16-bit logits, whole numbers of
// 32 bits.  L lanes share a token, each with P experts in chunks of eight neighbours; a lane sorts its
// chunks and keeps the K best of them, and lanes join their lists in log2(L) steps.  Few lanes with many
// experts do the least: a join costs the same however many lanes repeat it.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "rows.h"
#include "routing.h"

namespace mpk {
namespace {

constexpr double kLog2E = 1.4426950408889634;

// a b + c with c in scalar registers: the compiler would rather move c into vector registers first.
__device__ __forceinline__ double fma_const(double a, double b, double c)
{
    double r;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "s"(c));
    return r;
}

// 2^t for |t| <= 1/2 by Chebyshev interpolation of degree 10 (relative error 3e-16).  The library's exp
// takes twice the operations.
__device__ __forceinline__ double exp2_fraction(double t)
{
    double p = t * 7.072585949269224e-09 + 1.0208690299958306e-07;
    p = fma_const(p, t, 1.321544258792169e-06);
    p = fma_const(p, t, 1.5252657260200837e-05);
    p = fma_const(p, t, 0.0001540353044173605);
    p = fma_const(p, t, 0.0013333558230164974);
    p = fma_const(p, t, 0.009618129107606888);
    p = fma_const(p, t, 0.05550410866444772);
    p = fma_const(p, t, 0.24022650695910097);
    p = fma_const(p, t, 0.69314718055995);
    return fma_const(p, t, 1.0);
}

// 2^y for -1100 <= y <= 1000.
__device__ __forceinline__ double exp2_series(double y)
{
    const double whole = __builtin_rint(y);
    return __builtin_ldexp(exp2_fraction(y - whole), static_cast<int>(whole));
}

// exp(a) for |a| < 700: adding 1.5 2^52 leaves the exponent's whole part in the last bits.
__device__ __forceinline__ double exp_tame(double a)
{
    constexpr double kWhole = 6755399441055744.0;
    const double u = __builtin_fma(a, kLog2E, kWhole);
    const double whole = u - kWhole;
    const uint64_t p = __builtin_bit_cast(uint64_t, exp2_fraction(__builtin_fma(a, kLog2E, -whole)));
    const uint32_t hi = static_cast<uint32_t>(p >> 32) + (static_cast<uint32_t>(__builtin_bit_cast(uint64_t, u)) << 20);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | static_cast<uint32_t>(p));
}

// 1 / d for d in binary64's middle range: the instruction's 2^-24 and one of Newton's steps, or two.
__device__ __forceinline__ double reciprocal_fast(double d)
{
    const double r = __builtin_amdgcn_rcp(d);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
__device__ __forceinline__ double reciprocal(double d)
{
    const double r = reciprocal_fast(d);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

// sigmoid(z), or exp(z - m) for z <= m, of any z.
__device__ __forceinline__ double score_of(float z, float m, bool sigmoid)
{
    const double a = sigmoid ? -static_cast<double>(z) : static_cast<double>(z) - static_cast<double>(m);
    const double y = a * kLog2E;
    const double e = exp2_series(y < -1100.0 ? -1100.0 : y > 1000.0 ? 1000.0 : y);
    if (!sigmoid) return e;
    return y > 1000.0 ? 0.0 : reciprocal(1.0 + e);
}

// exp(z - m) in fp32, relative error 2^-24 (|z - m| + 2): x log2(e) with the constant in two parts.
__device__ __forceinline__ float share_to_fast(float z, float m)
{
    constexpr float hi = 1.44269502162933349609375f, lo = 1.925963033500e-8f;
    const float t = z - m;
    return exp2_hw(__builtin_fmaf(t, lo, t * hi));
}

// A token whose logits are all below this: its sigmoids are exp(z) to fp32's last bit, and from here on leave
// fp32's range, or its normal numbers, sooner than their shares do, which are a softmax's.
constexpr float kLow = -32.0f;

// A sigmoid of a token whose largest logit m is below kLow, relative to exp(m); 0 below 2^-1000 as in score_of.
constexpr float kNothing = -693.14718f;                  // -1000 ln 2
__device__ __forceinline__ float low_share(float z, float m)
{
    return z < kNothing ? 0.0f : share_to_fast(z, m);
}

constexpr int kIdBits = 10;                              // MP_ROUTE_MAX_EXPERTS is 2^10
constexpr uint64_t kIdMask = (1 << kIdBits) - 1;

// A bias of an expert that is closed, and what a c is above that is open.  (Other biases are held below
// 1e38 in size.)
constexpr float kClosed = -FLT_MAX;
constexpr float kBiasMost = 1e38f;
constexpr double kOpen = -2e38;
constexpr double kMost = 1e300;                          // the key of +inf: no key is a NaN's

// c (finite, not -0) as far as it counts: what is equal but for the rounding of sums is equal then.
__device__ __forceinline__ uint64_t rounded(double c)
{
    return (__builtin_bit_cast(uint64_t, c) + (kIdMask + 1) / 2) & ~kIdMask;
}

// Keys of type double or uint32_t.
template <class Key>
__device__ __forceinline__ Key no_key()
{
    if constexpr (std::is_same_v<Key, double>) return -__builtin_inf();
    else return 0;
}

// Of a negative c the larger last bits are the smaller number.
__device__ __forceinline__ double key_of(double c, int e)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, c) + (kIdMask + 1) / 2;
    const uint32_t hi = static_cast<uint32_t>(u >> 32);
    const uint32_t sign = static_cast<uint32_t>(static_cast<int32_t>(hi) >> 31);
    constexpr uint32_t mask = static_cast<uint32_t>(kIdMask);
    const uint32_t last = (static_cast<uint32_t>(e) ^ mask) ^ (sign & mask);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | ((static_cast<uint32_t>(u) & ~mask) | last));
}

// 16-bit logits: the order in a key's upper half, the expert in its lower one.  Two of a word are put in
// order at a time, -0 as 0; `size` becomes the largest magnitudes, above an infinity's where there is a NaN.
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

template <int DT>
constexpr uint32_t kInfBits = DT == kBF16 ? 0x7F80u : 0x7C00u;

__device__ __forceinline__ uint32_t order_of_pair(uint32_t w, u16x2& size)
{
    const i16x2 sign = __builtin_bit_cast(i16x2, w) >> i16x2{15, 15};
    const i16x2 most = __builtin_bit_cast(i16x2, w & 0x7FFF7FFFu);
    size = __builtin_elementwise_max(size, __builtin_bit_cast(u16x2, most));
    const i16x2 k = (most ^ sign) - sign;
    return __builtin_bit_cast(uint32_t, k) ^ 0x80008000u;
}

template <int DT>
__device__ __forceinline__ float logit_of_key(uint32_t key)
{
    const uint32_t o = key >> 16;
    return widen<DT>(static_cast<uint16_t>(o & 0x8000u ? o ^ 0x8000u : 0x10000u - o));
}

template <int DT, class Key, bool EXACT>
__device__ __forceinline__ bool is_open(Key key)
{
    if constexpr (EXACT) return key > kOpen;
    else if constexpr (DT == kFP32) return key > no_key<Key>();
    else return key > ((0x8000u - kInfBits<DT>) << 16 | 0xFFFFu);          // -inf and none
}

template <class Key>
__device__ __forceinline__ int key_expert(Key key)
{
    if constexpr (std::is_same_v<Key, double>) {
        const uint64_t u = __builtin_bit_cast(uint64_t, key);
        const int last = static_cast<int>(u & kIdMask);
        return u >> 63 ? last : static_cast<int>(kIdMask) - last;
    } else {
        return static_cast<int>(0xFFFFu - (key & 0xFFFFu));
    }
}

__device__ __forceinline__ double key_score(double key)
{
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~kIdMask);
}

// Maximum and minimum: one instruction each.  (A binary64 one is written out: the compiler puts a
// quieting of NaN before its own.  It depends on no unfinished result but through its operands.)
__device__ __forceinline__ double max_key(double a, double b)
{
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double min_key(double a, double b)
{
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_key(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t min_key(uint32_t a, uint32_t b) { return min(a, b); }

template <class Key>
__device__ __forceinline__ void order_pair(Key& a, Key& b)          // the larger first
{
    const Key hi = max_key(a, b);
    b = min_key(a, b);
    a = hi;
}

// Eight keys, the largest first, in 19 comparisons (Batcher's odd-even merge sort).
template <class Key>
__device__ __forceinline__ void sort8(Key (&k)[8])
{
    constexpr int pair[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                 {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int i = 0; i < 19; ++i) order_pair(k[pair[i][0]], k[pair[i][1]]);
}

// A bitonic list of K keys, the largest first.
template <int K, class Key>
__device__ __forceinline__ void sort_bitonic(Key (&k)[K])
{
#pragma unroll
    for (int d = K / 2; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (!(i & d)) order_pair(k[i], k[i + d]);
}

// Lane D away in groups that are alike below D (`across`).
template <int D, class Key>
__device__ __forceinline__ Key partner(Key v)
{
    // the row swaps give both values: which of them is the own one depends on the lane
    if constexpr (std::is_same_v<Key, double>) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = partner<D>(static_cast<uint32_t>(u)), hi = partner<D>(static_cast<uint32_t>(u >> 32));
        return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
    } else {
        uint32_t a, b;
        across<D>(v, a, b);
        if constexpr (D >= 16) return threadIdx.x & D ? a : b;
        else return b;
    }
}

template <int L, int D = 1, class Key>
__device__ __forceinline__ Key largest_key(Key v)
{
    if constexpr (D < L) return largest_key<L, 2 * D>(max_key(v, partner<D>(v)));
    return v;
}

// The K best of two sorted lists, the other one a lane's D away.
template <int D, int K, class Key>
__device__ __forceinline__ void join_lists(Key (&k)[K])
{
    Key other[K];
#pragma unroll
    for (int i = 0; i < K; ++i) other[i] = partner<D>(k[i]);
#pragma unroll
    for (int i = 0; i < K; ++i) k[i] = max_key(k[i], other[K - 1 - i]);
    sort_bitonic(k);
}

template <int L, int K, int D = 1, class Key>
__device__ __forceinline__ void join_lanes(Key (&k)[K])
{
    if constexpr (D < L) {
        join_lists<D>(k);
        join_lanes<L, K, 2 * D>(k);
    }
}

// The sum over the lanes that are a multiple of L apart.
template <int L>
__device__ __forceinline__ double tokens_sum(double v)
{
    if constexpr (L == kWave) return v;
    else if constexpr (L == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        constexpr int rotate8 = 0x128;              // of 16 lanes
        const int lo = __builtin_amdgcn_mov_dpp(static_cast<int>(u), rotate8, 0xF, 0xF, true);
        const int hi = __builtin_amdgcn_mov_dpp(static_cast<int>(u >> 32), rotate8, 0xF, 0xF, true);
        return tokens_sum<16>(v + __builtin_bit_cast(double, uint64_t(static_cast<uint32_t>(hi)) << 32 |
                                                                 static_cast<uint32_t>(lo)));
    } else {
        return tokens_sum<2 * L>(v + partner<L>(v));
    }
}

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr double kTiny = 1e-20;

// What a workgroup leaves of its tokens: experts + 1 sums of shares (the last: of squared lse), then as
// many counts (the last: tokens routed).
struct RouteSums {
    double* share;
    int32_t* load;
    double* part;       // for each workgroup that joins them: its part of the balance loss
    int32_t* done;      // and how many of those are done: cleared by the first workgroup
    int groups;         // workgroups
};

// Logits up to this size, and tokens whose largest is not below a quarter of it on that side (kLow for a sigmoid's
// sums: fp32 holds the scores and their sum's reciprocal then), have exponentials and sums in binary64's middle range.
constexpr float kTame = 340.0f;

// n, for comparisons that are formed where they are used and not, sixteen lane masks of them, kept over
// a loop.
__device__ __forceinline__ int here(int n)
{
    asm volatile("" : "+s"(n));
    return n;
}

// Eight neighbouring logits from element e of a row of n; `past` past its end.
template <int DT>
__device__ __forceinline__ void load8(const typename Fmt<DT>::T* x, int e, int n, float past, float* z)
{
    constexpr int E = Fmt<DT>::E;
    if (e + 8 <= n) {
#pragma unroll
        for (int i = 0; i < 8; i += E) {
            float f[E];
            unpack<DT>(load_vec<DT, false>(x + e + i), f);
#pragma unroll
            for (int j = 0; j < E; ++j) z[i + j] = f[j];
        }
    } else {
        const int end = here(n);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = e + j < end ? widen<DT>(x[e + j]) : past;
    }
}

// The same of 16-bit logits as they are.
template <int DT>
__device__ __forceinline__ u32x4 load8_raw(const uint16_t* x, int e, int n)
{
    if (e + 8 <= n) return load_vec<DT, false>(x + e);
    constexpr uint32_t gone = 0x8000u | kInfBits<DT>;
    const int end = here(n);
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = e + j < end ? x[e + j] : gone;
    return u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
}

// The waves of a workgroup share nothing but counts: what a wave writes to its own part of the shared
// memory its lanes read back in order.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Waves a SIMD that k_route's registers leave room for, without scratch.  Without sums that is one or two more
// (65536 x 256 by a bias 43 us, 52 in the form with sums; 131072 x 128 by logits 17.1 and 18.5; 131072 x
// 64 12.4 and 14.1).
template <int DT, int L, int P, bool EXACT, bool SUMS>
constexpr int route_waves()
{
    if (SUMS) return EXACT && P == 16 ? 2 : EXACT || DT == kFP32 ? 3 : 4;
    if (EXACT) return P == 8 ? 4 : DT == kFP16 && L == 8 ? 2 : 3;
    return DT == kFP32 ? (P == 8 ? 5 : 3) : P == 8 ? 7 : 5;
}

// Places for keys that the groups of a token are formed from: two for each chunk, or all experts where
// the groups' borders are not the chunks'.
__host__ __device__ __forceinline__ int group_keys(int n, int groups, int all)
{
    return groups == 1 ? 0 : n / groups % 8 == 0 ? all / 4 : all;
}

// L lanes per token, P experts a lane: expert (c L + lane) 8 + j is the lane's P's c 8 + j.
// Bound by the vector units.  131072 x 128 bf16, 8 of 128 by logits: 17 us against 7 us for reads and
// writes; of some 460 instructions for 16 experts a lane 206 sort.  65536 x 256 bf16, 8 of 256 by a bias in 4
// of 8 groups, with sums: 62 us, 84 instructions an expert, of which the binary64 score is 32; two
// waves a SIMD, all that 16 experts' keys leave room for, keep the units at work 70 of 100 cycles.  (The same
// without sums: 43 us; 60 with eight experts and twice the lanes a token, whose joins cost more than two more waves
// give.)  7 x 64: 2.5 us, a launch.
template <int DT, int L, int P, int K, bool EXACT, bool SUMS>
__global__ __launch_bounds__(kRouteThreads, (route_waves<DT, L, P, EXACT, SUMS>()))
void k_route(RouteArgs a, RouteSums w, int space_bytes)
{
    using T = typename Fmt<DT>::T;
    using Key = std::conditional_t<EXACT || DT == kFP32, double, uint32_t>;
    constexpr int R = kWave / L, C = P / 8, N = L * P;         // tokens a wave, chunks a lane, experts
    constexpr bool PACKED = std::is_same_v<Key, uint32_t>;
    extern __shared__ __align__(16) char space[];       // a part for each wave
    __shared__ int32_t count[N];
    __shared__ __align__(16) float bias_of[EXACT ? N : 1];
    __shared__ uint8_t group_no[N];
    __shared__ double square[kRouteWaves];
    __shared__ int32_t routed[kRouteWaves];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int sub = lane % L, slot = lane / L;
    const int n = a.x.vocab;
    const int width = n / a.groups;
    const bool sigmoid = a.sigmoid != 0;
    // this token's keys, the groups' and whether these are open
    const int keys = group_keys(n, a.groups, N);
    char* const own_space = space + wave * space_bytes;
    Key* const mine = reinterpret_cast<Key*>(own_space) + slot * (keys + a.groups);
    Key* const group_of = mine + keys;
    uint8_t* const open_of = reinterpret_cast<uint8_t*>(reinterpret_cast<Key*>(own_space) + R * (keys + a.groups)) +
                             slot * a.groups;
    // A lane's sums are fp32 (binary64 ones would take sixteen registers more than there are), of 2^22 tokens
    // over at least 1360 waves: below 3100 additions, 2^-12.4 relative if all were off the same way.
    // The lanes' are joined in binary64.
    float total[P] = {};
    double squares = 0.0;
    int tokens = 0;
    bool some_open = true;              // some expert that the bias leaves open
    if constexpr (SUMS) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *w.done = 0;
        for (int e = threadIdx.x; e < N; e += kRouteThreads) count[e] = 0;
        __syncthreads();
    }
    if (a.groups > 1) {
        for (int e = threadIdx.x; e < N; e += kRouteThreads) group_no[e] = static_cast<uint8_t>(e < n ? e / width : 0);
        __syncthreads();
    }
    if constexpr (EXACT) {
        some_open = false;
        for (int e = threadIdx.x; e < N; e += kRouteThreads) {
            const float v = e >= n ? -__builtin_inff() : a.bias != nullptr ? a.bias[e] : 0.0f;
            bias_of[e] = v > -__builtin_inff() ? __builtin_amdgcn_fmed3f(v, -kBiasMost, kBiasMost) : kClosed;
        }
        __syncthreads();
        for (int e = lane; e < N; e += kWave) some_open |= bias_of[e] > kClosed;
        some_open = __builtin_amdgcn_ballot_w64(some_open) != 0;
    }
    const int step = static_cast<int>(gridDim.x) * kRouteWaves * R;        // rows are below 2^22
    for (int first = (static_cast<int>(blockIdx.x) * kRouteWaves + wave) * R; first < a.x.rows; first += step) {
        int row = first + slot;
        asm volatile("" : "+v"(row));       // addresses are formed from it, not each kept and stepped
        const bool live = row < a.x.rows && (a.mask == nullptr || a.mask[row] != 0);
        const T* x = static_cast<const T*>(a.x.x) + int64_t(row) * a.x.stride;
        Key key[P];
        bool bad = false, tame = false;
        float m;
        u32x4 raw[PACKED ? C : 1];
        float z[PACKED ? 1 : P];
        if constexpr (PACKED) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                raw[c] = live ? load8_raw<DT>(x, (c * L + sub) * 8, n) : u32x4{0u, 0u, 0u, 0u};
            u16x2 size = {0, 0};
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const uint32_t o = order_of_pair(raw[i / 8][i % 8 / 2], size);
                const uint32_t last = 0xFFFFu - static_cast<uint32_t>((i / 8 * L + sub) * 8 + i % 8);
                key[i] = o << 16 | last;
                key[i + 1] = (o & 0xFFFF0000u) | (last - 1);
            }
            Key most = key[0];
#pragma unroll
            for (int i = 1; i < P; ++i) most = max_key(most, key[i]);
            m = logit_of_key<DT>(largest_key<L>(most));
            const bool nan = size.x > kInfBits<DT> || size.y > kInfBits<DT>;
            if (__builtin_amdgcn_ballot_w64(nan) != 0) bad = lanes_max<L>(nan ? 1.0f : 0.0f) > 0.0f;
            bad |= !sigmoid && m == __builtin_inff();
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (live) load8<DT>(x, (c * L + sub) * 8, n, EXACT ? -kTame : -__builtin_inff(), z + c * 8);
                else
                    for (int j = 0; j < 8; ++j) z[c * 8 + j] = 0.0f;
            }
            m = z[0];
#pragma unroll
            for (int i = 1; i < P; ++i) m = __builtin_fmaxf(m, z[i]);
            m = __builtin_fmaxf(lanes_max<L>(m), -FLT_MAX);
        }
        // Are all logits of the wave's tokens of a size that needs no care?  (What is past a token's
        // experts is at the lower end then, closed, and adds nothing that shows to a sum.)
        if constexpr (EXACT) {
            float lo = z[0], hi = z[0];
#pragma unroll
            for (int i = 1; i < P; ++i) {
                lo = __builtin_fminf(lo, z[i]);
                hi = __builtin_fmaxf(hi, z[i]);
            }
            bool odd = !(lo >= -kTame && hi <= kTame && m >= (SUMS && sigmoid ? kLow : -kTame / 4));
#pragma unroll
            for (int i = 0; i < P; i += 2) odd |= __builtin_isunordered(z[i], z[i + 1]);
            tame = __builtin_amdgcn_ballot_w64(odd) == 0;
        }
        if constexpr (!PACKED) if (!tame) {
            if constexpr (EXACT) {
                m = -FLT_MAX;
                const int end = here(n);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if ((i / 8 * L + sub) * 8 + i % 8 >= end) z[i] = -__builtin_inff();
                    m = __builtin_fmaxf(m, z[i]);
                }
                m = lanes_max<L>(m);
            }
#pragma unroll
            for (int i = 0; i < P; i += 2) bad |= __builtin_isunordered(z[i], z[i + 1]);
            // +inf is the largest then; nothing but -inf leaves the sum 0
            bad = lanes_max<L>(bad ? 1.0f : 0.0f) > 0.0f || (!sigmoid && m == __builtin_inff());
        }

        // the scores, where the choice or a sum over the tokens wants all of them
        double all = 0.0;
        bool some = live && some_open;  // is there an open expert?
        double part = 0.0;
        if constexpr (EXACT) {
            float s[P];                  // for the sums: shares, but scores of a tame sigmoid
            // four experts' arithmetic at a time: all sixteen at once would take all registers
            auto four = [](int i) {
                if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            };
            auto number = [&](int i) { return (i / 8 * L + sub) * 8 + i % 8; };
            // and what the three ways below have in common is not formed before them
            auto apart = [&](int i) { asm volatile("" : "+v"(z[i])::"memory"); };
            if (tame && sigmoid) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    apart(i);
                    const double c = reciprocal_fast(1.0 + exp_tame(-static_cast<double>(z[i])));
                    all += c;
                    s[i] = static_cast<float>(c);
                    key[i] = key_of(c + static_cast<double>(bias_of[number(i)]), number(i));
                    four(i);
                }
                all = lanes_sum<L>(all);
                part = reciprocal(all);
            } else if (tame) {
                const double top = static_cast<double>(m);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    apart(i);
                    key[i] = exp_tame(static_cast<double>(z[i]) - top);
                    all += key[i];
                    four(i);
                }
                all = lanes_sum<L>(all);
                part = reciprocal(all);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const double c = key[i] * part;
                    s[i] = static_cast<float>(c);
                    key[i] = key_of(c + static_cast<double>(bias_of[number(i)]), number(i));
                    four(i);
                }
            } else {
                bool any = false;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    apart(i);
                    key[i] = score_of(z[i], m, sigmoid);
                    all += key[i];
                    four(i);
                }
                all = lanes_sum<L>(all);
                part = all > 0.0 ? reciprocal(all) : 0.0;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const double p = key[i] * part, c = sigmoid ? key[i] : p;
                    s[i] = bad ? 0.0f : static_cast<float>(p);         // NaN times 0 would be in the sums
                    const float bias = z[i] > -__builtin_inff() ? bias_of[number(i)] : kClosed;
                    any |= bias > kClosed;
                    key[i] = key_of((bias > kClosed ? c : 0.0) + static_cast<double>(bias), number(i));
                    four(i);
                }
                if (bad) part = 0.0;
                some = live && !bad && lanes_max<L>(any ? 1.0f : 0.0f) > 0.0f;
            }
            if (SUMS) {
                const float f = !some ? 0.0f : sigmoid && tame ? static_cast<float>(part) : 1.0f;
#pragma unroll
                for (int i = 0; i < P; ++i) total[i] = __builtin_fmaf(s[i], f, total[i]);
            }
        } else {
            if constexpr (DT == kFP32) {
                bool any = false;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    key[i] = key_of(static_cast<double>(z[i] + 0.0f), (i / 8 * L + sub) * 8 + i % 8);      // -0 is 0
                    const bool in = z[i] > -__builtin_inff();
                    any |= in;
                    if (!in) key[i] = no_key<Key>();
                }
                if (sigmoid && m == __builtin_inff()) {         // its key would be a NaN's
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        if (z[i] == __builtin_inff()) key[i] = key_of(kMost, (i / 8 * L + sub) * 8 + i % 8);
                }
                some = live && !bad && lanes_max<L>(any ? 1.0f : 0.0f) > 0.0f;
            } else {
                some = live && !bad && m > -__builtin_inff();
                m = __builtin_fmaxf(m, -FLT_MAX);
            }
            if (SUMS || !(sigmoid || a.renormalise)) {
                float s[P], lane_sum = 0.0f;         // shares of a softmax, scores of a sigmoid
                if constexpr (PACKED) {
#pragma unroll
                    for (int c = 0; c < C; ++c) unpack<DT>(raw[c], reinterpret_cast<float(&)[8]>(s[c * 8]));
                } else {
#pragma unroll
                    for (int i = 0; i < P; ++i) s[i] = z[i];
                }
                auto score = [](float v) {
                    const float u = exp2_hw(-__builtin_fabsf(v) * static_cast<float>(kLog2E));
                    return (v >= 0.0f ? 1.0f : u) * __builtin_amdgcn_rcpf(1.0f + u);
                };
                const bool low = sigmoid && m < kLow;
                if (__builtin_amdgcn_ballot_w64(low) != 0) {
#pragma unroll
                    for (int i = 0; i < P; ++i) s[i] = low ? low_share(s[i], m) : score(s[i]);
                } else if (sigmoid) {
#pragma unroll
                    for (int i = 0; i < P; ++i) s[i] = score(s[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < P; ++i) s[i] = share_to_fast(s[i], m);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) lane_sum += s[i];
                all = lanes_sum<L>(static_cast<double>(lane_sum));
                part = all > 0.0 ? reciprocal(all) : 0.0;
                if (SUMS) {
                    const float f = some ? static_cast<float>(part) : 0.0f;
#pragma unroll
                    for (int i = 0; i < P; ++i) total[i] = __builtin_fmaf(some ? s[i] : 0.0f, f, total[i]);
                }
            }
        }
        const bool none = !live || bad;

        // groups whose borders are not the chunks': their experts one by one
        const bool by_chunk = width % 8 == 0;
        if (a.groups > 1) {
            wave_fence();
            if (!by_chunk) {
#pragma unroll
                for (int i = 0; i < P; ++i) mine[(i / 8 * L + sub) * 8 + i % 8] = key[i];
            }
        }
        Key list[K];
#pragma unroll
        for (int i = 0; i < K; ++i) list[i] = no_key<Key>();
        auto open_groups = [&](int per, int stride) {
            // group g: `per` places of `stride` keys, the first two of each place its largest
            wave_fence();
            for (int g = sub; g < a.groups; g += L) {
                Key best = no_key<Key>(), next = no_key<Key>();
                for (int i = 0; i < per; ++i) {
                    const Key u = mine[(g * per + i) * stride];
                    next = max_key(next, min_key(best, u));
                    best = max_key(best, u);
                    if (stride > 1) next = max_key(next, mine[(g * per + i) * stride + 1]);
                }
                if constexpr (EXACT) {
                    if (a.group_best == 2 && is_open<DT, Key, true>(best))
                        best = __builtin_bit_cast(
                            double, rounded(key_score(best) + (is_open<DT, Key, true>(next) ? key_score(next) : 0.0)));
                }
                group_of[g] = best;
            }
            wave_fence();
            for (int g = sub; g < a.groups; g += L) {
                const Key own = group_of[g];
                int before = 0;
                for (int o = 0; o < a.groups; ++o) {
                    const Key other = group_of[o];
                    before += other > own || (other == own && o < g);
                }
                open_of[g] = before < a.top_groups;
            }
            wave_fence();
        };
        if (a.groups > 1 && !by_chunk) {
            open_groups(width, 1);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int e = (i / 8 * L + sub) * 8 + i % 8;
                if (!open_of[group_no[e]]) key[i] = no_key<Key>();
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) sort8(reinterpret_cast<Key(&)[8]>(key[c * 8]));
        if (a.groups > 1 && by_chunk) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                mine[(c * L + sub) * 2] = key[c * 8];
                mine[(c * L + sub) * 2 + 1] = key[c * 8 + 1];
            }
            open_groups(width / 8, 2);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = (c * L + sub) * 8;
                if (!open_of[group_no[e]]) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) key[c * 8 + j] = no_key<Key>();
                }
            }
        }
        if constexpr (K == 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) list[i] = key[i];
            if constexpr (C == 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) list[i] = max_key(list[i], key[15 - i]);
                sort_bitonic(list);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) list[i] = key[i];
            if constexpr (C == 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) list[8 + i] = key[15 - i];
                sort_bitonic(list);
            }
        }
        join_lanes<L, K>(list);

        // the chosen ones: lane i (and i + L ..) of a token has the i-th
        double weight[(K + L - 1) / L];
        int expert[(K + L - 1) / L];
        double d = 0.0;
#pragma unroll
        for (int u = 0; u < (K + L - 1) / L; ++u) {
            Key own = no_key<Key>();
#pragma unroll
            for (int i = u * L; i < (u + 1) * L && i < K; ++i)
                if (i == u * L + sub) own = list[i];
            const bool there = !none && u * L + sub < a.top && is_open<DT, Key, EXACT>(own);
            expert[u] = there ? key_expert(own) : -1;
            float ze = 0.0f;
            if (there) ze = widen<DT>(x[expert[u]]);
            weight[u] = there ? score_of(ze, m, sigmoid) : 0.0;
            if (!sigmoid && (EXACT || !a.renormalise)) weight[u] *= part;
            d += weight[u];
        }
        d = lanes_sum<L>(d) + kTiny;
        const double unit = static_cast<double>(a.scale) * (a.renormalise ? reciprocal(d) : 1.0);
        // a softmax of nothing but -inf; without a bias some expert is open else
        const bool nan = live && (bad || (!sigmoid && (EXACT ? !(all > 0.0) : !some)));
#pragma unroll
        for (int u = 0; u < (K + L - 1) / L; ++u) {
            const int i = u * L + sub;
            if (i >= a.top || row >= a.x.rows) continue;
            a.weights[int64_t(row) * a.top + i] = nan ? __builtin_nanf("") : static_cast<float>(weight[u] * unit);
            a.ids[int64_t(row) * a.top + i] = expert[u];
            if (SUMS && expert[u] >= 0) atomicAdd(&count[expert[u]], 1);
        }
        if (SUMS && some && sub == 0) {
            ++tokens;
            if (!sigmoid) {
                const double lse = static_cast<double>(m) + log_sum(all);
                squares += lse * lse;
            }
        }
    }
    if (!SUMS) return;
    // a wave's tokens had the same lanes: their sums, then the waves', in this order
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const double v = tokens_sum<L>(static_cast<double>(total[i]));
        if (slot == 0) reinterpret_cast<double*>(own_space)[(i / 8 * L + sub) * 8 + i % 8] = v;
    }
    squares = lanes_sum<kWave>(squares);
    const double all_tokens = lanes_sum<kWave>(static_cast<double>(tokens));
    if (lane == 0) {
        square[wave] = squares;
        routed[wave] = static_cast<int32_t>(all_tokens);
    }
    __syncthreads();
    double* share = w.share + int64_t(blockIdx.x) * (n + 1);
    int32_t* load = w.load + int64_t(blockIdx.x) * (n + 1);
    for (int e = threadIdx.x; e <= n; e += kRouteThreads) {
        double v = 0.0;
        int32_t c = e < n ? count[e] : 0;
#pragma unroll
        for (int i = 0; i < kRouteWaves; ++i) {
            v += e < n ? reinterpret_cast<const double*>(space + i * space_bytes)[e] : square[i];
            if (e == n) c += routed[i];
        }
        share[e] = v;
        load[e] = c;
    }
}

// The workgroups' sums joined in a fixed order, 16 experts a workgroup (a row of a workgroup's sums is a
// line of 128 bytes).  The last workgroup to be done joins what the balance loss takes of each: a launch
// more would take 4 us.  (A release by few workgroups is cheap; by all those of a large grid it is not.)
constexpr int kFinishThreads = 1024;
constexpr int kFinishExperts = 16;
constexpr int kFinishMost = MP_ROUTE_MAX_EXPERTS / kFinishExperts + 1;

// 512 workgroups' sums of 256 experts: 6.8 us, of 128 workgroups' of 60: 4.6 us; bound by latency.
__global__ __launch_bounds__(kFinishThreads) void k_route_finish(RouteArgs a, RouteSums w)
{
    constexpr int SLICES = kFinishThreads / kFinishExperts, W = kFinishThreads / kWave, U = 4;
    __shared__ double s_part[W][kFinishExperts];
    __shared__ int64_t c_part[W][kFinishExperts], t_part[W];
    const int n = a.x.vocab, blocks = static_cast<int>(gridDim.x);
    const int col = threadIdx.x % kFinishExperts, slice = threadIdx.x / kFinishExperts;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int e = min(static_cast<int>(blockIdx.x) * kFinishExperts + col, n);
    double s = 0.0;
    int64_t c = 0, t = 0;
    for (int from = slice; from < w.groups; from += U * SLICES) {
        double v[U];
        int32_t k[U], r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = min(from + u * SLICES, w.groups - 1);
            v[u] = w.share[int64_t(g) * (n + 1) + e];
            k[u] = w.load[int64_t(g) * (n + 1) + e];
            r[u] = col == 0 ? w.load[int64_t(g) * (n + 1) + n] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (from + u * SLICES >= w.groups) continue;
            s += v[u];
            c += k[u];
            t += r[u];
        }
    }
#pragma unroll
    for (int d = kFinishExperts; d < kWave; d *= 2) {
        s += __shfl_xor(s, d);
        c += __shfl_xor(c, d);
        t += __shfl_xor(t, d);
    }
    if (lane < kFinishExperts) {
        s_part[wave][col] = s;
        c_part[wave][col] = c;
        if (col == 0) t_part[wave] = t;
    }
    __syncthreads();
    if (threadIdx.x >= kWave) return;
    s = 0.0;
    c = t = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        s += s_part[i][col];
        c += c_part[i][col];
        t += t_part[i];
    }
    const bool mine = lane < kFinishExperts && static_cast<int>(blockIdx.x) * kFinishExperts + col <= n;
    const double tokens = static_cast<double>(t), mean = t > 0 ? s / tokens : 0.0;
    if (mine) {
        a.load[e] = c;
        if (e < n && a.share != nullptr) a.share[e] = static_cast<float>(mean);
        if (e == n && a.aux != nullptr) a.aux[1] = static_cast<float>(mean);
    }
    if (a.aux == nullptr) return;
    if (w.groups == 0) {
        if (blockIdx.x == 0 && lane == 0) a.aux[0] = 0.0f;
        return;
    }
    double part = lanes_sum<kWave>(mine && e < n ? static_cast<double>(c) * mean : 0.0);
    int done = 0;
    if (lane == 0) {
        __hip_atomic_store(w.part + blockIdx.x, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        done = __hip_atomic_fetch_add(w.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(done) != blocks - 1) return;
    part = 0.0;
    for (int i = lane; i < blocks; i += kWave)
        part += __hip_atomic_load(w.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    part = lanes_sum<kWave>(part);
    if (lane == 0) a.aux[0] = t > 0 ? static_cast<float>(part * n / (a.top * tokens)) : 0.0f;
}

// With F the factor over the tokens routed, pull_e = F balance E load_e / (k N) and ds the gradient of
// the chosen experts' scores,
//   softmax  dx_e = s_e (pull_e + ds_e - sum_j s_j (pull_j + ds_j) + 2 F z lse)
//   sigmoid  dx_e = s_e (1 - s_e) ((pull_e - sum_j p_j pull_j) / sum s + ds_e),    p = s / sum s.
// (of a token whose logits are all below kLow s and sum s are relative to its largest one's, and ds is scaled instead).
// L lanes per token and P experts a lane, as in the choice.  fp32, a lane's sums over its experts too (nothing here is
// compared), which are joined in binary64.  65536 x 256 bf16 by sigmoid: 26 us, 2.7 TB/s read and written; the vector
// units are at work 71 of 100 cycles, two of 34 instructions an expert being an exponential and a reciprocal.
// At most 128 registers, for four waves a SIMD (one kernel would take 130).
template <int DT, int L, int P, bool SIGMOID>
__global__ __launch_bounds__(kRouteThreads, 4) void k_route_grad(RouteGradArgs a)
{
    using T = typename Fmt<DT>::T;
    constexpr int E = Fmt<DT>::E;
    constexpr int R = kWave / L, C = P / 8, N = L * P;
    constexpr int U = (MP_ROUTE_MAX_TOP + L - 1) / L;          // chosen experts a lane
    __shared__ float extra_of[kRouteWaves][R][N];              // ds by expert; 0 between tokens
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int sub = lane % L, slot = lane / L;
    const int n = a.x.vocab;
    float* const extra = extra_of[wave][slot];
#pragma unroll
    for (int i = 0; i < P; ++i) extra[i * L + sub] = 0.0f;
    double factor = 0.0;
    float pull[P] = {};
    if (a.load != nullptr) {
        const int64_t tokens = read_table(a.load + n);
        factor = tokens > 0 ? grad_factor(a.g) / static_cast<double>(tokens) : 0.0;
        const double unit = factor * static_cast<double>(a.balance) * n / a.top /
                            static_cast<double>(tokens > 0 ? tokens : 1);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = (i / 8 * L + sub) * 8 + i % 8;
            if (e < n) pull[i] = static_cast<float>(unit * static_cast<double>(a.load[e]));
        }
    }
    const double large = 2.0 * factor * static_cast<double>(a.large);
    const int step = static_cast<int>(gridDim.x) * kRouteWaves * R;        // rows are below 2^22
    for (int first = (static_cast<int>(blockIdx.x) * kRouteWaves + wave) * R; first < a.x.rows; first += step) {
        int row = first + slot;
        asm volatile("" : "+v"(row));       // addresses are formed from it, not each kept and stepped
        const bool in = row < a.x.rows;
        const bool live = in && (a.mask == nullptr || a.mask[row] != 0);
        const T* x = static_cast<const T*>(a.x.x) + int64_t(row) * a.x.stride;
        T* dx = static_cast<T*>(a.g.dx) + int64_t(row) * a.g.stride;
        int64_t id[U];
        float dw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = u * L + sub;
            id[u] = live && i < a.top ? a.ids[int64_t(row) * a.top + i] : -1;
            dw[u] = a.dweights != nullptr && id[u] >= 0 ? a.dweights[int64_t(row) * a.top + i] * a.scale : 0.0f;
        }
        float z[P];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (live) load8<DT>(x, (c * L + sub) * 8, n, -__builtin_inff(), z + c * 8);
            else
                for (int j = 0; j < 8; ++j) z[c * 8 + j] = -__builtin_inff();
        }
        float m = -FLT_MAX;
        bool bad = false, any = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            bad |= id[u] >= n;
            if (id[u] >= n) id[u] = -1;
            any |= id[u] >= 0;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            m = __builtin_fmaxf(m, z[i]);
            if (i % 2 == 0) bad |= __builtin_isunordered(z[i], z[i + 1]);
        }
        m = lanes_max<L>(m);
        bad = lanes_max<L>(bad ? 1.0f : 0.0f) > 0.0f || (!SIGMOID && m == __builtin_inff());
        any = lanes_max<L>(any ? 1.0f : 0.0f) > 0.0f;
        float s[P], slope[SIGMOID ? P : 1];        // slope: ds_e / dx_e of a sigmoid
        float lane_sum = 0.0f;
        auto score = [](float v, float& u) {       // a sigmoid, and exp(-|v|) over 1 + that, squared
            const float t = exp2_hw(-__builtin_fabsf(v) * static_cast<float>(kLog2E));
            const float r = __builtin_amdgcn_rcpf(1.0f + t);
            u = t * r * r;
            return v >= 0.0f ? r : t * r;
        };
        const bool low = SIGMOID && live && m < kLow;
        const bool some_low = __builtin_amdgcn_ballot_w64(low) != 0;
        if constexpr (!SIGMOID) {
#pragma unroll
            for (int i = 0; i < P; ++i) s[i] = share_to_fast(z[i], m);
        } else if (some_low) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                s[i] = score(z[i], slope[i]);
                if (low) s[i] = slope[i] = low_share(z[i], m);
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) s[i] = score(z[i], slope[i]);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) lane_sum += s[i];
        const double all = lanes_sum<L>(static_cast<double>(lane_sum));
        const bool nan = live && (bad || (!SIGMOID && !(all > 0.0)));
        const bool on = live && any && !nan;
        const double inverse = all > 0.0 ? reciprocal(all) : 0.0;
        const float part = static_cast<float>(inverse);
        // the chosen experts' scores and their gradient
        double ds[U];
        if (a.renormalise) {
            float ws[U];
            double d = 0.0, mean = 0.0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float unused;
                const float ze = id[u] >= 0 ? widen<DT>(x[id[u]]) : -__builtin_inff();
                if constexpr (SIGMOID) ws[u] = score(ze, unused);
                else ws[u] = share_to_fast(ze, m) * part;
                if (id[u] < 0) ws[u] = 0.0f;
                d += static_cast<double>(ws[u]);
                mean += static_cast<double>(dw[u]) * static_cast<double>(ws[u]);
            }
            d = reciprocal(lanes_sum<L>(d) + kTiny);
            mean = lanes_sum<L>(mean) * d;
#pragma unroll
            for (int u = 0; u < U; ++u) ds[u] = id[u] >= 0 ? (static_cast<double>(dw[u]) - mean) * d : 0.0;
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) ds[u] = static_cast<double>(dw[u]);
        }
        if (some_low) {
            const double down = low ? exp_of(static_cast<double>(m)) : 1.0;      // the scores are relative to it
#pragma unroll
            for (int u = 0; u < U; ++u) ds[u] *= down;
        }
        // each writes its own number where its ds will be: an expert that is there twice shows
        wave_fence();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (id[u] >= 0) extra[id[u]] = __int_as_float(u * L + sub + 1);
        wave_fence();
        bool twice = false;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (id[u] >= 0) twice |= __float_as_int(extra[id[u]]) != u * L + sub + 1;
        wave_fence();
        if (__builtin_amdgcn_ballot_w64(twice) != 0) {
            // its parts add up, in the list's order
            double same[U] = {};
            for (int i = 0; i < a.top; ++i) {
#pragma unroll
                for (int v = 0; v < U; ++v) {
                    if (i / L != v) continue;
                    const int from = slot * L + i % L;
                    const int64_t other = __shfl(id[v], from);
                    const double part_of = __shfl(ds[v], from);
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (other == id[u]) same[u] += part_of;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) ds[u] = same[u];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (id[u] >= 0) extra[id[u]] = static_cast<float>(ds[u]);
        wave_fence();
        float to[P];
        double dot = 0.0;
        {
            float lane_dot = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                to[i] = extra[(i / 8 * L + sub) * 8 + i % 8];
                if constexpr (!SIGMOID) {
                    s[i] *= part;
                    to[i] += pull[i];
                    lane_dot = __builtin_fmaf(s[i], to[i], lane_dot);
                } else {
                    lane_dot = __builtin_fmaf(s[i], pull[i], lane_dot);
                }
            }
            dot = lanes_sum<L>(static_cast<double>(lane_dot));
        }
        wave_fence();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (id[u] >= 0) extra[id[u]] = 0.0f;
        float base;
        if constexpr (SIGMOID) base = static_cast<float>(dot * inverse);
        else base = static_cast<float>((large != 0.0 ? large * (static_cast<double>(m) + log_sum(all)) : 0.0) - dot);
        const float off = nan ? __builtin_nanf("") : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * L + sub) * 8;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = c * 8 + j;
                // (slope * part is below 1; part alone times a pull might leave fp32's range)
                if constexpr (SIGMOID) f[j] = __builtin_fmaf(slope[i] * part, pull[i] - base, slope[i] * to[i]);
                else f[j] = s[i] * (to[i] + base);
                if (!on) f[j] = off;
            }
            if (!in) continue;
            if (e + 8 <= n) {
#pragma unroll
                for (int j = 0; j < 8; j += E)
                    store_vec<DT>(dx + e + j, pack<DT>(reinterpret_cast<const float(&)[E]>(f[j])));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (e + j < n) store_one<DT>(dx + e + j, f[j]);
            }
        }
    }
}

// out = bias + speed sign(mean load - load), one workgroup a layer; a skipped step leaves the bias.
// 256 experts: 4.5 us, a launch and two dependent reads.
__global__ __launch_bounds__(kRouteThreads) void k_route_bias(RouteBiasArgs a)
{
    __shared__ int64_t part[kRouteWaves];
    const int64_t layer = blockIdx.x;
    const int n = a.experts;
    const bool skip = a.skipped != nullptr && *a.skipped != 0;
    auto load_of = [&](int e) {
        int64_t c = 0;
        for (int i = 0; i < a.n_loads; ++i) c += a.load[(int64_t(i) * a.layers + layer) * (n + 1) + e];
        return c;
    };
    int64_t all = 0;
    for (int e = threadIdx.x; e < n; e += kRouteThreads) all += load_of(e);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) all += __shfl_xor(all, d);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = all;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int i = 0; i < kRouteWaves; ++i) all += part[i];
    for (int e = threadIdx.x; e < n; e += kRouteThreads) {
        const int64_t off = all - load_of(e) * n;
        const float step = off == 0 ? 0.0f : off > 0 ? a.speed : -a.speed;
        const float bias = a.bias[layer * n + e];
        a.out[layer * n + e] = skip ? bias : bias + step;            // (-0 + 0 is 0)
    }
}

// Workgroups of a launch over the tokens.
int64_t route_grid(int64_t rows, int lanes, int64_t most)
{
    const int per = kRouteWaves * (kWave / lanes);
    const int64_t grid = (rows + per - 1) / per;
    return grid < most ? grid : most;
}

template <int DT, int L, int P, int K, bool EXACT>
void route_shape(const RouteArgs& a, RouteSums& w, hipStream_t s)
{
    // As many workgroups as are resident at once: a start costs a wave a part of a token's work (131072 x 128
    // bf16 16.1 us, 16.5 with a workgroup for every 32 tokens; 65536 x 256 by a bias in groups 42.5 and 43.9, without
    // groups 35.7 and 35.0), and with sums each leaves its own.
    const bool sums = a.load != nullptr;
    int64_t most = 256 * (sums ? route_waves<DT, L, P, EXACT, true>() : route_waves<DT, L, P, EXACT, false>());
    if (sums)
        most = std::min<int64_t>(most, (MP_ROUTE_WORKSPACE_BYTES - kFinishMost * 8 - 16) / (12 * (int64_t(a.x.vocab) + 1)));
    const int64_t grid = route_grid(a.x.rows, L, most);
    if (a.load != nullptr) {
        w.groups = static_cast<int>(grid);
        w.part = static_cast<double*>(a.workspace);
        w.done = reinterpret_cast<int32_t*>(w.part + kFinishMost);
        w.share = w.part + kFinishMost + 1;
        w.load = reinterpret_cast<int32_t*>(w.share + grid * (a.x.vocab + 1));
    }
    if (grid == 0) return;
    constexpr int R = kWave / L, N = L * P;
    constexpr int key_bytes = EXACT || DT == kFP32 ? 8 : 4;
    int space = 0;
    if (a.groups > 1) space = R * ((group_keys(a.x.vocab, a.groups, N) + a.groups) * key_bytes + a.groups);
    if (sums && space < N * 8) space = N * 8;
    space = (space + 15) / 16 * 16;
    const unsigned blocks = static_cast<unsigned>(grid), bytes = static_cast<unsigned>(space * kRouteWaves);
    if (sums) k_route<DT, L, P, K, EXACT, true><<<blocks, kRouteThreads, bytes, s>>>(a, w, space);
    else k_route<DT, L, P, K, EXACT, false><<<blocks, kRouteThreads, bytes, s>>>(a, w, space);
}

template <int DT, int K, bool EXACT>
void route_key(const RouteArgs& a, RouteSums& w, hipStream_t s)
{
    if (a.x.vocab <= 64) route_shape<DT, 8, 8, K, EXACT>(a, w, s);
    else if (a.x.vocab <= 128) route_shape<DT, 8, 16, K, EXACT>(a, w, s);
    else if (a.x.vocab <= 256) route_shape<DT, 16, 16, K, EXACT>(a, w, s);
    else if (a.x.vocab <= 512) route_shape<DT, 32, 16, K, EXACT>(a, w, s);
    else route_shape<DT, 64, 16, K, EXACT>(a, w, s);
}

template <int DT>
void route_dt(const RouteArgs& a, RouteSums& w, hipStream_t s)
{
    const bool exact = a.bias != nullptr || (a.groups > 1 && a.group_best == 2);
    if (a.top <= 8) exact ? route_key<DT, 8, true>(a, w, s) : route_key<DT, 8, false>(a, w, s);
    else exact ? route_key<DT, 16, true>(a, w, s) : route_key<DT, 16, false>(a, w, s);
}

template <int DT, int L, int P>
void grad_shape(const RouteGradArgs& a, hipStream_t s)
{
    const unsigned grid = static_cast<unsigned>(route_grid(a.x.rows, L, 1024));
    if (a.sigmoid) k_route_grad<DT, L, P, true><<<grid, kRouteThreads, 0, s>>>(a);
    else k_route_grad<DT, L, P, false><<<grid, kRouteThreads, 0, s>>>(a);
}

template <int DT>
void grad_dt(const RouteGradArgs& a, hipStream_t s)
{
    if (a.x.vocab <= 64) grad_shape<DT, 8, 8>(a, s);
    else if (a.x.vocab <= 128) grad_shape<DT, 8, 16>(a, s);
    else if (a.x.vocab <= 256) grad_shape<DT, 16, 16>(a, s);
    else if (a.x.vocab <= 512) grad_shape<DT, 32, 16>(a, s);
    else grad_shape<DT, 64, 16>(a, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s)
{
    RouteSums w{};
    if (dtype == kBF16) route_dt<kBF16>(a, w, s);
    else if (dtype == kFP16) route_dt<kFP16>(a, w, s);
    else route_dt<kFP32>(a, w, s);
    if (a.load != nullptr) {
        const unsigned cols = static_cast<unsigned>(a.x.vocab) / kFinishExperts + 1;
        k_route_finish<<<cols, kFinishThreads, 0, s>>>(a, w);
    }
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, int dtype, hipStream_t s)
{
    if (dtype == kBF16) grad_dt<kBF16>(a, s);
    else if (dtype == kFP16) grad_dt<kFP16>(a, s);
    else grad_dt<kFP32>(a, s);
    return hipGetLastError();
}

hipError_t launch_route_bias(const RouteBiasArgs& a, hipStream_t s)
{
    k_route_bias<<<static_cast<unsigned>(a.layers), kRouteThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace mpk
