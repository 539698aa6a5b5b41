// HIP kernels of the losses over vocabulary logits, written for CDNA4 (gfx950).
//
// One row of V logits gives, with k = log2(e) / T and m = max_j x_j,
//   s = sum_j exp2((x_j - m) k),   lse = m / T + ln s,   q_j = exp2((x_j - m) k) / s.
// A lane keeps a running (m, s) over its share of the row -- s is rescaled when
// m grows, so the row is read once -- and the shares are joined in binary64 in
// a fixed order.  What a loss needs of the row is then a handful of numbers:
// the target's log-probability (m and ln s enter it apart: a probability near 1 keeps
// the digits that s has -- a part of 2^-24 that lies in the lane of the row's
// maximum is lost in that lane's fp32 sum, in another lane it counts down to 2^-52)
// or the k teacher entries.  The gradient of every loss
// here is dx_j = a q_j, with a few elements (the target, the teacher's ids) that take
// another value: these are stored over the dense ones afterwards.
//
// All of it is bound by HBM: 2 bytes read and 2 written per 16-bit logit
// against about 15 VALU operations.
#include <float.h>

#include "internal.h"
#include "losses.h"

namespace mpk {
namespace {

// Global pointers become global_load/global_store, not flat instructions; a
// uniform address that nothing writes while the kernel runs (targets, per-row
// inputs, the loss scale, a count) is one scalar load.
#define MPK_GLOBAL __attribute__((address_space(1)))
#define MPK_CONST __attribute__((address_space(4)))

template <class T>
__device__ __forceinline__ T read_table(const T* p)
{
    return *(const MPK_CONST T*)(p);
}

constexpr int kBF16 = MP_BF16, kFP16 = MP_FP16, kFP32 = MP_FP32;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// What a format of logits is: E elements per 16-byte vector, of type T.  Vectors
// are loaded and stored at addresses that are aligned to the element only:
// gfx950's global_load_dwordx4 takes any address (an access that crosses a line
// costs one more line).
typedef u32x4 vec_align2 __attribute__((aligned(2)));
typedef u32x4 vec_align4 __attribute__((aligned(4)));

template <int DT>
struct Fmt {
    using T = uint16_t;
    using Vec = vec_align2;
    static constexpr int E = 8;
};
template <>
struct Fmt<kFP32> {
    using T = float;
    using Vec = vec_align4;
    static constexpr int E = 4;
};

template <int DT>
__device__ __forceinline__ float widen(typename Fmt<DT>::T h)
{
    if constexpr (DT == kFP32) return h;
    else if constexpr (DT == kBF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
    else return static_cast<float>(__builtin_bit_cast(_Float16, h));
}

// Logits that exceed the infinity cache are read past it (NT); smaller ones are
// left where the layer before has just put them and a second pass will look for
// them: LogitsView::stream says which.  Measured, cross-entropy bf16, logits in the
// cache: 2048 x 50304 67 us against 80 with NT loads, 1024 x 50304 37 against 44;
// not in the cache, 4096 x 50304 152 us with NT against 156, statistics of
// 8192 x 128256 318 against 357.
template <int DT, bool NT>
__device__ __forceinline__ u32x4 load_vec(const typename Fmt<DT>::T* p)
{
    const MPK_GLOBAL typename Fmt<DT>::Vec* q = (const MPK_GLOBAL typename Fmt<DT>::Vec*)(p);
    return NT ? __builtin_nontemporal_load(q) : *q;
}

// The gradient is read by another kernel, later, and stored past the caches: 3-10%
// faster than plain stores at every size but the smallest, where they are equal.
template <int DT>
__device__ __forceinline__ void store_vec(typename Fmt<DT>::T* p, u32x4 v)
{
    MPK_GLOBAL typename Fmt<DT>::Vec* q = (MPK_GLOBAL typename Fmt<DT>::Vec*)(p);
    __builtin_nontemporal_store(v, q);
}

template <int DT>
__device__ __forceinline__ void unpack(u32x4 v, float (&f)[Fmt<DT>::E])
{
    if constexpr (DT == kFP32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
    } else if constexpr (DT == kBF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = v[i];      // a bit cast of v[i] itself takes element 0
            const f16x2 h = __builtin_bit_cast(f16x2, u);
            f[2 * i] = static_cast<float>(h.x);
            f[2 * i + 1] = static_cast<float>(h.y);
        }
    }
}

// Round to nearest, ties to even (v_cvt_pk_bf16_f32, v_cvt_pk_f16_f32): at most
// half a step of the output's type, the only rounding below fp32 here.
template <int DT>
__device__ __forceinline__ u32x4 pack(const float (&f)[Fmt<DT>::E])
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == kFP32) {
            v[i] = __float_as_uint(f[i]);
        } else {
            f32x2 t;
            t.x = f[2 * i];
            t.y = f[2 * i + 1];
            if constexpr (DT == kBF16)
                v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(t, bf16x2));
            else
                v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(t, f16x2));
        }
    }
    return v;
}

template <int DT>
__device__ __forceinline__ void store_one(typename Fmt<DT>::T* p, float f)
{
    MPK_GLOBAL typename Fmt<DT>::T* q = (MPK_GLOBAL typename Fmt<DT>::T*)(p);
    if constexpr (DT == kFP32) *q = f;
    else if constexpr (DT == kBF16) *q = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
    else *q = __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}

// How n elements are dealt to lanes: `head` single ones up to the first 16-byte
// boundary of `align` (the array that is written, else the one that is read),
// nvec whole vectors, `tail` single ones.  Lanes 0 .. head-1 take the head and
// lanes E .. E+tail-1 the tail, besides their vectors.
template <int DT>
struct Span {
    int head, nvec, n;

    __device__ __forceinline__ Span(const void* align, int count) : n(count)
    {
        constexpr int E = Fmt<DT>::E;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(align) & 15u);
        head = (off ? 16 - off : 0) / static_cast<int>(sizeof(typename Fmt<DT>::T));
        if (head > n) head = n;
        nvec = (n - head) / E;
    }
    // The element that lane tid takes singly, or -1.
    __device__ __forceinline__ int single(int tid) const
    {
        constexpr int E = Fmt<DT>::E;
        if (tid < head) return tid;
        const int e = head + nvec * E + (tid - E);
        return tid >= E && tid < 2 * E && e < n ? e : -1;
    }
};

__device__ __forceinline__ float exp2_hw(float x)
{
    return __builtin_amdgcn_exp2f(x);   // v_exp_f32: 1 ulp; results below 2^-126 may be 0
}

// A lane's running maximum and sum.  m starts at the lowest finite value, so
// that -inf elements give exp2(-inf) = 0 and never inf - inf.
struct Acc {
    float m = -FLT_MAX;
    float s = 0.0f;
};

// x - m is exact or nearly so; the product with k is corrected by k's own
// rounding error, which would otherwise tilt every probability the same way
// (up to 6e-8 (x - m) / T: it shows in the KL terms).  k_lo > 0, so x = -inf
// gives -inf and not inf - inf.
__device__ __forceinline__ float scaled(float x, float m, float k_hi, float k_lo)
{
    const float t = x - m;
    return __builtin_fmaf(t, k_lo, t * k_hi);
}

// q_j s for a gradient: the correction only counts for fp32 results.
template <int DT>
__device__ __forceinline__ float share_of(float x, float m, float k_hi, float k_lo)
{
    if constexpr (DT == kFP32) return exp2_hw(scaled(x, m, k_hi, k_lo));
    else return exp2_hw((x - m) * k_hi);
}

template <int N>
__device__ __forceinline__ void add(Acc& a, const float (&f)[N], float k_hi, float k_lo)
{
    float g = a.m;
#pragma unroll
    for (int i = 0; i < N; ++i) g = __builtin_fmaxf(g, f[i]);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += exp2_hw(scaled(f[i], g, k_hi, k_lo));
    a.s = a.s * exp2_hw((a.m - g) * k_hi) + s;
    a.m = g;
}

// The largest of a teacher's values v and of the student's logits x at its entries:
// the sums over the entries are formed relative to both.
struct TeacherMax {
    float v = -FLT_MAX;
    float x = -__builtin_inff();
};

struct Stat {
    float m;          // the row's maximum, the sum relative to it
    double s;
    float tm, xm;     // with distillation: the largest v and x of the list, the sums of
    double ts, tc;    // e = exp2((v - tm) k) and e ((v - tm) - (x - xm))
};

// A lane's value and its partner's D lanes away, for reductions whose earlier steps
// have made groups of D lanes alike: within 16 lanes by DPP (the mirrors then
// stand for an exchange of 4 and of 8), beyond by gfx950's row swaps, which give
// both values to all lanes.  A reduction of a wave is some 10 cycles a step this
// way; through the LDS crossbar (ds_bpermute) a step waits over 100.
template <int D>
__device__ __forceinline__ void across(uint32_t v, uint32_t& a, uint32_t& b)
{
    if constexpr (D == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        a = r[0];
        b = r[1];
    } else if constexpr (D == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        a = r[0];
        b = r[1];
    } else {
        constexpr int ctrl = D == 1   ? 0xB1      // quad_perm [1, 0, 3, 2]
                             : D == 2 ? 0x4E      // quad_perm [2, 3, 0, 1]
                             : D == 4 ? 0x141     // row_half_mirror
                                      : 0x140;    // row_mirror
        a = v;
        b = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), ctrl, 0xF, 0xF, true));
    }
}

// Maximum and sum over groups of WIDTH lanes, in all of them.  (The order of the
// two operands differs between lanes, the result does not.)
template <int WIDTH, int D = 1>
__device__ __forceinline__ float lanes_max(float v)
{
    if constexpr (D < WIDTH) {
        uint32_t a, b;
        across<D>(__float_as_uint(v), a, b);
        return lanes_max<WIDTH, 2 * D>(__builtin_fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    return v;
}

template <int WIDTH, int D = 1>
__device__ __forceinline__ double lanes_sum(double v)
{
    if constexpr (D < WIDTH) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        uint32_t a0, b0, a1, b1;
        across<D>(static_cast<uint32_t>(u), a0, b0);
        across<D>(static_cast<uint32_t>(u >> 32), a1, b1);
        const double a = __builtin_bit_cast(double, uint64_t(a1) << 32 | a0);
        const double b = __builtin_bit_cast(double, uint64_t(b1) << 32 | b0);
        return lanes_sum<WIDTH, 2 * D>(a + b);
    }
    return v;
}

// (m, s) joined over groups of WIDTH lanes.
template <int WIDTH>
__device__ __forceinline__ void join_lanes(float& m, double& s, float k_hi, float k_lo)
{
    const float own = m;
    m = lanes_max<WIDTH>(m);
    s = lanes_sum<WIDTH>(s * static_cast<double>(exp2_hw(scaled(own, m, k_hi, k_lo))));
}

// Join every lane's share; the result is valid in the first wave, whose lanes
// alone go on to the row's formula.  The teacher's sums are not formed yet; what the
// lanes have put in shared memory is there for them.
template <int THREADS, bool DISTILL>
__device__ __forceinline__ Stat join(const Acc& a, const TeacherMax& t, float k_hi, float k_lo)
{
    constexpr int W = THREADS / kWave;
    __shared__ float m[3][W];
    __shared__ double s[W];
    Stat r{};
    r.m = a.m;
    r.s = static_cast<double>(a.s);
    join_lanes<kWave>(r.m, r.s, k_hi, k_lo);
    if constexpr (DISTILL) {
        r.tm = lanes_max<kWave>(t.v);
        r.xm = lanes_max<kWave>(t.x);
    }
    if constexpr (W > 1) {
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        if (lane == 0) {
            m[0][wave] = r.m;
            s[wave] = r.s;
            if constexpr (DISTILL) {
                m[1][wave] = r.tm;
                m[2][wave] = r.xm;
            }
        }
        __syncthreads();
        if (wave == 0) {
            r.m = m[0][lane % W];
            r.s = s[lane % W];
            join_lanes<W>(r.m, r.s, k_hi, k_lo);
            if constexpr (DISTILL) {
                r.tm = lanes_max<W>(m[1][lane % W]);
                r.xm = lanes_max<W>(m[2][lane % W]);
            }
        }
    } else if constexpr (DISTILL) {
        __syncthreads();
    }
    return r;
}

// Sums of N doubles per lane, valid in all lanes.
template <int THREADS, int N>
__device__ __forceinline__ void block_sum(double (&v)[N])
{
    constexpr int W = THREADS / kWave;
    __shared__ double part[W][N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = lanes_sum<kWave>(v[i]);
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.0;
#pragma unroll
        for (int j = 0; j < W; ++j) v[i] += part[j][i];
    }
}

// ln s for s > 0 with an absolute error of about 4e-8 + 1e-8: s = 2^e f with f
// in [1/sqrt 2, sqrt 2), ln f in fp32 corrected for the rounding of f.
__device__ __forceinline__ double log_sum(double s)
{
    if (!(s > 0.0) || __builtin_isinf(s)) return s == 0.0 ? -__builtin_inf() : s;
    int e;
    double f = frexp(s, &e);
    if (f < 0.70710678118654752) {
        f *= 2.0;
        --e;
    }
    const float ff = static_cast<float>(f);
    const double rest = (f - static_cast<double>(ff)) / static_cast<double>(ff);
    return e * 0.69314718055994531 + static_cast<double>(logf(ff)) + rest;
}

__device__ __forceinline__ double grad_factor(const GradView& g)
{
    double f = g.scale;
    if (g.dev_scale != nullptr) f *= static_cast<double>(read_table(g.dev_scale));
    if (g.dev_count != nullptr) f /= static_cast<double>(read_table(g.dev_count));
    return f;
}

// exp(d), relative error about 2^-23: the exponent is split in binary64, so its
// size costs nothing, and the fraction's power of two taken in fp32.  (The row
// formulas avoid the library's binary64 functions: their polynomials' constants
// would sit in registers next to a row's data.)
__device__ __forceinline__ double exp_of(double d)
{
    const double y = d * 1.4426950408889634;
    const double whole = __builtin_rint(y < -2000.0 ? -2000.0 : y > 2000.0 ? 2000.0 : y);
    const float part = exp2_hw(static_cast<float>(y - whole));
    return __builtin_ldexp(static_cast<double>(part), static_cast<int>(whole));
}

// exp(d) - d - 1.  Below |d| = 1/2 the terms nearly cancel: there the series
// d^2/2 (1 + d/3 (1 + d/4 (...))), relative error below 2^-22, its first left-out term below
// 2^-27 of it.  From 1/2 on exp's own 2^-23 counts exp(d) / k3 times: 11 times at d = 1/2 (2^-19.5),
// 6 at -1/2, 4 at 1, less farther out.
__device__ __forceinline__ double k3_of(double d)
{
    if (__builtin_fabs(d) < 0.5) {
        const float t = static_cast<float>(d);
        float p = 1.0f;
#pragma unroll
        for (int i = 10; i >= 3; --i) p = __builtin_fmaf(t * (1.0f / i), p, 1.0f);
        return 0.5 * d * d * static_cast<double>(p);
    }
    const double e = exp_of(d);
    return __builtin_isinf(e) ? e : e - d - 1.0;      // d = inf is not inf - inf
}

// exp(d) - 1, with its digits near 0 and without d itself far from it (-1 at d = -inf).
__device__ __forceinline__ double expm1_of(double d)
{
    return __builtin_fabs(d) < 0.5 ? d + k3_of(d) : exp_of(d) - 1.0;
}

// What a row's formula takes besides the logits: requested when the row is, so
// that the first wave does not wait for it between the statistics and the gradient.
struct RowIn {
    int64_t target;
    double w;
    double factor;              // of the gradient
    float advantage, old_logp, ref_logp, teacher_lse;
    // no target, or no weight: nothing of the row is used
    __device__ __forceinline__ bool off() const { return target < 0 || w == 0.0; }
};

template <bool DISTILL>
__device__ __forceinline__ RowIn row_in(const LossArgs& a, int64_t row)
{
    RowIn r{};
    r.w = a.weights != nullptr ? static_cast<double>(read_table(a.weights + row)) : 1.0;
    if constexpr (DISTILL) {
        if (a.teacher_lse != nullptr) r.teacher_lse = read_table(a.teacher_lse + row);
    } else {
        r.target = read_table(a.targets + row);
        if (a.kind == kPolicy) {
            r.advantage = read_table(a.advantage + row);
            r.old_logp = read_table(a.old_logp + row);
            if (a.ref_logp != nullptr) r.ref_logp = read_table(a.ref_logp + row);
        }
    }
    if (a.g.dx != nullptr) r.factor = grad_factor(a.g);
    return r;
}

// The row's loss from lp; writes the per-row outputs (lane 0) and returns
// dL/dlp.
__device__ __forceinline__ double target_loss(const LossArgs& a, int64_t row, const RowIn& in, double lp,
                                              double lse, bool writes)
{
    const double w = in.w;
    double loss = 0.0, slope = 0.0, kl = 0.0;
    if (a.kind == kXent) {
        loss = -w * lp;
        slope = -w;
    } else if (a.kind == kPolicy) {
        const double adv = static_cast<double>(in.advantage);
        const double rho = exp_of(lp - static_cast<double>(in.old_logp));
        const double lo = 1.0 - static_cast<double>(a.clip_low);
        const double hi = 1.0 + static_cast<double>(a.clip_high);
        if (adv != 0.0) {
            const double free = rho * adv;
            const double cut = (rho < lo ? lo : rho > hi ? hi : rho) * adv;
            loss = cut < free ? -cut : -free;          // NaN ends up in loss and slope
            slope = cut < free ? 0.0 : -free;
        } else if (lp != lp) {
            loss = slope = lp;
        }
        if (a.ref_logp != nullptr) {
            const double d = static_cast<double>(in.ref_logp) - lp;
            kl = k3_of(d);
            const double c = static_cast<double>(a.kl_coef);
            if (c != 0.0) {
                loss += c * kl;
                slope -= c * expm1_of(d);      // not kl + d: kl has lost the 1 where d is large
            }
        }
        loss *= w;
        slope *= w;
    }
    if (writes) {
        if (a.loss != nullptr) a.loss[row] = static_cast<float>(loss);
        if (a.logp != nullptr) a.logp[row] = static_cast<float>(lp);
        if (a.lse != nullptr) a.lse[row] = static_cast<float>(lse);
        if (a.kl != nullptr) a.kl[row] = static_cast<float>(kl);
    }
    return slope;
}

// A switched-off row: nothing of it is read, its outputs are 0.
template <int DT, int THREADS>
__device__ __forceinline__ void zero_row(typename Fmt<DT>::T* dx, int n)
{
    const Span<DT> sp(dx, n);
    const u32x4 z = {0u, 0u, 0u, 0u};
    const int tid = threadIdx.x;
    for (int i = tid; i < sp.nvec; i += THREADS)
        store_vec<DT>(dx + sp.head + int64_t(i) * Fmt<DT>::E, z);
    const int e = sp.single(tid);
    if (e >= 0) store_one<DT>(dx + e, 0.0f);
}

// Entry i of the teacher's values, without a branch on their type: the 16-bit
// halves of an fp32 value, or a 16-bit value twice.
__device__ __forceinline__ float teacher_value(const LossArgs& a, int64_t i)
{
    const uint16_t* h = static_cast<const uint16_t*>(a.teacher_values);
    const bool wide = a.teacher_dtype == kFP32;
    h += wide ? 2 * i : i;
    const uint32_t lo = h[0], hi = h[wide ? 1 : 0];
    const float f = __uint_as_float(hi << 16 | (wide ? lo : 0u));      // fp32 and bf16
    return a.teacher_dtype == kFP16 ? widen<kFP16>(static_cast<uint16_t>(lo)) : f;
}

// The teacher's side of one row.  Every lane takes entries tid, tid + THREADS, ..: the first is
// requested apart (`take`), so that its id is there early and the student's logit at it can be
// on its way while the row is read.  ids (absent: -1, past the vocabulary: kPast), values and the
// student's logits end up in shared memory for the sums and the stores over the dense gradient.
template <int DT, int THREADS>
struct TeacherRow {
    using T = typename Fmt<DT>::T;
    static constexpr int kPast = -2;
    const LossArgs& a;
    const T* x;
    int64_t base;
    int32_t* id;
    float* v;
    float* xs;

    __device__ __forceinline__ TeacherRow(const LossArgs& args, int64_t row, const T* logits, char* lds)
        : a(args), x(logits), base(row * args.k), id(reinterpret_cast<int32_t*>(lds)),
          v(reinterpret_cast<float*>(lds) + padded(args.k)), xs(v + padded(args.k))
    {
    }
    // the ids are compared four at a time: up to the next multiple of 4 they are -1
    static __host__ __device__ __forceinline__ int padded(int k) { return (k + 3) & ~3; }
    struct Entry {
        int64_t id;
        float v, x;
    };
    __device__ __forceinline__ Entry take(int e) const
    {
        const int at = min(e, a.k - 1);           // past the end: not put
        return Entry{a.teacher_ids[base + at], teacher_value(a, base + at), 0.0f};
    }
    __device__ __forceinline__ void look_up(Entry& r) const
    {
        r.x = widen<DT>(x[r.id >= 0 && r.id < a.x.vocab ? r.id : 0]);
    }
    __device__ __forceinline__ void put(TeacherMax& top, const Entry& r, int e) const
    {
        if (e >= a.k) {
            if (e < padded(a.k)) id[e] = -1;
            return;
        }
        const bool in = r.id >= 0 && r.id < a.x.vocab;
        id[e] = in ? static_cast<int32_t>(r.id) : r.id < 0 ? -1 : kPast;
        v[e] = r.v;
        xs[e] = r.x;
        if (!in) return;
        top.v = __builtin_fmaxf(top.v, r.v);
        top.x = __builtin_fmaxf(top.x, r.x);
    }
    // The sums over the list, by the lanes of the first wave after `join`: differences of logits
    // in binary64, so that what all of a list have in common (the type's lowest value, at worst)
    // costs nothing.
    __device__ __forceinline__ void sums(Stat& st) const
    {
        if (st.xm == -__builtin_inff()) st.xm = 0.0f;      // the student has none of them: any finite
        const double tm = static_cast<double>(st.tm), xm = static_cast<double>(st.xm);
        double ts = 0.0, tc = 0.0;
        for (int e = threadIdx.x; e < a.k; e += kWave) {
            const int i = id[e];
            if (i == kPast) ts = __builtin_nan("");
            if (i < 0) continue;
            const float p = exp2_hw(scaled(v[e], st.tm, a.x.k_hi, a.x.k_lo));
            const double share = static_cast<double>(p);
            ts += share;
            // a share of 0 adds 0 whatever the student has
            if (p != 0.0f) tc += share * ((static_cast<double>(v[e]) - tm) - (static_cast<double>(xs[e]) - xm));
        }
        st.ts = lanes_sum<kWave>(ts);
        st.tc = lanes_sum<kWave>(tc);
    }
};

__device__ __forceinline__ void off_outputs(const LossArgs& a, int64_t row)
{
    if (threadIdx.x != 0) return;
    if (a.loss != nullptr) a.loss[row] = 0.0f;
    if (a.logp != nullptr) a.logp[row] = 0.0f;
    if (a.lse != nullptr) a.lse[row] = 0.0f;
    if (a.kl != nullptr) a.kl[row] = 0.0f;
}

template <int DT, int THREADS>
__device__ __forceinline__ void off_row(const LossArgs& a, int64_t row, typename Fmt<DT>::T* dx)
{
    off_outputs(a, row);
    if (dx != nullptr) zero_row<DT, THREADS>(dx, a.x.vocab);
}

// What the first wave tells the others: dx_j = c exp2((x_j - m) k), and the
// value of the target's element; with distillation a share is share
// exp2((v - tm) k).  off: no entry has a share, the row counts as switched off.
struct RowGrad {
    float m, c, fix;
    float tm, share;
    int off;
};

// The row's loss from its statistics: the outputs are written (`writes`) and the
// gradient's numbers broadcast.  Only the first wave holds st; all lanes return
// the same.
template <int THREADS, bool DISTILL>
__device__ __forceinline__ RowGrad row_formula(const LossArgs& a, int64_t row, const RowIn& in,
                                               const Stat& st, float xt, bool writes = true)
{
    __shared__ RowGrad out;
    if (threadIdx.x < kWave) {
        const double ln_s = log_sum(st.s);
        const double w = in.w, factor = in.factor;
        double mult;
        RowGrad r{};
        if constexpr (DISTILL) {
            // log p_e = (v_e - tm) / T + at and log q_e = (x_e - xm) / T + log_q, at = -ln ts with the
            // list's own normaliser (the shares sum to 1; a given one scales them all): only
            // differences of logits enter, whatever their size.
            double at = -log_sum(st.ts), one = 1.0 / st.ts;
            if (a.teacher_lse != nullptr) {
                at = static_cast<double>(st.tm) * a.x.inv_t - static_cast<double>(in.teacher_lse);
                one = exp_of(at);
            }
            const double mass = a.teacher_lse != nullptr ? st.ts * one : 1.0;
            r.off = st.ts == 0.0 || mass == 0.0;
            const double log_q =
                (static_cast<double>(st.xm) - static_cast<double>(st.m)) * a.x.inv_t - ln_s;
            const double loss = st.tc * one * a.x.inv_t + mass * (at - log_q);
            if (writes && threadIdx.x == 0) a.loss[row] = static_cast<float>(w * loss);
            mult = factor * w * mass;
            if (!(st.ts >= 0.0)) mult = __builtin_nan("");
            r.tm = st.tm;
            r.share = static_cast<float>(factor * w * one);
        } else {
            const double lse = static_cast<double>(st.m) * a.x.inv_t + ln_s;
            const double lp = (static_cast<double>(xt) - static_cast<double>(st.m)) * a.x.inv_t - ln_s;
            mult = -factor * target_loss(a, row, in, lp, lse, writes && threadIdx.x == 0);
            if (in.target >= a.x.vocab) mult = __builtin_nan("");
            r.fix = static_cast<float>(mult * expm1_of(lp));
        }
        r.m = st.m;
        r.c = static_cast<float>(mult / st.s);
        if (threadIdx.x == 0) out = r;
    }
    __syncthreads();      // also: the logits that are needed singly are read, in place is fine
    return out;
}

// The elements that differ from the dense gradient, after all of it is stored:
// the target's, or each teacher's id's, q_id mass - sum of the shares of that id.
// An id that comes twice is stored twice, the same value.  Every entry is compared
// with all k, four at a time.
template <int DT, int THREADS>
__device__ __forceinline__ void store_shares(const TeacherRow<DT, THREADS>& t, typename Fmt<DT>::T* dx,
                                             const RowGrad& r)
{
    const int k = t.a.k;
    const float k_hi = t.a.x.k_hi, k_lo = t.a.x.k_lo;
    // the values become shares; each lane its own entries
    for (int e = threadIdx.x; e < t.padded(k); e += THREADS)
        t.v[e] = t.id[e] >= 0 ? exp2_hw(scaled(t.v[e], r.tm, k_hi, k_lo)) : 0.0f;
    __syncthreads();
    for (int e = threadIdx.x; e < k; e += THREADS) {
        const int id = t.id[e];
        if (id < 0) continue;
        float p = 0.0f;
#pragma unroll 4
        for (int i = 0; i < k; i += 4) {
            const i32x4 four = *reinterpret_cast<const i32x4*>(t.id + i);
            const f32x4 share = *reinterpret_cast<const f32x4*>(t.v + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) p += four[j] == id ? share[j] : 0.0f;
        }
        store_one<DT>(dx + id, share_of<DT>(t.xs[e], r.m, k_hi, k_lo) * r.c - r.share * p);
    }
}

// The statistics of whole vectors [from, nvec) of a row, 4 requested at a time.
template <int DT, int THREADS, bool NT>
__device__ __forceinline__ void stream_stats(Acc& acc, const typename Fmt<DT>::T* body, int from, int nvec,
                                             float k_hi, float k_lo)
{
    constexpr int E = Fmt<DT>::E, U = 4;
    int i = from + static_cast<int>(threadIdx.x);
    for (; i < nvec - (U - 1) * THREADS; i += U * THREADS) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load_vec<DT, NT>(body + int64_t(i + u * THREADS) * E);
#pragma unroll
        for (int u = 0; u < U; u += 2) {
            float f[2][E];
            unpack<DT>(v[u], f[0]);
            unpack<DT>(v[u + 1], f[1]);
            add(acc, reinterpret_cast<const float(&)[2 * E]>(f), k_hi, k_lo);
        }
    }
    for (; i < nvec; i += THREADS) {
        float f[E];
        unpack<DT>(load_vec<DT, NT>(body + int64_t(i) * E), f);
        add(acc, f, k_hi, k_lo);
    }
}

// The dense gradient of whole vectors [from, nvec) of a row.
template <int DT, int THREADS, bool NT>
__device__ __forceinline__ void stream_grad(const RowGrad& r, const typename Fmt<DT>::T* body,
                                            typename Fmt<DT>::T* dbody, int from, int nvec, float k_hi,
                                            float k_lo)
{
    constexpr int E = Fmt<DT>::E, U = 4;
    auto one = [&](u32x4 v, int i) {
        float f[E];
        unpack<DT>(v, f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = share_of<DT>(f[j], r.m, k_hi, k_lo) * r.c;
        store_vec<DT>(dbody + int64_t(i) * E, pack<DT>(f));
    };
    int i = from + static_cast<int>(threadIdx.x);
    for (; i < nvec - (U - 1) * THREADS; i += U * THREADS) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load_vec<DT, NT>(body + int64_t(i + u * THREADS) * E);
#pragma unroll
        for (int u = 0; u < U; ++u) one(v[u], i + u * THREADS);
    }
    for (; i < nvec; i += THREADS) one(load_vec<DT, NT>(body + int64_t(i) * E), i);
}

// The statistics alone, one row per workgroup.  Bound by HBM reads: 8192 x 128256
// bf16 318 us, 6.6 TB/s; 2048 x 50304 38 us.  128, 512 or 1024 lanes and 2 or 8
// vectors in flight are within 3% there, and slower for few or short rows.
template <int DT, int THREADS, bool DISTILL>
__global__ __launch_bounds__(THREADS) void k_rows_stats(LossArgs a)
{
    using T = typename Fmt<DT>::T;
    extern __shared__ __align__(16) char lds[];
    const int64_t row = blockIdx.x;
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    const RowIn in = row_in<DISTILL>(a, row);
    if (in.off()) return off_row<DT, THREADS>(a, row, nullptr);
    const int64_t target = in.target;
    const TeacherRow<DT, THREADS> t(a, row, x, lds);
    const float xt = DISTILL ? 0.0f : target < n ? widen<DT>(x[target]) : __builtin_nanf("");
    const Span<DT> sp(x, n);
    const int one = sp.single(threadIdx.x);
    Acc acc;
    if (one >= 0) {
        const float f[1] = {widen<DT>(x[one])};
        add(acc, f, a.x.k_hi, a.x.k_lo);
    }
    if (a.x.stream) stream_stats<DT, THREADS, true>(acc, x + sp.head, 0, sp.nvec, a.x.k_hi, a.x.k_lo);
    else stream_stats<DT, THREADS, false>(acc, x + sp.head, 0, sp.nvec, a.x.k_hi, a.x.k_lo);
    TeacherMax top;
    if constexpr (DISTILL) {
        for (int e = threadIdx.x; e < t.padded(a.k); e += THREADS) {
            auto entry = t.take(e);
            t.look_up(entry);
            t.put(top, entry, e);
        }
    }
    Stat st = join<THREADS, DISTILL>(acc, top, a.x.k_hi, a.x.k_lo);
    if (DISTILL && threadIdx.x < kWave) t.sums(st);
    const RowGrad r = row_formula<THREADS, DISTILL>(a, row, in, st, xt);
    if (DISTILL && r.off) off_row<DT, THREADS>(a, row, nullptr);
}

// One row per workgroup, held in registers between the statistics and the
// gradient: NV vectors a lane, the first FULL of them inside the row for every
// lane, all requested before the first is used.  REST: the row goes on past
// them, and that part is read twice.
//
// Bound by HBM, in the pattern of one row per workgroup: 8192 x 128256 bf16, a
// tenth of the rows off, 730 us, 5.5 TB/s (a bare copy in this shape 5.4-5.6; with
// the exponentials left out the time is the same); 4096 x 50304 bf16 152 us, 5.4.
// Reading the row a second time instead took 1185 us; a persistent workgroup that
// requests the next row while it stores this one 880.
template <int DT, int THREADS, int NV, int FULL, bool REST, bool DISTILL>
__global__ __launch_bounds__(THREADS) void k_rows_held(LossArgs a)
{
    using T = typename Fmt<DT>::T;
    constexpr int E = Fmt<DT>::E;
    extern __shared__ __align__(16) char lds[];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    T* dx = static_cast<T*>(a.g.dx) + row * a.g.stride;
    const RowIn in = row_in<DISTILL>(a, row);
    if (in.off()) return off_row<DT, THREADS>(a, row, dx);
    const int64_t target = in.target;

    const float k_hi = a.x.k_hi, k_lo = a.x.k_lo;
    const Span<DT> sp(dx, n);
    const TeacherRow<DT, THREADS> t(a, row, x, lds);
    typename TeacherRow<DT, THREADS>::Entry entry;
    if constexpr (DISTILL) entry = t.take(tid);
    // lanes past the end take the last vector once more, and drop it when it is used
    u32x4 v[NV > 0 ? NV : 1];
    auto at = [&](int i) {
        const int e = i * THREADS + tid;
        return x + sp.head + (i < FULL ? e : min(e, sp.nvec - 1)) * E;
    };
    if (a.x.stream) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = load_vec<DT, true>(at(i));
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = load_vec<DT, false>(at(i));
    }
    const int one = sp.single(tid);
    const float single = one >= 0 ? widen<DT>(x[one]) : -__builtin_inff();
    const float xt = DISTILL ? 0.0f : target < n ? widen<DT>(x[target]) : __builtin_nanf("");
    if constexpr (DISTILL) t.look_up(entry);
    Acc acc;
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
        float f[2 * E];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float g[E];
            unpack<DT>(v[i + h], g);
#pragma unroll
            for (int j = 0; j < E; ++j)
                f[h * E + j] = i + h < FULL || (i + h) * THREADS + tid < sp.nvec ? g[j]
                                                                             : -__builtin_inff();
        }
        add(acc, f, k_hi, k_lo);
        // The gradient unpacks the vectors again: kept unpacked, they would take twice the
        // registers.  The sums stay here, too: moved past the teacher's entries, they would keep
        // a second copy of the vectors alive.
        asm volatile("" : "+v"(v[i]), "+v"(v[i + 1]), "+v"(acc.m), "+v"(acc.s));
    }
    {
        const float f[1] = {single};
        add(acc, f, k_hi, k_lo);
    }
    if constexpr (REST)
        stream_stats<DT, THREADS, false>(acc, x + sp.head, NV * THREADS, sp.nvec, k_hi, k_lo);
    TeacherMax top;
    if constexpr (DISTILL) {
        t.put(top, entry, tid);
        for (int e = tid + THREADS; e < t.padded(a.k); e += THREADS) {
            entry = t.take(e);
            t.look_up(entry);
            t.put(top, entry, e);
        }
    }
    Stat st = join<THREADS, DISTILL>(acc, top, k_hi, k_lo);
    if (DISTILL && tid < kWave) t.sums(st);
    const RowGrad r = row_formula<THREADS, DISTILL>(a, row, in, st, xt);
    if (DISTILL && r.off) return off_row<DT, THREADS>(a, row, dx);
    if constexpr (REST)
        stream_grad<DT, THREADS, true>(r, x + sp.head, dx + sp.head, NV * THREADS, sp.nvec, k_hi, k_lo);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[E];
        unpack<DT>(v[i], f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = share_of<DT>(f[j], r.m, k_hi, k_lo) * r.c;
        if (i < FULL || i * THREADS + tid < sp.nvec)
            store_vec<DT>(dx + sp.head + (i * THREADS + tid) * E, pack<DT>(f));
    }
    if (one >= 0) store_one<DT>(dx + one, share_of<DT>(single, r.m, k_hi, k_lo) * r.c);
    if constexpr (DISTILL) {
        store_shares<DT, THREADS>(t, dx, r);
    } else {
        __syncthreads();                // the dense gradient is stored
        if (tid == 0 && target < n) store_one<DT>(dx + target, r.fix);
    }
}

// Few rows, less than the chip has room for: a row is cut into parts of kPartVecs
// vectors, one workgroup each.  The first launch leaves every part's (m, s) in
// the workspace -- part 0 also takes what is read singly: the ends of the row,
// the target's logit, the teacher's sums, all before any gradient is stored.  In
// the second every workgroup joins its row's parts and stores its part of the
// gradient; part 0 writes the outputs.  Two launches of 3-4 us each for one row of
// 128256 bf16, 6 and 7 us for 61 (against 12 and 20 us as whole rows).
constexpr int kPartThreads = 256;
constexpr int kPartHeld = 4;                              // vectors a lane
constexpr int kPartVecs = kPartThreads * kPartHeld;
constexpr int kMaxParts = kWave;                          // joined by one wave

struct PartSum {
    double s;
    float m;
    float unused;
};

struct PartRow {
    double ts, tc;
    float tm, xm;
    float xt, unused;
};

// Workspace of a split launch: rows * parts PartSum, then rows PartRow.
struct Parts {
    PartSum* sum;
    PartRow* row;
    int parts, vecs;       // per row; vectors of a part
};

template <int DT, bool DISTILL>
__global__ __launch_bounds__(kPartThreads) void k_part_stats(LossArgs a, Parts w)
{
    using T = typename Fmt<DT>::T;
    extern __shared__ __align__(16) char lds[];
    const int64_t row = blockIdx.x / static_cast<unsigned>(w.parts);
    const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(w.parts));
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    const int64_t target = DISTILL ? 0 : read_table(a.targets + row);
    if (target < 0 || (a.weights != nullptr && read_table(a.weights + row) == 0.0f)) return;
    const void* align = a.g.dx != nullptr ? static_cast<const T*>(a.g.dx) + row * a.g.stride : x;
    const Span<DT> sp(align, n);
    const TeacherRow<DT, kPartThreads> t(a, row, x, lds);
    Acc acc;
    TeacherMax top;
    float xt = 0.0f;
    if (part == 0) {
        const int one = sp.single(threadIdx.x);
        if (one >= 0) {
            const float f[1] = {widen<DT>(x[one])};
            add(acc, f, a.x.k_hi, a.x.k_lo);
        }
        if constexpr (DISTILL) {
            for (int e = threadIdx.x; e < a.k; e += kPartThreads) {
                auto entry = t.take(e);
                t.look_up(entry);
                t.put(top, entry, e);
            }
        } else {
            xt = target < n ? widen<DT>(x[target]) : __builtin_nanf("");
        }
    }
    const int lo = part * w.vecs;
    stream_stats<DT, kPartThreads, false>(acc, x + sp.head, lo, min(lo + w.vecs, sp.nvec), a.x.k_hi,
                                          a.x.k_lo);
    Stat st = join<kPartThreads, DISTILL>(acc, top, a.x.k_hi, a.x.k_lo);
    if (DISTILL && part == 0 && threadIdx.x < kWave) t.sums(st);
    if (threadIdx.x == 0) {
        w.sum[row * w.parts + part] = PartSum{st.s, st.m, 0.0f};
        if (part == 0) w.row[row] = PartRow{st.ts, st.tc, st.tm, st.xm, xt, 0.0f};
    }
}

template <int DT, bool DISTILL>
__global__ __launch_bounds__(kPartThreads) void k_part_grad(LossArgs a, Parts w)
{
    using T = typename Fmt<DT>::T;
    constexpr int E = Fmt<DT>::E;
    extern __shared__ __align__(16) char lds[];
    // without a gradient: one workgroup a row, for the outputs
    const unsigned blocks = a.g.dx != nullptr ? w.parts : 1;
    const int64_t row = blockIdx.x / blocks;
    const int part = static_cast<int>(blockIdx.x % blocks);
    const int tid = threadIdx.x;
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    T* dx = a.g.dx != nullptr ? static_cast<T*>(a.g.dx) + row * a.g.stride : nullptr;
    const RowIn in = row_in<DISTILL>(a, row);
    const int64_t target = in.target;
    const float k_hi = a.x.k_hi, k_lo = a.x.k_lo;
    const Span<DT> sp(dx, n);
    const int lo = part * w.vecs, hi = min(lo + w.vecs, sp.nvec);
    const int one = part == 0 ? sp.single(tid) : -1;
    auto zero = [&] {
        if (part == 0) off_outputs(a, row);
        if (dx == nullptr) return;
        const u32x4 z = {0u, 0u, 0u, 0u};
        for (int i = lo + tid; i < hi; i += kPartThreads) store_vec<DT>(dx + sp.head + int64_t(i) * E, z);
        if (one >= 0) store_one<DT>(dx + one, 0.0f);
    };
    if (in.off()) return zero();

    u32x4 v[kPartHeld];
    float single = 0.0f;
    if (dx != nullptr) {
#pragma unroll
        for (int i = 0; i < kPartHeld; ++i)
            v[i] = load_vec<DT, false>(x + sp.head + int64_t(max(min(lo + i * kPartThreads + tid, hi - 1), 0)) * E);
        if (one >= 0) single = widen<DT>(x[one]);
    }
    const TeacherRow<DT, kPartThreads> t(a, row, x, lds);
    if constexpr (DISTILL) {
        if (dx != nullptr) {
            TeacherMax unused;
            for (int e = tid; e < t.padded(a.k); e += kPartThreads) {
                auto entry = t.take(e);
                // the ids that lie in this part: nobody else stores there
                const int64_t at = entry.id - sp.head;
                const bool ends = at < 0 || at >= int64_t(sp.nvec) * E;
                const bool mine = ends ? part == 0 : at >= int64_t(lo) * E && at < int64_t(hi) * E;
                if (!mine || entry.id >= n) entry.id = -1;
                t.look_up(entry);
                t.put(unused, entry, e);
            }
        }
    }
    Stat st{};
    st.m = -FLT_MAX;
    float xt = 0.0f;
    if (tid < kWave) {
        if (tid < w.parts) {
            const PartSum p = w.sum[row * w.parts + tid];
            st.m = p.m;
            st.s = p.s;
        }
        join_lanes<kWave>(st.m, st.s, k_hi, k_lo);
        const PartRow r = w.row[row];
        st.tm = r.tm;
        st.xm = r.xm;
        st.ts = r.ts;
        st.tc = r.tc;
        xt = r.xt;
    }
    const RowGrad r = row_formula<kPartThreads, DISTILL>(a, row, in, st, xt, part == 0);
    if (DISTILL && r.off) return zero();
    if (dx == nullptr) return;
#pragma unroll
    for (int i = 0; i < kPartHeld; ++i) {
        float f[E];
        unpack<DT>(v[i], f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = share_of<DT>(f[j], r.m, k_hi, k_lo) * r.c;
        const int at = lo + i * kPartThreads + tid;
        if (at < hi) store_vec<DT>(dx + sp.head + int64_t(at) * E, pack<DT>(f));
    }
    stream_grad<DT, kPartThreads, false>(r, x + sp.head, dx + sp.head, lo + kPartVecs, hi, k_hi, k_lo);
    if (one >= 0) store_one<DT>(dx + one, share_of<DT>(single, r.m, k_hi, k_lo) * r.c);
    if constexpr (DISTILL) {
        store_shares<DT, kPartThreads>(t, dx, r);
    } else {
        const int64_t at = target - sp.head;
        const bool ends = at < 0 || at >= int64_t(sp.nvec) * E;
        const bool mine = ends ? part == 0 : at >= int64_t(lo) * E && at < int64_t(hi) * E;
        __syncthreads();                // this part of the dense gradient is stored
        if (mine && tid == 0 && target < n) store_one<DT>(dx + target, r.fix);
    }
}

// The gradient of log-probabilities from their lse.  With L = lse log2(e) split
// into two floats, log2 q = (x k_hi - L_hi) + (x k_lo - L_lo): the first is one
// fma, whose result is small where q matters; the second is left out for 16-bit
// results: it is at most 1.8e-7 of lse, and they are rounded at 2^-8 or 2^-11.
constexpr int kGradThreads = 256;
constexpr int kGradSpan = 64;       // consecutive chunks an XCD takes

// Workgroup b of G runs on XCD b mod 8: this renumbering gives each XCD runs of
// kGradSpan consecutive chunks (the last, incomplete turn keeps its numbers).
__device__ __forceinline__ unsigned xcd_chunk(unsigned b, unsigned G)
{
    constexpr unsigned turn = kGradSpan * kXcds;
    if (b >= G / turn * turn) return b;
    const unsigned t = b / turn, within = b % turn;
    return t * turn + within % kXcds * kGradSpan + within / kXcds;
}

template <int DT>
__global__ __launch_bounds__(kGradThreads) void k_logprob_grad(LogitsView v, GradView g,
                                                               const int64_t* targets,
                                                               const float* lse, const float* dlogp,
                                                               int chunks, int chunk_vecs)
{
    using T = typename Fmt<DT>::T;
    constexpr int E = Fmt<DT>::E;
    const unsigned block = xcd_chunk(blockIdx.x, gridDim.x);
    const int64_t row = block / static_cast<unsigned>(chunks);
    const int chunk = static_cast<int>(block % static_cast<unsigned>(chunks));
    const int tid = threadIdx.x;
    const int n = v.vocab;
    const T* x = static_cast<const T*>(v.x) + row * v.stride;
    T* dx = static_cast<T*>(g.dx) + row * g.stride;
    const Span<DT> sp(dx, n);
    const int lo = chunk * chunk_vecs;
    const int hi = min(lo + chunk_vecs, sp.nvec);
    const int one = chunk == 0 ? sp.single(tid) : -1;
    const int64_t target = read_table(targets + row);
    const float d = read_table(dlogp + row);
    if (target < 0 || d == 0.0f) {
        const u32x4 z = {0u, 0u, 0u, 0u};
        for (int i = lo + tid; i < hi; i += kGradThreads)
            store_vec<DT>(dx + sp.head + int64_t(i) * E, z);
        if (one >= 0) store_one<DT>(dx + one, 0.0f);
        return;
    }
    const double slope = grad_factor(g) * static_cast<double>(d);
    const float c = target < n ? static_cast<float>(-slope) : __builtin_nanf("");
    const double l2 = static_cast<double>(read_table(lse + row)) * 1.4426950408889634;
    const float l_hi = static_cast<float>(l2);
    const float l_lo = __builtin_isinf(l_hi) ? 0.0f : static_cast<float>(l2 - static_cast<double>(l_hi));
    auto q = [&](float f) {
        float y = __builtin_fmaf(f, v.k_hi, -l_hi);
        if constexpr (DT == kFP32) y += __builtin_fmaf(f, v.k_lo, -l_lo);
        return exp2_hw(y);
    };
    // the target's element belongs to one lane: it stores it over its own vector
    const int te = target < n ? static_cast<int>(target) : -1;
    bool mine = false;
    float xt = 0.0f;
    if (te >= 0) {
        const int tv = te < sp.head ? -1 : (te - sp.head) / E;
        mine = tv >= 0 && tv < sp.nvec ? (tv >= lo && tv < hi && (tv - lo) % kGradThreads == tid)
                                       : one == te;
        if (mine) xt = widen<DT>(x[te]);
    }
    float single = one >= 0 ? widen<DT>(x[one]) : 0.0f;
    auto vec = [&](u32x4 raw, int i) {
        float f[E];
        unpack<DT>(raw, f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = q(f[j]) * c;
        store_vec<DT>(dx + sp.head + int64_t(i) * E, pack<DT>(f));
    };
    if (v.stream) {
        for (int i = lo + tid; i < hi; i += kGradThreads)
            vec(load_vec<DT, true>(x + sp.head + int64_t(i) * E), i);
    } else {
        for (int i = lo + tid; i < hi; i += kGradThreads)
            vec(load_vec<DT, false>(x + sp.head + int64_t(i) * E), i);
    }
    if (one >= 0) store_one<DT>(dx + one, q(single) * c);
    if (mine) {
        const double lp = static_cast<double>(xt) * v.inv_t - static_cast<double>(read_table(lse + row));
        store_one<DT>(dx + te, static_cast<float>(-slope * expm1_of(lp)));
    }
}

// One workgroup per pair, in a fixed order: the two sequences' sums, the loss,
// and dlogp of their rows; one more workgroup for the rows outside every sequence.
// A launch's time and two memory latencies: 4-5 us for 8 pairs of 256 rows.
constexpr int kPairThreads = 256;

__device__ __forceinline__ int64_t clamp_row(int64_t r, int64_t rows)
{
    return r < 0 ? 0 : r > rows ? rows : r;
}

__global__ __launch_bounds__(kPairThreads) void k_pairs(PairArgs a)
{
    const int tid = threadIdx.x;
    const int64_t pair = blockIdx.x, pairs = a.n_pairs;
    if (pair == pairs) {
        const int64_t first = clamp_row(read_table(a.seq_start), a.rows);
        const int64_t last = clamp_row(read_table(a.seq_start + 2 * pairs), a.rows);
        for (int64_t r = tid; r < first; r += kPairThreads) a.dlogp[r] = 0.0f;
        for (int64_t r = last + tid; r < a.rows; r += kPairThreads) a.dlogp[r] = 0.0f;
        return;
    }
    // sums of lp and counts of targets of the chosen and the rejected sequence, reduced together
    double v[4] = {0.0, 0.0, 0.0, 0.0};
    int64_t begin[2], end[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t seq = pair + i * pairs;
        begin[i] = clamp_row(read_table(a.seq_start + seq), a.rows);
        end[i] = clamp_row(read_table(a.seq_start + seq + 1), a.rows);
#pragma unroll 4
        for (int64_t r = begin[i] + tid; r < end[i]; r += kPairThreads) {
            v[2 * i] += static_cast<double>(a.logp[r]);
            v[2 * i + 1] += a.targets[r] >= 0 ? 1.0 : 0.0;
        }
    }
    block_sum<kPairThreads>(v);
    double pi[2], per[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        per[i] = !a.length_mean ? 1.0 : v[2 * i + 1] > 0.0 ? 1.0 / v[2 * i + 1] : 0.0;
        pi[i] = v[2 * i] * per[i];
    }
    double ref[2] = {0.0, 0.0};
    if (a.ref_logp != nullptr) {
        ref[0] = static_cast<double>(read_table(a.ref_logp + pair));
        ref[1] = static_cast<double>(read_table(a.ref_logp + pairs + pair));
    }
    const double delta = (pi[0] - ref[0]) - (pi[1] - ref[1]);
    double loss, slope;                 // dloss/dD
    if (a.kind == MP_PREF_SIGMOID) {
        // -log sigmoid(+-h) = log(1 + exp(-|h|)) + max(-+h, 0), the latter with weight 1 - eps below
        // h = 0 and eps above; no weight leaves it out, infinite (a sequence of probability 0) or not
        const double h = a.beta * delta - a.margin;
        const double u = exp(-fabs(h));
        const double weight = h < 0.0 ? 1.0 - a.label_smoothing : a.label_smoothing;
        loss = log1p(u) + (weight != 0.0 ? weight * fabs(h) : 0.0);
        const double sig_neg = h >= 0.0 ? u / (1.0 + u) : 1.0 / (1.0 + u);    // sigmoid(-h)
        slope = a.beta * (a.label_smoothing * (1.0 - sig_neg) - (1.0 - a.label_smoothing) * sig_neg);
    } else {
        const double off = delta - 0.5 / a.beta;
        loss = off * off;
        slope = 2.0 * off;
    }
    if (tid == 0) {
        a.loss[pair] = static_cast<float>(loss);
        a.seq_logp[pair] = static_cast<float>(pi[0]);
        a.seq_logp[pairs + pair] = static_cast<float>(pi[1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float d = static_cast<float>((i == 0 ? slope : -slope) * per[i]);
        for (int64_t r = begin[i] + tid; r < end[i]; r += kPairThreads)
            a.dlogp[r] = a.targets[r] >= 0 ? d : 0.0f;
    }
}

// One workgroup, so that the count needs no cleared memory: 2-4 us for 8192
// targets, a launch's time.
constexpr int kCountThreads = 1024;

__global__ __launch_bounds__(kCountThreads) void k_target_count(int64_t n, const int64_t* targets,
                                                                int64_t* count)
{
    __shared__ int64_t part[kCountThreads / kWave];
    int64_t c = 0;
    // a ballot per wave and 64 targets, 8 requested at a time; lanes past n take the last one again
    for (int64_t from = 0; from < n; from += 8 * kCountThreads) {
        int64_t t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t i = from + u * kCountThreads + threadIdx.x;
            t[u] = targets[i < n ? i : n - 1];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool in = from + u * kCountThreads + threadIdx.x < n;
            c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(in && t[u] >= 0));
        }
    }
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = c;
    __syncthreads();
    if (threadIdx.x == 0) {
        c = 0;
#pragma unroll
        for (int i = 0; i < kCountThreads / kWave; ++i) c += part[i];
        *count = c;
    }
}

unsigned teacher_lds(const LossArgs& a)
{
    return 12u * static_cast<unsigned>(TeacherRow<kBF16, 64>::padded(a.k));
}

template <int DT, int THREADS, int NV, int FULL, bool REST = false>
void held(const LossArgs& a, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(a.x.rows));
    if (a.kind == kDistill)
        k_rows_held<DT, THREADS, NV, FULL, REST, true><<<grid, THREADS, teacher_lds(a), s>>>(a);
    else
        k_rows_held<DT, THREADS, NV, FULL, REST, false><<<grid, THREADS, 0, s>>>(a);
}

template <int DT, int THREADS>
void stats(const LossArgs& a, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(a.x.rows));
    if (a.kind == kDistill)
        k_rows_stats<DT, THREADS, true><<<grid, THREADS, teacher_lds(a), s>>>(a);
    else
        k_rows_stats<DT, THREADS, false><<<grid, THREADS, 0, s>>>(a);
}

// Split the rows over several workgroups?  Fills `w` in the workspace if so.
// A whole row takes a workgroup's own time (cross-entropy with gradient, bf16:
// 8.1 us for 20000 logits, 11.8 for 50304, 19.3 for 128256, up to about 100 rows
// alike); its parts take 10 us however long the row and grow with the rows, being
// read twice.  Split against whole: 128256 logits, 1 row 10.7 us against 19.3, 61
// rows 15.1 against 20.7, 100 rows 19.3 against 21.5, 192 rows 31.4 against 25.1;
// 50304 logits, 1 row 10.4 against 11.8, 100 rows 13.8 against 13.4; 20000 logits,
// 1 row 9.6 against 8.1; 60000 fp32 logits, 1 row 10.2 against 12.3, 32 rows 12.5
// against 13.1, 100 rows 17.8 against 15.2.
template <int DT>
constexpr int kSplitRows = Fmt<DT>::E == 8 ? 100 : 40;
constexpr int kSplitVocab = 48 * 1024;

template <int DT>
bool split(const LossArgs& a, Parts* w)
{
    const int nvec = a.x.vocab / Fmt<DT>::E;
    if (a.workspace == nullptr || a.x.rows > kSplitRows<DT> || a.x.vocab < kSplitVocab) return false;
    int vecs = kPartVecs;
    while ((nvec + vecs - 1) / vecs > kMaxParts) vecs += kPartVecs;
    w->vecs = vecs;
    w->parts = (nvec + vecs - 1) / vecs;
    const size_t sums = sizeof(PartSum) * a.x.rows * w->parts;
    if (sums + sizeof(PartRow) * a.x.rows > MP_LOSS_WORKSPACE_BYTES) return false;
    w->sum = static_cast<PartSum*>(a.workspace);
    w->row = reinterpret_cast<PartRow*>(static_cast<char*>(a.workspace) + sums);
    return true;
}

constexpr int64_t kCacheBytes = int64_t(256) << 20;      // the infinity cache of an MI355X

template <int DT>
int64_t logits_bytes(const LogitsView& x)
{
    return int64_t(x.rows) * x.vocab * static_cast<int64_t>(sizeof(typename Fmt<DT>::T));
}

template <int DT>
void rows_dt(LossArgs a, hipStream_t s)
{
    a.x.stream = logits_bytes<DT>(a.x) > kCacheBytes;
    Parts w;
    if (split<DT>(a, &w)) {
        const unsigned rows = static_cast<unsigned>(a.x.rows);
        const dim3 all(rows * w.parts), grid(a.g.dx != nullptr ? rows * w.parts : rows);
        if (a.kind == kDistill) {
            k_part_stats<DT, true><<<all, kPartThreads, teacher_lds(a), s>>>(a, w);
            k_part_grad<DT, true><<<grid, kPartThreads, teacher_lds(a), s>>>(a, w);
        } else {
            k_part_stats<DT, false><<<all, kPartThreads, 0, s>>>(a, w);
            k_part_grad<DT, false><<<grid, kPartThreads, 0, s>>>(a, w);
        }
        return;
    }
    // A row has nvec or (its head taken off) nvec - 1 whole vectors: past THREADS * FULL, every
    // lane has FULL of them.  Below 2 there may be none.
    const int nvec = a.x.vocab / Fmt<DT>::E;
    if (a.g.dx == nullptr)
        return nvec <= 64 * 8 && (a.kind != kDistill || a.k <= 64) ? stats<DT, 64>(a, s)
                                                                   : stats<DT, 256>(a, s);
    if (nvec < 2) return held<DT, 64, 0, 0, true>(a, s);
    // a wave a row, unless a teacher's list needs more lanes: 30 rows of 3551 with 201 entries
    // 40 us with one wave, 8 us with four
    if (a.kind == kDistill && a.k > 64 && nvec <= 256 * 4) return held<DT, 256, 4, 0>(a, s);
    // (a lane's vectors past the row's end still take their arithmetic: 16384 x 1000 bf16 20.5 us
    // with 2 vectors a lane, 24.5 with 4; 16384 x 10000 124 us with 6, 131 with 8)
    if (nvec <= 64 * 2) return held<DT, 64, 2, 0>(a, s);
    if (nvec <= 64 * 4) return held<DT, 64, 4, 2>(a, s);
    if (nvec <= 64 * 8) return held<DT, 64, 8, 4>(a, s);
    if (nvec <= 256 * 4) return held<DT, 256, 4, 2>(a, s);
    if (nvec <= 256 * 6) return held<DT, 256, 6, 4>(a, s);
    if (nvec <= 256 * 8) return held<DT, 256, 8, 6>(a, s);
    // Up to 64 K (fp32: 32 K) logits, where two rows fit a compute unit.  16-bit logits have twice
    // the arithmetic per byte and gain from the smaller workgroup, whose waves wait less for each
    // other: 8192 x 20000 bf16 124 us against 137 with 1024 lanes, distillation over 4096 x
    // 50304 fp16 178 against 204.  fp32 loses: 4096 x 16000 95 us against 92.
    if constexpr (Fmt<DT>::E == 8) {
        if (nvec <= 512 * 6) return held<DT, 512, 6, 4>(a, s);
        if (nvec <= 512 * 8) return held<DT, 512, 8, 6>(a, s);
        if (nvec <= 512 * 10) return held<DT, 512, 10, 8>(a, s);
        if (nvec <= 512 * 12) return held<DT, 512, 12, 10>(a, s);
        if (nvec <= 512 * 14) return held<DT, 512, 14, 12>(a, s);
        if (nvec <= 512 * 16) return held<DT, 512, 16, 14>(a, s);
    } else {
        if (nvec <= 1024 * 4) return held<DT, 1024, 4, 2>(a, s);
        if (nvec <= 1024 * 6) return held<DT, 1024, 6, 4>(a, s);
        if (nvec <= 1024 * 8) return held<DT, 1024, 8, 6>(a, s);
    }
    if (nvec <= 1024 * 10) return held<DT, 1024, 10, 8>(a, s);
    if (nvec <= 1024 * 12) return held<DT, 1024, 12, 10>(a, s);
    if (nvec <= 1024 * 14) return held<DT, 1024, 14, 12>(a, s);
    if (nvec <= 1024 * 16) return held<DT, 1024, 16, 14>(a, s);
    if (nvec <= 1024 * 20) return held<DT, 1024, 20, 16>(a, s);
    held<DT, 1024, 16, 16, true>(a, s);
}

template <int DT>
void grad_dt(LogitsView x, const int64_t* targets, const float* lse, const float* dlogp,
             const GradView& g, hipStream_t s)
{
    // Here the pass before has read the logits, and read all of them: past half the cache little of
    // them is left.  Statistics and gradient of 2048 x 50304 bf16 (206 MB): 102 us with NT loads
    // against 116 where they came from memory, 118 against 113 where they started in the cache;
    // 1024 x 50304: 64 against 62, and 63 against 61.
    x.stream = logits_bytes<DT>(x) > kCacheBytes / 2;
    // Chunks of 2 vectors a lane, runs of 64 of them on an XCD: what is in flight is then one
    // compact piece of memory (pass over 3087 x 128256 bf16 with a third of the rows off: 207 us,
    // 6.5 TB/s; 8 vectors 246 us; without the runs 216 us).  More where the launch would get too large.
    const int nvec = x.vocab / Fmt<DT>::E + 1;
    int per = 2 * kGradThreads;
    while (static_cast<int64_t>((nvec + per - 1) / per) * x.rows > (int64_t(1) << 23)) per *= 2;
    const int chunks = (nvec + per - 1) / per;
    k_logprob_grad<DT><<<static_cast<unsigned>(chunks) * static_cast<unsigned>(x.rows), kGradThreads,
                         0, s>>>(x, g, targets, lse, dlogp, chunks, per);
}

}  // namespace

hipError_t launch_target_count(int64_t n, const int64_t* targets, int64_t* count, hipStream_t s)
{
    k_target_count<<<1, kCountThreads, 0, s>>>(n, targets, count);
    return hipGetLastError();
}

hipError_t launch_rows(const LossArgs& a, int dtype, hipStream_t s)
{
    if (dtype == kBF16) rows_dt<kBF16>(a, s);
    else if (dtype == kFP16) rows_dt<kFP16>(a, s);
    else rows_dt<kFP32>(a, s);
    return hipGetLastError();
}

hipError_t launch_logprob_grad(const LogitsView& x, const int64_t* targets, const float* lse,
                               const float* dlogp, const GradView& g, int dtype, hipStream_t s)
{
    if (dtype == kBF16) grad_dt<kBF16>(x, targets, lse, dlogp, g, s);
    else if (dtype == kFP16) grad_dt<kFP16>(x, targets, lse, dlogp, g, s);
    else grad_dt<kFP32>(x, targets, lse, dlogp, g, s);
    return hipGetLastError();
}

hipError_t launch_pairs(const PairArgs& a, hipStream_t s)
{
    k_pairs<<<static_cast<unsigned>(a.n_pairs + 1), kPairThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace mpk
