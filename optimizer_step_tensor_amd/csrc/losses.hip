// HIP kernels of the losses over vocabulary logits, written for CDNA4 (gfx950).
//
// One row of V logits gives, with k = log2(e) / T and m = max_j x_j,
//   s = sum_j exp2((x_j - m) k),   lse = m / T + ln s,   q_j = exp2((x_j - m) k) / s.
// A lane keeps a running (m, s) over its share of the row -- s is rescaled when
// m grows, so the row is read once -- and the shares are joined in binary64 in
// a fixed order.  What a loss needs of the row is then a handful of numbers:
// the target's log-probability (m and ln s enter it apart, so a probability
// near 1 keeps its digits) or the k teacher entries.  The gradient of every loss
// here is dx_j = a q_j, with a few elements (the target, the teacher's ids) that take
// another value: these are stored over the dense ones afterwards.
//
// All of it is bound by HBM: 2 bytes read and 2 written per 16-bit logit
// against about 15 VALU operations.
#include <float.h>

#include "device.h"
#include "losses.h"

namespace mpk {
namespace {

constexpr int kBF16 = MP_BF16, kFP16 = MP_FP16, kFP32 = MP_FP32;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
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
    else return widen16<DT>(h);
}

template <int DT>
__device__ __forceinline__ u32x4 load_vec(const typename Fmt<DT>::T* p)
{
    return *(const MPK_GLOBAL typename Fmt<DT>::Vec*)(p);
}

template <int DT>
__device__ __forceinline__ void store_vec(typename Fmt<DT>::T* p, u32x4 v)
{
    *(MPK_GLOBAL typename Fmt<DT>::Vec*)(p) = v;
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
    else *q = static_cast<uint16_t>(round16<DT>(f));
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

struct Stat {
    float m;
    double s;
};

// Join every lane's share; the result is valid in the first wave, whose lanes
// alone go on to the row's formula.
template <int THREADS>
__device__ __forceinline__ Stat join(const Acc& a, float k_hi, float k_lo)
{
    constexpr int W = THREADS / kWave;
    __shared__ float sm[W];
    __shared__ double ss[W];
    float m = a.m;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d));
    double s = static_cast<double>(a.s * exp2_hw(scaled(a.m, m, k_hi, k_lo)));
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) s += __shfl_xor(s, d);
    if constexpr (W == 1) return Stat{m, s};
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    if (lane == 0) {
        sm[wave] = m;
        ss[wave] = s;
    }
    __syncthreads();
    if (wave != 0) return Stat{m, s};
    m = sm[lane % W];
    s = ss[lane % W];
    float top = m;
#pragma unroll
    for (int d = 1; d < W; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
    s *= exp2_hw(scaled(m, top, k_hi, k_lo));
#pragma unroll
    for (int d = 1; d < W; d <<= 1) s += __shfl_xor(s, d);
    return Stat{top, s};
}

// Sum of one double per lane, valid in all lanes.  Shared memory of its own.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v)
{
    constexpr int W = THREADS / kWave;
    __shared__ double part[W];
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
    if constexpr (W == 1) return v;
    __syncthreads();                     // the last use of part[] is over
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) v += part[i];
    return v;
}

template <int THREADS>
__device__ __forceinline__ float block_max(float v)
{
    constexpr int W = THREADS / kWave;
    __shared__ float part[W];
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v = __builtin_fmaxf(v, __shfl_xor(v, d));
    if constexpr (W == 1) return v;
    __syncthreads();
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) v = __builtin_fmaxf(v, part[i]);
    return v;
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

// exp(d) - d - 1.  Below 1/2 the three terms nearly cancel: there the series
// d^2/2 (1 + d/3 (1 + d/4 (...))), whose first left-out term is below 1e-11 of it.
__device__ __forceinline__ double k3_of(double d)
{
    if (fabs(d) < 0.5) {
        double p = 1.0;
#pragma unroll
        for (int i = 11; i >= 3; --i) p = 1.0 + d * (1.0 / i) * p;
        return 0.5 * d * d * p;
    }
    return exp(d) - d - 1.0;
}

// The row's loss from lp; writes the per-row outputs (lane 0) and returns
// dL/dlp.
__device__ __forceinline__ double target_loss(const LossArgs& a, int64_t row, double w, double lp,
                                              double lse, bool writes)
{
    double loss = 0.0, slope = 0.0, kl = 0.0;
    if (a.kind == kXent) {
        loss = -w * lp;
        slope = -w;
    } else if (a.kind == kPolicy) {
        const double adv = static_cast<double>(read_table(a.advantage + row));
        const double rho = exp(lp - static_cast<double>(read_table(a.old_logp + row)));
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
            const double d = static_cast<double>(read_table(a.ref_logp + row)) - lp;
            kl = k3_of(d);
            const double c = static_cast<double>(a.kl_coef);
            if (c != 0.0) {
                loss += c * kl;
                slope -= c * (kl + d);
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
    for (int i = tid; i < sp.nvec; i += THREADS) store_vec<DT>(dx + sp.head + i * Fmt<DT>::E, z);
    const int e = sp.single(tid);
    if (e >= 0) store_one<DT>(dx + e, 0.0f);
}

__device__ __forceinline__ float teacher_value(const LossArgs& a, int64_t i)
{
    if (a.teacher_dtype == kFP32) return static_cast<const float*>(a.teacher_values)[i];
    const uint16_t h = static_cast<const uint16_t*>(a.teacher_values)[i];
    return a.teacher_dtype == kBF16 ? widen16<kBF16>(h) : widen16<kFP16>(h);
}

// The teacher's side of one row, in shared memory: ids (absent: -1), shares p
// and the student's logits at the ids, taken before any gradient is stored.
struct TeacherRow {
    int32_t* id;
    float* p;
    float* x;
    double mass;        // sum of p
    double cross;       // sum of p (log p - x / T): the loss is this + mass * lse
};

template <int DT, int THREADS>
__device__ __forceinline__ TeacherRow teacher_row(const LossArgs& a, int64_t row,
                                                  const typename Fmt<DT>::T* x, char* lds)
{
    TeacherRow t;
    t.id = reinterpret_cast<int32_t*>(lds);
    t.p = reinterpret_cast<float*>(lds) + a.k;
    t.x = t.p + a.k;
    const int tid = threadIdx.x;
    const int64_t base = row * a.k;
    double norm;
    if (a.teacher_lse != nullptr) {
        norm = static_cast<double>(read_table(a.teacher_lse + row));
    } else {
        float top = -FLT_MAX;
        for (int e = tid; e < a.k; e += THREADS)
            if (a.teacher_ids[base + e] >= 0) top = __builtin_fmaxf(top, teacher_value(a, base + e));
        top = block_max<THREADS>(top);
        double s = 0.0;
        for (int e = tid; e < a.k; e += THREADS)
            if (a.teacher_ids[base + e] >= 0)
                s += exp2_hw(scaled(teacher_value(a, base + e), top, a.x.k_hi, a.x.k_lo));
        norm = static_cast<double>(top) * a.x.inv_t + log_sum(block_sum<THREADS>(s));
    }
    double mass = 0.0, cross = 0.0;
    for (int e = tid; e < a.k; e += THREADS) {
        const int64_t id = a.teacher_ids[base + e];
        float p = 0.0f, xe = 0.0f;
        if (id >= a.x.vocab) {
            mass = cross = __builtin_nan("");
        } else if (id >= 0) {
            const double lp = static_cast<double>(teacher_value(a, base + e)) * a.x.inv_t - norm;
            p = expf(static_cast<float>(lp));
            xe = widen<DT>(x[id]);
            mass += static_cast<double>(p);
            if (p != 0.0f)
                cross += static_cast<double>(p) * (lp - static_cast<double>(xe) * a.x.inv_t);
        }
        t.id[e] = id >= 0 && id < a.x.vocab ? static_cast<int32_t>(id) : -1;
        t.p[e] = p;
        t.x[e] = xe;
    }
    t.mass = block_sum<THREADS>(mass);
    t.cross = block_sum<THREADS>(cross);
    return t;
}

template <int DT, int THREADS>
__device__ __forceinline__ void off_row(const LossArgs& a, int64_t row, typename Fmt<DT>::T* dx)
{
    if (threadIdx.x == 0) {
        if (a.loss != nullptr) a.loss[row] = 0.0f;
        if (a.logp != nullptr) a.logp[row] = 0.0f;
        if (a.lse != nullptr) a.lse[row] = 0.0f;
        if (a.kl != nullptr) a.kl[row] = 0.0f;
    }
    if (dx != nullptr) zero_row<DT, THREADS>(dx, a.x.vocab);
}

// The elements of the teacher's ids: q_id mass - sum of the shares of that id.
// An id that comes twice is stored twice, the same value.  k comparisons per
// entry: for k <= 256 a small part of the row's time.
template <int DT, int THREADS>
__device__ __forceinline__ void store_shares(const TeacherRow& t, int k, typename Fmt<DT>::T* dx,
                                             float m, float k_hi, float k_lo, float c,
                                             float share)
{
    for (int e = threadIdx.x; e < k; e += THREADS) {
        const int id = t.id[e];
        if (id < 0) continue;
        float p = 0.0f;
        for (int i = 0; i < k; ++i) p += t.id[i] == id ? t.p[i] : 0.0f;
        store_one<DT>(dx + id, share_of<DT>(t.x[e], m, k_hi, k_lo) * c - share * p);
    }
}

// What the first wave tells the others: dx_j = c exp2((x_j - m) k), and the
// value of the target's element (or the factor of a teacher's share).
struct RowGrad {
    float m, c, fix;
};

// The row's loss from its statistics: the outputs are written and the gradient's
// numbers broadcast.  Only the first wave holds st; all lanes return the same.
template <int DT, int THREADS, bool DISTILL>
__device__ __forceinline__ RowGrad row_formula(const LossArgs& a, int64_t row, const Stat& st, double w,
                                               int64_t target, float xt, const TeacherRow& t)
{
    __shared__ RowGrad out;
    if (threadIdx.x < kWave) {
        const double ln_s = log_sum(st.s);
        const double lse = static_cast<double>(st.m) * a.x.inv_t + ln_s;
        const double factor = a.g.dx != nullptr ? grad_factor(a.g) : 0.0;
        double mult, fix;
        if constexpr (DISTILL) {
            if (threadIdx.x == 0) a.loss[row] = static_cast<float>(w * (t.cross + t.mass * lse));
            fix = factor * w;
            mult = fix * t.mass;
        } else {
            const double lp = (static_cast<double>(xt) - static_cast<double>(st.m)) * a.x.inv_t - ln_s;
            mult = -factor * target_loss(a, row, w, lp, lse, threadIdx.x == 0);
            if (target >= a.x.vocab) mult = __builtin_nan("");
            fix = mult * expm1(lp);
        }
        if (threadIdx.x == 0)
            out = RowGrad{st.m, static_cast<float>(mult / st.s), static_cast<float>(fix)};
    }
    __syncthreads();      // also: the logits that are needed singly are read, in place is fine
    return out;
}

// The elements that differ from the dense gradient, after all of it is stored.
template <int DT, int THREADS, bool DISTILL>
__device__ __forceinline__ void store_exceptions(const LossArgs& a, const TeacherRow& t, int64_t target,
                                                 typename Fmt<DT>::T* dx, const RowGrad& r)
{
    __syncthreads();
    if constexpr (DISTILL) {
        store_shares<DT, THREADS>(t, a.k, dx, r.m, a.x.k_hi, a.x.k_lo, r.c, r.fix);
    } else {
        if (threadIdx.x == 0 && target < a.x.vocab) store_one<DT>(dx + target, r.fix);
    }
}

// One row per workgroup, any length; the row is read a second time for the
// gradient.
template <int DT, int THREADS, bool DISTILL>
__global__ __launch_bounds__(THREADS) void k_rows(LossArgs a)
{
    using T = typename Fmt<DT>::T;
    constexpr int E = Fmt<DT>::E;
    extern __shared__ char lds[];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    T* dx = a.g.dx != nullptr ? static_cast<T*>(a.g.dx) + row * a.g.stride : nullptr;
    const int64_t target = DISTILL ? 0 : read_table(a.targets + row);
    const double w = a.weights != nullptr ? static_cast<double>(read_table(a.weights + row)) : 1.0;
    if (target < 0 || w == 0.0) return off_row<DT, THREADS>(a, row, dx);
    TeacherRow t;
    if constexpr (DISTILL) {
        t = teacher_row<DT, THREADS>(a, row, x, lds);
        if (t.mass == 0.0) return off_row<DT, THREADS>(a, row, dx);
    }
    const float xt = DISTILL ? 0.0f : target < n ? widen<DT>(x[target]) : __builtin_nanf("");

    const float k_hi = a.x.k_hi, k_lo = a.x.k_lo;
    const Span<DT> sp(dx != nullptr ? static_cast<const void*>(dx) : x, n);
    const int one = sp.single(tid);
    Acc acc;
    float single = 0.0f;
    if (one >= 0) {
        single = widen<DT>(x[one]);
        const float f[1] = {single};
        add(acc, f, k_hi, k_lo);
    }
    for (int i = tid; i < sp.nvec; i += THREADS) {
        float f[E];
        unpack<DT>(load_vec<DT>(x + sp.head + i * E), f);
        add(acc, f, k_hi, k_lo);
    }
    const Stat st = join<THREADS>(acc, k_hi, k_lo);
    const RowGrad r = row_formula<DT, THREADS, DISTILL>(a, row, st, w, target, xt, t);
    if (dx == nullptr) return;
    for (int i = tid; i < sp.nvec; i += THREADS) {
        float f[E];
        unpack<DT>(load_vec<DT>(x + sp.head + i * E), f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = share_of<DT>(f[j], r.m, k_hi, k_lo) * r.c;
        store_vec<DT>(dx + sp.head + i * E, pack<DT>(f));
    }
    if (one >= 0) store_one<DT>(dx + one, share_of<DT>(single, r.m, k_hi, k_lo) * r.c);
    store_exceptions<DT, THREADS, DISTILL>(a, t, target, dx, r);
}

// One row per workgroup, held in registers between the statistics and the
// gradient: NV vectors a lane, the first FULL of them inside the row for every
// lane, all requested before the first is used.
template <int DT, int THREADS, int NV, int FULL, bool DISTILL>
__global__ __launch_bounds__(THREADS) void k_rows_held(LossArgs a)
{
    using T = typename Fmt<DT>::T;
    constexpr int E = Fmt<DT>::E;
    extern __shared__ char lds[];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int n = a.x.vocab;
    const T* x = static_cast<const T*>(a.x.x) + row * a.x.stride;
    T* dx = static_cast<T*>(a.g.dx) + row * a.g.stride;
    const int64_t target = DISTILL ? 0 : read_table(a.targets + row);
    const double w = a.weights != nullptr ? static_cast<double>(read_table(a.weights + row)) : 1.0;
    if (target < 0 || w == 0.0) return off_row<DT, THREADS>(a, row, dx);

    const float k_hi = a.x.k_hi, k_lo = a.x.k_lo;
    const Span<DT> sp(dx, n);
    // lanes past the end take the last vector once more, and drop it when it is used
    u32x4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * THREADS + tid;
        v[i] = load_vec<DT>(x + sp.head + (i < FULL ? e : min(e, sp.nvec - 1)) * E);
    }
    const int one = sp.single(tid);
    float single = one >= 0 ? widen<DT>(x[one]) : -__builtin_inff();
    const float xt = DISTILL ? 0.0f : target < n ? widen<DT>(x[target]) : __builtin_nanf("");
    TeacherRow t;
    if constexpr (DISTILL) {
        t = teacher_row<DT, THREADS>(a, row, x, lds);
        if (t.mass == 0.0) return off_row<DT, THREADS>(a, row, dx);
    }
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
        // the gradient unpacks the vectors again: kept unpacked, they would take twice the registers
        asm("" : "+v"(v[i]), "+v"(v[i + 1]));
    }
    {
        const float f[1] = {single};
        add(acc, f, k_hi, k_lo);
    }
    const Stat st = join<THREADS>(acc, k_hi, k_lo);
    const RowGrad r = row_formula<DT, THREADS, DISTILL>(a, row, st, w, target, xt, t);
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
    store_exceptions<DT, THREADS, DISTILL>(a, t, target, dx, r);
}

// The gradient of log-probabilities from their lse.  With L = lse log2(e) split
// into two floats, log2 q = (x k_hi - L_hi) + (x k_lo - L_lo): the first is one
// fma, whose result is small where q matters; the second only counts for fp32
// results (a 16-bit result is rounded at 2^-9 or 2^-12).
constexpr int kGradThreads = 256;

template <int DT>
__global__ __launch_bounds__(kGradThreads) void k_logprob_grad(LogitsView v, GradView g,
                                                               const int64_t* targets,
                                                               const float* lse, const float* dlogp,
                                                               int chunks, int chunk_vecs)
{
    using T = typename Fmt<DT>::T;
    constexpr int E = Fmt<DT>::E;
    const int64_t row = blockIdx.x / static_cast<unsigned>(chunks);
    const int chunk = static_cast<int>(blockIdx.x % static_cast<unsigned>(chunks));
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
        for (int i = lo + tid; i < hi; i += kGradThreads) store_vec<DT>(dx + sp.head + i * E, z);
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
    for (int i = lo + tid; i < hi; i += kGradThreads) {
        float f[E];
        unpack<DT>(load_vec<DT>(x + sp.head + i * E), f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = q(f[j]) * c;
        store_vec<DT>(dx + sp.head + i * E, pack<DT>(f));
    }
    if (one >= 0) store_one<DT>(dx + one, q(single) * c);
    if (mine) {
        const double lp = static_cast<double>(xt) * v.inv_t - static_cast<double>(read_table(lse + row));
        store_one<DT>(dx + te, static_cast<float>(-slope * expm1(lp)));
    }
}

// One workgroup per pair, in a fixed order: the two sequences' sums, the loss,
// and dlogp of their rows; one more workgroup for the rows outside every sequence.
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
    double pi[2], per[2];
    int64_t begin[2], end[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t seq = pair + i * pairs;
        begin[i] = clamp_row(read_table(a.seq_start + seq), a.rows);
        end[i] = clamp_row(read_table(a.seq_start + seq + 1), a.rows);
        double sum = 0.0, live = 0.0;
        for (int64_t r = begin[i] + tid; r < end[i]; r += kPairThreads) {
            sum += static_cast<double>(a.logp[r]);
            live += a.targets[r] >= 0 ? 1.0 : 0.0;
        }
        sum = block_sum<kPairThreads>(sum);
        per[i] = 1.0;
        if (a.length_mean) {
            live = block_sum<kPairThreads>(live);
            per[i] = live > 0.0 ? 1.0 / live : 0.0;
        }
        pi[i] = sum * per[i];
    }
    double ref[2] = {0.0, 0.0};
    if (a.ref_logp != nullptr) {
        ref[0] = static_cast<double>(read_table(a.ref_logp + pair));
        ref[1] = static_cast<double>(read_table(a.ref_logp + pairs + pair));
    }
    const double delta = (pi[0] - ref[0]) - (pi[1] - ref[1]);
    double loss, slope;                 // dloss/dD
    if (a.kind == MP_PREF_SIGMOID) {
        // -log sigmoid(+-h) = log(1 + exp(-|h|)) + max(-+h, 0)
        const double h = a.beta * delta - a.margin;
        const double u = exp(-fabs(h));
        const double soft = log1p(u);
        loss = soft + (1.0 - a.label_smoothing) * (h < 0.0 ? -h : 0.0) +
               a.label_smoothing * (h > 0.0 ? h : 0.0);
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

constexpr int kCountThreads = 1024;

__global__ __launch_bounds__(kCountThreads) void k_target_count(int64_t n, const int64_t* targets,
                                                                int64_t* count)
{
    __shared__ int64_t part[kCountThreads / kWave];
    int64_t c = 0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += kCountThreads) c += targets[i] >= 0 ? 1 : 0;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) c += __shfl_xor(c, d);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = c;
    __syncthreads();
    if (threadIdx.x == 0) {
        c = 0;
#pragma unroll
        for (int i = 0; i < kCountThreads / kWave; ++i) c += part[i];
        *count = c;
    }
}

constexpr int kRowThreads = 256;

template <int DT, int THREADS, int NV, int FULL>
void held(const LossArgs& a, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(a.x.rows));
    if (a.kind == kDistill)
        k_rows_held<DT, THREADS, NV, FULL, true><<<grid, THREADS, 12u * a.k, s>>>(a);
    else
        k_rows_held<DT, THREADS, NV, FULL, false><<<grid, THREADS, 0, s>>>(a);
}

template <int DT>
void rows_dt(const LossArgs& a, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(a.x.rows));
    // A row has nvec or (its head taken off) nvec - 1 whole vectors: past THREADS * FULL, every
    // lane has FULL of them.
    const int nvec = a.x.vocab / Fmt<DT>::E;
    if (a.g.dx != nullptr && nvec >= 2) {
        if (nvec <= 64 * 4) return held<DT, 64, 4, 0>(a, s);
        if (nvec <= 64 * 8) return held<DT, 64, 8, 4>(a, s);
        if (nvec <= 256 * 4) return held<DT, 256, 4, 2>(a, s);
        if (nvec <= 256 * 8) return held<DT, 256, 8, 4>(a, s);
        if (nvec <= 1024 * 4) return held<DT, 1024, 4, 2>(a, s);
        if (nvec <= 1024 * 6) return held<DT, 1024, 6, 4>(a, s);
        if (nvec <= 1024 * 8) return held<DT, 1024, 8, 6>(a, s);
        if (nvec <= 1024 * 10) return held<DT, 1024, 10, 8>(a, s);
        if (nvec <= 1024 * 12) return held<DT, 1024, 12, 10>(a, s);
        if (nvec <= 1024 * 14) return held<DT, 1024, 14, 12>(a, s);
        if (nvec <= 1024 * 16) return held<DT, 1024, 16, 14>(a, s);
    }
    if (a.kind == kDistill)
        k_rows<DT, kRowThreads, true><<<grid, kRowThreads, 12u * a.k, s>>>(a);
    else
        k_rows<DT, kRowThreads, false><<<grid, kRowThreads, 0, s>>>(a);
}

template <int DT>
void grad_dt(const LogitsView& x, const int64_t* targets, const float* lse, const float* dlogp,
             const GradView& g, hipStream_t s)
{
    // chunks of at least 8 vectors a lane; few enough that the launch stays in range
    const int nvec = x.vocab / Fmt<DT>::E + 1;
    int per = 8 * kGradThreads;
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
