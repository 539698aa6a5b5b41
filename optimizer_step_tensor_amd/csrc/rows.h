// What the kernels over rows of logits share (losses.hip, scores.hip, routing.hip):
// formats and their vectors, reductions over lanes, the functions of row formulas.
#pragma once

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

constexpr int64_t kCacheBytes = int64_t(256) << 20;      // the infinity cache of an MI355X

template <int DT>
int64_t logits_bytes(const LogitsView& x)
{
    return int64_t(x.rows) * x.vocab * static_cast<int64_t>(sizeof(typename Fmt<DT>::T));
}

}  // namespace
}  // namespace mpk
