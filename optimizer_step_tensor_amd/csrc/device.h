// Device code shared by the update step's kernels (kernels.hip) and the losses'
// (losses.hip): the 16-bit formats, address spaces, table
// reads and the renumbering of workgroups over the XCDs.
#pragma once

#include "internal.h"

namespace mpk {
namespace {

// ---------------------------------------------------------------------------
// 16-bit formats ("Mixed precision, loss scaling, gradient accumulation, and
// activation checkpointing", section 2 "Two 16-bit formats").
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ float widen16(uint32_t h);

template <>
__device__ __forceinline__ float widen16<MP_BF16>(uint32_t h)
{
    return __uint_as_float(h << 16);                     // bf16 is the top half of fp32
}

template <>
__device__ __forceinline__ float widen16<MP_FP16>(uint32_t h)
{
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
}

// Round to nearest, ties to even.  NaN -> the format's quiet NaN, sign kept.
template <int DT>
__device__ __forceinline__ uint32_t round16(float x);

template <>
__device__ __forceinline__ uint32_t round16<MP_BF16>(float x)
{
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return ((u >> 16) & 0x8000u) | 0x7FC0u;
    // Adding 0x7FFF plus the lowest kept bit carries into the kept half exactly
    // when the dropped half is above one half, or equal to it with an odd kept
    // half; a carry out of the largest finite value lands on infinity.
    u += 0x7FFFu + ((u >> 16) & 1u);
    return u >> 16;
}

template <>
__device__ __forceinline__ uint32_t round16<MP_FP16>(float x)
{
    if (x != x) return ((__float_as_uint(x) >> 16) & 0x8000u) | 0x7E00u;
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));   // v_cvt_f16_f32, RNE
}

// Pointers are cast to the global address space so the compiler emits
// global_load/global_store (not flat) instructions.
#define MPK_GLOBAL __attribute__((address_space(1)))

// A read from a table that nothing writes while the pass runs: the plan's chunk
// and tensor tables, a gradset's pointer table, the FP8 output table, a weight
// written by an earlier launch.  Through the constant address space, a load at
// a uniform address becomes one scalar load served by the scalar cache; as a
// plain load in a pass that also stores, the compiler must assume the stores
// may change the table and issues a vector load from every wave instead, all
// of the grid's waves then hitting the same few L2 lines (the accumulations
// ran 3-7% slower reading a device-resident weight that way).
#define MPK_CONST __attribute__((address_space(4)))
// A struct is read as 8-byte words (a struct copy would bind a reference in
// the generic address space and lose the constant one).
template <class T, bool SCALAR = MPK_SCALAR_TABLES>
__device__ __forceinline__ T read_table(const T* p)
{
    if constexpr (!SCALAR) {
        return *p;
    } else if constexpr (sizeof(T) <= 8) {
        return *(const MPK_CONST T*)(p);
    } else {
        static_assert(sizeof(T) % 8 == 0 && alignof(T) >= 8, "a table entry of 8-byte words");
        struct Words {
            uint64_t w[sizeof(T) / 8];
        } x;
        const MPK_CONST uint64_t* q = (const MPK_CONST uint64_t*)(p);
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 8); ++i) x.w[i] = q[i];
        return __builtin_bit_cast(T, x);
    }
}

// The chunk block b of a G-block grid starts at.  Workgroup b runs on XCD
// b mod 8; this renumbering gives each XCD SPAN consecutive chunks per turn of
// 8 * SPAN blocks.  It permutes 0..G-1: blocks of the last, incomplete turn
// keep their own number.
template <int SPAN = MPK_XCD_SPAN>
__device__ __forceinline__ int64_t xcd_first_chunk(int64_t b, int64_t G)
{
    constexpr int64_t span = SPAN;
    constexpr int64_t turn = span * kXcds;
    if (span <= 1 || b >= (G / turn) * turn) return b;
    const int64_t t = b / turn, within = b % turn;
    return t * turn + (within % kXcds) * span + within / kXcds;
}

}  // namespace
}  // namespace mpk
