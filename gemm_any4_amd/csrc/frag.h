// Small device pieces shared by the adapter, 8-bit activation and input
// gradient kernels: 16-byte accesses at any 2-byte alignment, matrix-core
// operands, and fp32 values as sums of three bf16 parts.
#pragma once

#include <hip/hip_runtime.h>

#include "any4.h"

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
// the same 16 bytes where only the elements are aligned (rows of an odd
// number of bf16 or fp32 values): one load or store all the same
typedef u32x4_t u32x4_a2_t __attribute__((aligned(2)));
typedef f32x4_t f32x4_a4_t __attribute__((aligned(4)));

constexpr int WAVE = 64;

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

__device__ __forceinline__ uint32_t f32_to_bf16(float f)
{
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));   // nearest even
}

// 8 bf16 at p, of which only the first `valid` (any integer) are in the row:
// the others read as 0 and their memory is not touched.  WHOLE: the row is a
// multiple of 8 long, so that all 8 are in it or none.
template <bool WHOLE = false>
__device__ __forceinline__ u32x4_t load8(const uint16_t* p, int valid)
{
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (WHOLE ? valid > 0 : valid >= 8)
        return *reinterpret_cast<const u32x4_a2_t*>(p);
    if constexpr (WHOLE)
        return v;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid)
            v[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    return v;
}

template <bool WHOLE = false>
__device__ __forceinline__ void store8(uint16_t* p, u32x4_t v, int valid)
{
    if (WHOLE ? valid > 0 : valid >= 8) {
        *reinterpret_cast<u32x4_a2_t*>(p) = v;
        return;
    }
    if constexpr (WHOLE)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid)
            p[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i & 1)));
}

// Column t of the 8 x 8 block whose row u is R[u] (8 bf16): the 8 values a
// lane gives the matrix cores along the summed dimension.
template <int t>
__device__ __forceinline__ bf16x8_t column(const u32x4_t (&R)[8])
{
    constexpr uint32_t sel = t & 1 ? 0x07060302u : 0x05040100u;
    u32x4_t f;
#pragma unroll
    for (int p = 0; p < 4; ++p)
        f[p] = __builtin_amdgcn_perm(R[2 * p + 1][t / 2], R[2 * p][t / 2], sel);
    return __builtin_bit_cast(bf16x8_t, f);
}

__device__ __forceinline__ f32x4_t mfma(bf16x8_t a, bf16x8_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// f = hi + mid + lo exactly, each part with the 8 significant bits of a bf16
// (cut, not rounded, so hi cannot overflow; parts below 2^-126 are lost).
// An fp32 factor enters the matrix cores as these three: the products with
// bf16 values are then those of the fp32 factor itself.  An infinity or NaN
// stays whole in hi.
struct Split3 {
    bf16x8_t part[3];
};

__device__ __forceinline__ Split3 split3(const float (&f)[8])
{
    u32x4_t hi, mid, lo;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        uint32_t h[2], m[2], l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float v = f[2 * p + e];
            h[e] = __float_as_uint(v);
            float rest = v - __uint_as_float(h[e] & 0xffff0000u);
            rest = (h[e] & 0x7f800000u) == 0x7f800000u ? 0.0f : rest;
            m[e] = __float_as_uint(rest);
            l[e] = __float_as_uint(rest - __uint_as_float(m[e] & 0xffff0000u));
        }
        hi[p] = __builtin_amdgcn_perm(h[1], h[0], 0x07060302u);
        mid[p] = __builtin_amdgcn_perm(m[1], m[0], 0x07060302u);
        lo[p] = __builtin_amdgcn_perm(l[1], l[0], 0x07060302u);
    }
    return {{__builtin_bit_cast(bf16x8_t, hi), __builtin_bit_cast(bf16x8_t, mid),
             __builtin_bit_cast(bf16x8_t, lo)}};
}

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline any4_status launch_status() { return hipGetLastError() == hipSuccess ? ANY4_OK : ANY4_E_HIP; }

}  // namespace
