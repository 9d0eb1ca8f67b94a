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
// the others read as 0 and their memory is not touched.
__device__ __forceinline__ u32x4_t load8(const uint16_t* p, int valid)
{
    if (valid >= 8)
        return *reinterpret_cast<const u32x4_a2_t*>(p);
    u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid)
            v[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    return v;
}

__device__ __forceinline__ void store8(uint16_t* p, u32x4_t v, int valid)
{
    if (valid >= 8) {
        *reinterpret_cast<u32x4_a2_t*>(p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid)
            p[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i & 1)));
}

// A bf16 matrix below 2 GiB, read and written 8 elements at a time at 32-bit
// element offsets through bounds-checked buffer accesses (an offset past the
// end reads 0 and writes nothing), without branches between the loads: what a
// lane does not need, it asks for past the end.
//   WHOLE   16-byte aligned with rows a multiple of 8 long: all 8 elements are in
//           a row or none.
//   else    a lane may stand at an odd element; fetch() reads the aligned dwords
//           that hold its elements, and finish() shifts them into place once
//           they are there.  A wave that reaches a row's end (edge, uniform)
//           reads only the dwords with elements of the row, one by one, and
//           clears the rest.  (Single elements under branches made such a
//           wave wait for each: 2048 x 4099, rank 64, 38 us for the expand
//           kernel against 17 us at 4096 columns.)
constexpr uint32_t OOR = 0x80000000u;

template <bool WHOLE>
struct Matrix {
    struct Piece {
        u32x4_t v;
        uint32_t last;      // not WHOLE: the fifth dword
    };
    uint16_t* p;
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t skew;          // bytes from the first dword's start to the first element

    __device__ __forceinline__ Matrix(const uint16_t* base, size_t elements) : p(const_cast<uint16_t*>(base))
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(base);
        skew = WHOLE ? 0u : static_cast<uint32_t>(at) & 2u;
        const size_t bytes = !base ? 0 : WHOLE ? elements * 2 : (skew + elements * 2 + 3) & ~static_cast<size_t>(3);
        rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at - skew), static_cast<short>(0),
                                                 static_cast<int>(bytes), 0x00020000);
    }
    // the first `valid` (any integer) of the 8 elements from `at` on; zeros behind
    __device__ __forceinline__ Piece fetch(uint32_t at, int valid, bool edge) const
    {
        Piece o;
        o.last = 0u;
        if constexpr (WHOLE) {
            o.v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, valid > 0 ? at * 2 : OOR, 0, 0);
        } else {
            const uint32_t from = at * 2 + skew, odd = from & 2u, low = from - odd;
            if (edge) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o.v[i] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, 2 * i - static_cast<int>(odd >> 1) < valid && valid > 0 ? low + 4 * i : OOR, 0, 0);
            } else {
                o.v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, valid > 0 ? low : OOR, 0, 0);
            }
            o.last = __builtin_amdgcn_raw_buffer_load_b32(rsrc, odd && valid >= 8 ? low + 16 : OOR, 0, 0);
        }
        return o;
    }
    __device__ __forceinline__ u32x4_t finish(const Piece& x, uint32_t at, int valid, bool edge) const
    {
        if constexpr (WHOLE) {
            return x.v;
        } else {
            const uint32_t by = ((at * 2 + skew) & 2u) * 8;
            u32x4_t o = {__builtin_amdgcn_alignbit(x.v[1], x.v[0], by), __builtin_amdgcn_alignbit(x.v[2], x.v[1], by),
                         __builtin_amdgcn_alignbit(x.v[3], x.v[2], by), __builtin_amdgcn_alignbit(x.last, x.v[3], by)};
            if (edge) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] &= valid >= 2 * i + 2 ? 0xffffffffu : valid == 2 * i + 1 ? 0xffffu : 0u;
            }
            return o;
        }
    }
    __device__ __forceinline__ void store(uint32_t at, u32x4_t v, int valid, bool edge) const
    {
        if constexpr (WHOLE) {
            __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, valid > 0 ? at * 2 : OOR, 0, 0);
        } else {
            if (edge)
                store8(p + at, v, valid);
            else if (valid > 0)
                *reinterpret_cast<u32x4_a2_t*>(p + at) = v;
        }
    }
};

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

// Between writes and reads of LDS that belongs to one wave, by other lanes than
// wrote: LDS serves a wave's instructions in the order in which they were
// issued, so there is nothing to wait for, and no instruction here; the fences
// keep the compiler from exchanging them.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// A wave's block of 16 rows x 128 bf16, loaded as it lies in memory (lane
// 16 g + c has 16 bytes of row 4 i + g, columns 8 c on: a load covers whole 256-byte
// pieces of rows), turned through LDS of the wave's own into matrix-core
// operands (lane 16 g + c: row c, columns 32 i + 8 g on).  Loaded as operands, 64
// lanes ask for 64 different places, and the vector cache answers one a clock:
// 16 bytes a clock for a CU.
constexpr int TURN_PITCH = 17;                  // 16-byte pieces of a staged row: 16 rows in 64 banks
constexpr int TURN_PIECES = 16 * TURN_PITCH;

__device__ __forceinline__ void turn16(u32x4_t* own, const u32x4_t (&in)[4], u32x4_t (&out)[4])
{
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        own[(4 * i + g) * TURN_PITCH + c] = in[i];
    wave_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = own[c * TURN_PITCH + 4 * i + g];
    wave_sync();
}

// f = hi + mid + lo exactly, each part with the 8 significant bits of a bf16
// (cut, not rounded, so hi cannot overflow; parts below 2^-126 are lost).
// An fp32 factor enters the matrix cores as these three: the products with
// bf16 values are then those of the fp32 factor itself.  An infinity stays whole
// in hi.  A NaN may be cut to an infinity there (a payload in the low half alone),
// but what is left of it is a quiet NaN, which mid holds.
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
            rest = (h[e] & 0x7fffffffu) == 0x7f800000u ? 0.0f : rest;
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

// Values that are kept in bf16 or in fp32 (f32): eight of a row at `at` on, of which the
// first `valid` (any integer) are in the row.
__device__ __forceinline__ void get_values(const void* p, int f32, size_t at, int valid, float (&v)[8])
{
    if (f32) {
        const float* q = static_cast<const float*>(p) + at;
        if (valid >= 8) {
            const f32x4_t a = *reinterpret_cast<const f32x4_a4_t*>(q), b = *reinterpret_cast<const f32x4_a4_t*>(q + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = i < valid ? q[i] : 0.0f;
        }
        return;
    }
    const u32x4_t x = load8(static_cast<const uint16_t*>(p) + at, valid);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = bf16_to_f32(x[i / 2] >> (16 * (i & 1)) & 0xffffu);
}

__device__ __forceinline__ void put_values(void* p, int f32, size_t at, int valid, const float (&v)[8])
{
    if (f32) {
        float* q = static_cast<float*>(p) + at;
        if (valid >= 8) {
            *reinterpret_cast<f32x4_a4_t*>(q) = f32x4_t{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4_a4_t*>(q + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < valid)
                    q[i] = v[i];
        }
        return;
    }
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = f32_to_bf16(v[2 * i]) | f32_to_bf16(v[2 * i + 1]) << 16;
    store8(static_cast<uint16_t*>(p) + at, o, valid);
}

__device__ __forceinline__ void put_value(void* p, int f32, size_t at, float v)
{
    if (f32)
        static_cast<float*>(p)[at] = v;
    else
        static_cast<uint16_t*>(p)[at] = static_cast<uint16_t>(f32_to_bf16(v));
}

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline any4_status launch_status() { return hipGetLastError() == hipSuccess ? ANY4_OK : ANY4_E_HIP; }

}  // namespace
