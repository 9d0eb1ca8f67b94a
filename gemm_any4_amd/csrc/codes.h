// A quantised layer's weights in registers, shared by the kernels that decode
// packed codes beside a product (gemm_dx.hip, ffn.hip).
#pragma once

#include "frag.h"

namespace {

enum { FMT_ANY4, FMT_INT4, FMT_ANY2, FMT_ANY3 };

// ---------------------------------------------------------------------------
// a row's weights
// ---------------------------------------------------------------------------
// The row's table lies in registers as bytes, low and high halves apart, and
// v_perm looks four codes up at a time.
// The slot of row n, k 128 * chunk + 32 * quarter + 0 .. 31.
template <int FMT>
__device__ __forceinline__ void fetch_codes(const uint8_t* packed, int n, int Kc, int chunk, int quarter, uint32_t (&code)[4])
{
    constexpr int BYTES = FMT == FMT_ANY2 ? 8 : FMT == FMT_ANY3 ? 12 : 16;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        packed + ((static_cast<size_t>(n / 16) * Kc + chunk) * 64 + quarter * 16 + n % 16) * BYTES);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        code[i] = i < BYTES / 4 ? src[i] : 0u;
}

// A row's table, and its scale and offset for 128 k.
struct RowTable {
    u32x4_t table[2];
    uint32_t alpha, beta;
};

template <int FMT>
__device__ __forceinline__ RowTable fetch_table(const uint16_t* lut, const uint16_t* alpha, const uint16_t* beta, int n, int Kc,
                                                int chunk, int g)
{
    RowTable r;
    r.table[0] = r.table[1] = u32x4_t{0u, 0u, 0u, 0u};
    const size_t grp = static_cast<size_t>(n) * (Kc * 128 / g) + chunk * 128 / g;
    r.alpha = alpha[grp];
    r.beta = beta[grp];
    if constexpr (FMT != FMT_INT4) {
        typedef u32x4_t __attribute__((aligned(2))) table_t;
        const table_t* l = reinterpret_cast<const table_t*>(lut + static_cast<size_t>(n) * 16);
        r.table[0] = l[0];
        if constexpr (FMT == FMT_ANY4)
            r.table[1] = l[1];
    }
    return r;
}

// The row's weights for each code, as bytes: lo[i / 4] holds the low bytes of
// codes i .. i + 3, hi their high bytes.  (Scaling and rounding the table's 4 to
// 16 entries costs less than doing so for each of the 32 weights.)
template <int FMT>
struct ByteTable {
    static constexpr int ENTRIES = FMT == FMT_ANY2 ? 4 : FMT == FMT_ANY3 ? 8 : 16;
    uint32_t lo[ENTRIES / 4], hi[ENTRIES / 4];

    ByteTable() = default;
    __device__ __forceinline__ explicit ByteTable(const RowTable& r)
    {
        const float a = bf16_to_f32(r.alpha), b = bf16_to_f32(r.beta);
        uint32_t v[ENTRIES / 2];
#pragma unroll
        for (int i = 0; i < ENTRIES / 2; ++i) {
            const uint32_t e = r.table[i / 4][i % 4];
            const float x = FMT == FMT_INT4 ? static_cast<float>(2 * i) : __uint_as_float(e << 16);
            const float y = FMT == FMT_INT4 ? static_cast<float>(2 * i + 1) : __uint_as_float(e & 0xffff0000u);
            v[i] = f32_to_bf16(fmaf(a, x, b)) | f32_to_bf16(fmaf(a, y, b)) << 16;
        }
#pragma unroll
        for (int i = 0; i < ENTRIES / 4; ++i) {
            lo[i] = __builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], 0x06040200u);
            hi[i] = __builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], 0x07050301u);
        }
    }
    // The weights of the four codes in the bytes of s: (s0, s1) and (s2, s3).
    __device__ __forceinline__ void find(uint32_t s, uint32_t& v01, uint32_t& v23) const
    {
        uint32_t l, h;
        if constexpr (FMT == FMT_ANY2) {
            l = __builtin_amdgcn_perm(0u, lo[0], s);
            h = __builtin_amdgcn_perm(0u, hi[0], s);
        } else if constexpr (FMT == FMT_ANY3) {
            l = __builtin_amdgcn_perm(lo[1], lo[0], s);
            h = __builtin_amdgcn_perm(hi[1], hi[0], s);
        } else {
            const uint32_t low3 = s & 0x07070707u;
            const uint32_t upper = __builtin_amdgcn_perm(0u, 0xff00u, s >> 3 & 0x01010101u);      // 0xff where the code is 8 .. 15
            l = (__builtin_amdgcn_perm(lo[1], lo[0], low3) & ~upper) | (__builtin_amdgcn_perm(lo[3], lo[2], low3) & upper);
            h = (__builtin_amdgcn_perm(hi[1], hi[0], low3) & ~upper) | (__builtin_amdgcn_perm(hi[3], hi[2], low3) & upper);
        }
        v01 = __builtin_amdgcn_perm(h, l, 0x05010400u);
        v23 = __builtin_amdgcn_perm(h, l, 0x07030602u);
    }
};

// The 32 weights of a row's slot, as bf16: of each eight k, out holds (0, 2),
// (4, 6), (1, 3) and (5, 7): first_k(i) and two on.
__device__ __forceinline__ constexpr int first_k(int i) { return 8 * (i / 4) + 4 * (i & 1) + (i >> 1 & 1); }

template <int FMT>
__device__ __forceinline__ void decode(const ByteTable<FMT>& t, const uint32_t (&code)[4], uint32_t (&out)[16])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t even, odd;      // the codes of the eight's even and odd k, one a byte
        if constexpr (FMT == FMT_ANY2) {
            const uint32_t w = code[i / 2] >> (16 * (i % 2));     // two bits each
            even = (w & 3u) | (w & 0x30u) << 4 | (w & 0x300u) << 8 | (w & 0x3000u) << 12;
            odd = (w >> 2 & 3u) | (w >> 2 & 0x30u) << 4 | (w >> 2 & 0x300u) << 8 | (w >> 2 & 0x3000u) << 12;
        } else if constexpr (FMT == FMT_ANY3) {
            // four pairs of six bits; the last four from the bytes' top bits
            const uint32_t w = i < 3 ? code[i < 3 ? i : 0]
                                     : (code[0] >> 6 & 0x03030303u) | (code[1] >> 4 & 0x0c0c0c0cu) | (code[2] >> 2 & 0x30303030u);
            even = w & 0x07070707u;
            odd = w >> 3 & 0x07070707u;
        } else {
            even = code[i] & 0x0f0f0f0fu;
            odd = code[i] >> 4 & 0x0f0f0f0fu;
        }
        t.find(even, out[4 * i], out[4 * i + 1]);
        t.find(odd, out[4 * i + 2], out[4 * i + 3]);
    }
}

// The same weights in order, eight at a time: out holds (8i, 8i + 1) .. (8i + 6, 8i + 7).
// The codes' bytes are laid out in pairs before the lookup, and which half of a
// 16-entry table a code is in comes from its top bit by v_perm's selectors 8 .. 11 (the
// sign of every other byte as a whole byte): 26 instructions for eight weights (27
// above, not in order).
template <int FMT>
__device__ __forceinline__ void decode8(const ByteTable<FMT>& t, const uint32_t (&code)[4], int i, uint32_t (&out)[4])
{
    if constexpr (FMT == FMT_ANY2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {            // k % 4 below 2, and the others
            const uint32_t w = code[i / 2] >> (4 * j), even = w & 0x03030303u, odd = w >> 2 & 0x03030303u;
            const uint32_t s = __builtin_amdgcn_perm(odd, even, i % 2 ? 0x07030602u : 0x05010400u);
            const uint32_t l = __builtin_amdgcn_perm(0u, t.lo[0], s), h = __builtin_amdgcn_perm(0u, t.hi[0], s);
            out[j] = __builtin_amdgcn_perm(h, l, 0x05010400u);
            out[2 + j] = __builtin_amdgcn_perm(h, l, 0x07030602u);
        }
    } else if constexpr (FMT == FMT_ANY3) {
        const uint32_t w = i < 3 ? code[i < 3 ? i : 0]
                                 : (code[0] >> 6 & 0x03030303u) | (code[1] >> 4 & 0x0c0c0c0cu) | (code[2] >> 2 & 0x30303030u);
        const uint32_t even = w & 0x07070707u, odd = w >> 3 & 0x07070707u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t s = __builtin_amdgcn_perm(odd, even, j ? 0x07030602u : 0x05010400u);
            const uint32_t l = __builtin_amdgcn_perm(t.lo[1], t.lo[0], s), h = __builtin_amdgcn_perm(t.hi[1], t.hi[0], s);
            out[2 * j] = __builtin_amdgcn_perm(h, l, 0x05010400u);
            out[2 * j + 1] = __builtin_amdgcn_perm(h, l, 0x07030602u);
        }
    } else {
        const uint32_t w = code[i], even = w & 0x07070707u, odd = w >> 4 & 0x07070707u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {            // codes (0, 1, 4, 5), (2, 3, 6, 7)
            const uint32_t s = __builtin_amdgcn_perm(odd, even, j ? 0x07030501u : 0x06020400u);
            const uint32_t upper = j ? __builtin_amdgcn_perm(w, w << 4, 0x0b090a08u) : __builtin_amdgcn_perm(w << 8, w << 12, 0x0b090a08u);
            const uint32_t l = (__builtin_amdgcn_perm(t.lo[1], t.lo[0], s) & ~upper) | (__builtin_amdgcn_perm(t.lo[3], t.lo[2], s) & upper);
            const uint32_t h = (__builtin_amdgcn_perm(t.hi[1], t.hi[0], s) & ~upper) | (__builtin_amdgcn_perm(t.hi[3], t.hi[2], s) & upper);
            out[j] = __builtin_amdgcn_perm(h, l, 0x05010400u);
            out[2 + j] = __builtin_amdgcn_perm(h, l, 0x07030602u);
        }
    }
}

template <int FMT>
__device__ __forceinline__ void decode_in_order(const ByteTable<FMT>& t, const uint32_t (&code)[4], uint32_t (&out)[16])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v[4];
        decode8(t, code, i, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            out[4 * i + j] = v[j];
    }
}

// Neighbouring lanes hold rows n and n + 1 of the same k: the pair of rows for
// first_k(i) (even lanes) or two k on (odd lanes).
__device__ __forceinline__ uint32_t pair_rows(uint32_t v, bool odd)
{
    const uint32_t other = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xf, 0xf, true));
    return __builtin_amdgcn_perm(other, v, odd ? 0x03020706u : 0x05040100u);     // one instruction, its selector kept
}

// 16 bytes a lane from the buffer to 1 KB of LDS, lane after lane.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint16_t* to, int at, int step)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, at, step, 0, 0);
}

// dy with rows padded to Np by zeros, where its own rows are not whole steps
// of aligned 16-byte pieces.
__global__ __launch_bounds__(256) void k_pad_rows(const uint16_t* __restrict__ dy, uint16_t* __restrict__ out, int N, int Np,
                                                  size_t pieces)
{
    const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
    if (i >= pieces)
        return;
    const int per = Np / 8;
    const size_t m = i / per;
    const int n = static_cast<int>(i % per) * 8;
    reinterpret_cast<u32x4_t*>(out)[i] = load8(dy + m * N + n, N - n);
}

}  // namespace
