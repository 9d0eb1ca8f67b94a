// dx = dy * W, the gradient of a quantised layer's input (W [N][K] in any4,
// plain int4, any2 or any3).  The C ABI is declared in include/any4.h.
//
//     dx[m][k] = sum_n dy[m][n] w[n][k],   w the any4_dequant values (bf16)
//
// The sum runs over the rows of W, while a packed tile holds 16 rows x 128 k
// with each row's k together.  So the layer is first dequantised and turned,
// W^T [K][N] (k_dequant_t), which makes the product one of two matrices whose
// summed dimension is contiguous (k_dx).
#include "frag.h"

namespace {

enum { FMT_ANY4, FMT_INT4, FMT_ANY2, FMT_ANY3 };

constexpr int STEP = 64;             // n of one step of the product; W^T rows are padded to it

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

// Neighbouring lanes hold rows n and n + 1 of the same k: the pair of rows for
// first_k(i) (even lanes) or two k on (odd lanes).
__device__ __forceinline__ uint32_t pair_rows(uint32_t v, bool odd)
{
    const uint32_t other = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xf, 0xf, true));
    return __builtin_amdgcn_perm(other, v, odd ? 0x03020706u : 0x05040100u);     // one instruction, its selector kept
}

// ---------------------------------------------------------------------------
// W^T
// ---------------------------------------------------------------------------
constexpr int DT_THREADS = 256;
constexpr int DT_STRIDE = 36;                          // dwords of a staged row of 64 n
constexpr int DT_QUARTER = 32 * DT_STRIDE + 16;        // of 32 such rows: the four quarters' writes in other banks

// A workgroup turns 64 rows x 128 k: each wave decodes one packed tile (a lane
// the 32 k of one row), neighbouring lanes pair up their rows' values, and
// the block leaves through LDS as 128-byte pieces of W^T's rows.  Bound by its
// writes (14336 x 4096: 29 MB read, 117 MB written).
template <int FMT>
__global__ __launch_bounds__(DT_THREADS) void k_dequant_t(const uint8_t* __restrict__ packed,
                                                          const uint16_t* __restrict__ lut,
                                                          const uint16_t* __restrict__ alpha,
                                                          const uint16_t* __restrict__ beta,
                                                          uint16_t* __restrict__ wt, int N, int K, int g, int Np)
{
    __shared__ __attribute__((aligned(16))) uint32_t turned[4 * DT_QUARTER];
    const int Kc = K / 128, c = blockIdx.x % Kc, n0 = blockIdx.x / Kc * 64;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, j = lane & 15, kq = lane >> 4;
    const int n = n0 + 16 * w + j;
    uint32_t out[16] = {};                  // rows behind the last: weights of 0
    if (n < N) {
        uint32_t code[4];
        fetch_codes<FMT>(packed, n, Kc, c, kq, code);
        decode(ByteTable<FMT>(fetch_table<FMT>(lut, alpha, beta, n, Kc, c, g)), code, out);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        turned[kq * DT_QUARTER + (first_k(i) + 2 * (j & 1)) * DT_STRIDE + 8 * w + j / 2] = pair_rows(out[i], j & 1);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = tid + DT_THREADS * i, k = q / 8, e = q % 8;
        *reinterpret_cast<u32x4_t*>(wt + static_cast<size_t>(c * 128 + k) * Np + n0 + 8 * e) =
            *reinterpret_cast<const u32x4_t*>(&turned[k / 32 * DT_QUARTER + k % 32 * DT_STRIDE + 4 * e]);
    }
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

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------
// A workgroup takes BM rows of dy x BN rows of W^T, 64 n a step; each wave has
// 16*RM x 16*RN of the outputs.  Both tiles go to LDS by direct loads, the next
// step's while this one is multiplied: one barrier a step.  Bound by the matrix
// cores and the LDS reads that feed them (a wave's 128 x 64 outputs: 12 reads of
// 1 KB for 32 products); 4096 x 14336 x 4096 takes 368 us, 1307 TFLOP/s (the median
// launch; the fastest 350, averages of whole runs 373 to 414; 128 x 128 tiles of
// four 64 x 64 waves: 645 us).  A row of a tile is eight 16-byte pieces; piece q
// stands at q ^ key(row), keys chosen so that the 16 lanes of an operand read
// touch all 64 banks once.
struct DxArgs {
    const uint16_t* dy;     // [M][Np]
    const uint16_t* wt;     // [K][Np]
    uint16_t* dx;           // [M][K]
    float* part;            // [S][M][K] or null (S = 1)
    int M, K, Np, S;
};

// rows of dy are read as operands 16 in a row; rows of W^T by row_of()
__device__ __forceinline__ int key_dy(int r) { return r >> 1 & 7; }
__device__ __forceinline__ int key_wt(int r) { return (r >> 1 & 1) | (r >> 4 & 3) << 1; }
// row of W^T (of 64) that operand t's lane row rho holds: a lane's outputs are
// then 16 adjacent k
__device__ __forceinline__ int row_of(int t, int rho) { return 16 * (rho >> 2) + 4 * t + (rho & 3); }

// 16 bytes a lane from the buffer to 1 KB of LDS, lane after lane.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint16_t* to, int at, int step)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, at, step, 0, 0);
}

// WM x WN waves of RM x 4 blocks of 16 x 16.
template <int WM, int WN, int RM>
__global__ __launch_bounds__(64 * WM * WN) void k_dx(const DxArgs p)
{
    constexpr int BM = WM * RM * 16, BN = WN * 64, WAVES = WM * WN;
    constexpr int LA = BM / 8 / WAVES, LB = BN / 8 / WAVES;      // load instructions of a wave a step
    // two buffers of their own each, so that loads into one are known not to
    // touch reads of the other
    __shared__ __attribute__((aligned(16))) uint16_t sa0[BM * STEP], sb0[BN * STEP], sa1[BM * STEP], sb1[BN * STEP];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, g = lane >> 4;
    const int tiles_k = p.K / BN, tiles_m = (p.M + BM - 1) / BM, tiles = tiles_k * tiles_m;
    // workgroups go to the eight XCDs in turn: each XCD gets a run of tiles, four
    // rows of tiles high, whose operands its L2 then shares
    int id = blockIdx.x;
    if (tiles % 8 == 0)
        id = id % 8 * (tiles / 8) + id / 8;
    constexpr int HIGH = 4;
    const int band = id / (HIGH * tiles_k), high = tiles_m - band * HIGH < HIGH ? tiles_m - band * HIGH : HIGH;
    const int in_band = id - band * HIGH * tiles_k;
    const int m0 = (band * HIGH + in_band % high) * BM, k0 = in_band / high * BN;
    const int steps = p.Np / STEP;
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * blockIdx.y / p.S);
    const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (blockIdx.y + 1) / p.S);

    // a wave's load instruction fills 8 rows of a tile; lane: row lane / 8, place
    // lane % 8.  Rows behind the last read as 0.
    const size_t pitch = static_cast<size_t>(p.Np) * 2;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(p.dy) + m0 * static_cast<size_t>(p.Np), static_cast<short>(0),
        static_cast<int>((p.M - m0 < BM ? p.M - m0 : BM) * pitch), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(p.wt) + k0 * static_cast<size_t>(p.Np), static_cast<short>(0), static_cast<int>(BN * pitch), 0x00020000);
    int ga[LA], gb[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int r = (w * LA + i) * 8 + lane / 8;
        ga[i] = static_cast<int>(r * pitch) + ((lane & 7) ^ key_dy(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int r = (w * LB + i) * 8 + lane / 8;
        gb[i] = static_cast<int>(r * pitch) + ((lane & 7) ^ key_wt(r)) * 16;
    }
    auto fetch = [&](int st, uint16_t* sa, uint16_t* sb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LA; ++i)
            load_lds(ra, sa + (w * LA + i) * 8 * STEP, ga[i], st * STEP * 2);
#pragma unroll
        for (int i = 0; i < LB; ++i)
            load_lds(rb, sb + (w * LB + i) * 8 * STEP, gb[i], st * STEP * 2);
    };
    f32x4_t acc[RM][4];     // [rows of dy][rows of W^T]
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
            acc[i][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int wm = (w / WN) * (RM * 16), wk = (w % WN) * 64;
    // operand reads: 16 rows of dy on, or 4 of W^T, the key is the same, so one
    // address each and constant distances; the second half of a step is four
    // pieces on, bit 2 of the piece
    const int oa = (wm + c) * STEP, ob = (wk + row_of(0, c)) * STEP;
    const int pa = g ^ key_dy(wm + c), pb = g ^ key_wt(wk + row_of(0, c));
    auto multiply = [&](const uint16_t* sa, const uint16_t* sb) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            bf16x8_t a[RM], b[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                b[t] = *reinterpret_cast<const bf16x8_t*>(sb + ob + (pb ^ 4 * kk) * 8 + 4 * t * STEP);
#pragma unroll
            for (int i = 0; i < RM; ++i)
                a[i] = *reinterpret_cast<const bf16x8_t*>(sa + oa + (pa ^ 4 * kk) * 8 + 16 * i * STEP);
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc[i][t] = mfma(b[t], a[i], acc[i][t]);
        }
    };
    // this step's tiles are in, and every wave has read the other buffer
    auto meet = [&]() __attribute__((always_inline)) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };
    if (s0 < s1)
        fetch(s0, sa0, sb0);
    // the loads stay where they stand (sched_barrier): sunk to the next barrier
    // they cost a sixth of the time
    int st = s0;
    for (; st + 1 < s1; st += 2) {
        meet();
        fetch(st + 1, sa1, sb1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(sa0, sb0);
        __builtin_amdgcn_sched_barrier(0);
        meet();
        if (st + 2 < s1)
            fetch(st + 2, sa0, sb0);
        __builtin_amdgcn_sched_barrier(0);
        multiply(sa1, sb1);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (st < s1) {
        meet();
        multiply(sa0, sb0);
    }
    // lane: row c of dy, k 16g .. 16g + 15 of the wave's 64
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int m = m0 + wm + 16 * i + c;
        if (m >= p.M)
            continue;
        const size_t at = static_cast<size_t>(m) * p.K + k0 + wk + 16 * g;
        if (p.part) {
            f32x4_t* o = reinterpret_cast<f32x4_t*>(p.part + static_cast<size_t>(blockIdx.y) * p.M * p.K + at);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                o[t] = acc[i][t];
        } else {
            u32x4_t o[2];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    o[t / 2][2 * (t % 2) + e] = f32_to_bf16(acc[i][t][2 * e]) | f32_to_bf16(acc[i][t][2 * e + 1]) << 16;
            u32x4_t* d = reinterpret_cast<u32x4_t*>(p.dx + at);
            d[0] = o[0];
            d[1] = o[1];
        }
    }
}

// ---------------------------------------------------------------------------
// few rows: the layer decoded on its way into the product
// ---------------------------------------------------------------------------
// Up to FEW_M rows the weights are the work, so they are read packed and once.
// A wave takes a chunk of 128 k and 64 rows of W a step, a row a lane, whose
// table and scales then serve 128 weights.  32 k at a time, neighbouring lanes
// pair their values, LDS of the wave's own turns the block (wave_sync, no
// barrier), and the matrix cores multiply it with dy, whose rows come in
// 128-byte pieces and are turned the same way (loaded as operands they cost the
// vector cache a clock for every lane).  The next step's weights are asked for
// once this one's tables stand (14336 x 4096, 128 rows: 38 us, one more
// without).  Eight waves share the rows out, and their sums meet in LDS at the
// end; further splits of the rows leave fp32 partial sums.  What bounds it is a
// step's chain of LDS and vector work (lookups and pairing, four instructions a
// weight) with two waves a SIMD.
// FEW_M, whole calls: 256 rows 4096 x 4096 26 us, turned first 35; 14336 x 4096 63
// and 92; 4096 x 14336 72 and 86; 512 x 512 9 and 11; 320 rows 4096 x 4096 43 and 37.
constexpr int FEW_M = 256;
constexpr int FEW_THREADS = 512;
// Dwords of a turned row of 64 n: the 16 rows of an operand read lie in 64 banks.
// Every other pair of rows has its halves exchanged, so that even and odd lanes
// write to other banks too.
constexpr int FEW_STRIDE = 36;
constexpr int FEW_PITCH = 9;         // 16-byte pieces of a staged row of dy

struct FewArgs {
    const uint16_t* dy;     // [M][N]
    const uint8_t* packed;
    const uint16_t* lut;
    const uint16_t* alpha;
    const uint16_t* beta;
    uint16_t* dx;
    float* part;            // [S][M][K] or null (S = 1)
    int M, N, K, g, S;
};

// 16 * MB rows of dy x 128 k a workgroup.
template <int FMT, int MB, bool WHOLE>
__global__ __launch_bounds__(FEW_THREADS) void k_dx_few(const FewArgs p)
{
    constexpr int WAVES = FEW_THREADS / WAVE, TURNED = 32 * FEW_STRIDE / 4, STAGED = 16 * FEW_PITCH;     // 16-byte pieces a wave
    constexpr int SUMS = MB > 1 ? 2 : 1;         // blocks of 16 rows whose sums meet at once
    constexpr int ROOM = TURNED + STAGED > 8 * WAVE * SUMS ? TURNED + STAGED : 8 * WAVE * SUMS;
    __shared__ u32x4_t room[WAVES * ROOM];       // the waves' blocks, and afterwards their sums
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, g = lane >> 4;
    const int Kc = p.K / 128, chunk = blockIdx.x % Kc, m0 = blockIdx.x / Kc * (16 * MB);
    const int steps = (p.N + 63) / 64, parts = p.S * WAVES, at = blockIdx.y * WAVES + w;
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * at / parts);
    const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (at + 1) / parts);
    const Matrix<WHOLE> dy(p.dy, static_cast<size_t>(p.M) * p.N);
    typedef typename Matrix<WHOLE>::Piece Piece;
    uint32_t* turned = reinterpret_cast<uint32_t*>(room + w * (TURNED + STAGED));
    u32x4_t* staged = room + w * (TURNED + STAGED) + TURNED;

    f32x4_t acc[MB][8];      // [rows of dy][16 k each]
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int b = 0; b < 8; ++b)
            acc[i][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t next[4][4];
    RowTable r;
    auto fetch_weights = [&](int st) __attribute__((always_inline)) {
        const int row = st * 64 + lane < p.N ? st * 64 + lane : 0;
        r = fetch_table<FMT>(p.lut, p.alpha, p.beta, row, Kc, chunk, p.g);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            fetch_codes<FMT>(p.packed, row, Kc, chunk, q, next[q]);
    };
    if (s0 < s1)
        fetch_weights(s0);
    for (int st = s0; st < s1; ++st) {
        // lane: piece lane % 8 of row 8 h + lane / 8
        Piece x[MB][2];
        const bool edge = st * 64 + 64 > p.N;
        const int n = st * 64 + 8 * (lane & 7);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = m0 + 16 * i + 8 * h + lane / 8;
                x[i][h] = dy.fetch(static_cast<uint32_t>(m) * p.N + n, m < p.M ? p.N - n : 0, edge);
            }
        bf16x8_t d[MB][2];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = m0 + 16 * i + 8 * h + lane / 8;
                staged[(8 * h + lane / 8) * FEW_PITCH + (lane & 7)] =
                    dy.finish(x[i][h], static_cast<uint32_t>(m) * p.N + n, p.N - n, edge);
            }
            wave_sync();
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
                d[i][kk] = __builtin_bit_cast(bf16x8_t, staged[c * FEW_PITCH + 4 * kk + g]);
            wave_sync();
        }
        ByteTable<FMT> t(r);
        if (st * 64 + lane >= p.N)      // rows behind the last: weights of 0
#pragma unroll
            for (int i = 0; i < ByteTable<FMT>::ENTRIES / 4; ++i)
                t.lo[i] = t.hi[i] = 0u;
        uint32_t code[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                code[q][i] = next[q][i];
        if (st + 1 < s1)
            fetch_weights(st + 1);
        __builtin_amdgcn_sched_barrier(0);      // asked for here, not where they are used
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t v[16];
            decode(t, code[q], v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                turned[(first_k(i) + 2 * (lane & 1)) * FEW_STRIDE + (lane / 2 ^ 16 * ((first_k(i) >> 1 ^ lane) & 1))] =
                    pair_rows(v[i], lane & 1);
            wave_sync();
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const bf16x8_t wv = *reinterpret_cast<const bf16x8_t*>(&turned[(16 * b + c) * FEW_STRIDE + (16 * kk ^ 8 * (c & 2)) + 4 * g]);
#pragma unroll
                    for (int i = 0; i < MB; ++i)
                        acc[i][2 * q + b] = mfma(wv, d[i][kk], acc[i][2 * q + b]);
                }
            wave_sync();
        }
    }
    f32x4_t* red = reinterpret_cast<f32x4_t*>(room);      // [SUMS][WAVES][8][WAVE]
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        if (i % SUMS == 0) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < SUMS; ++e)
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    red[((e * WAVES + w) * 8 + b) * WAVE + lane] = acc[i + e][b];
            __syncthreads();
        }
        f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};             // wave w: the sums of its 16 k
#pragma unroll
        for (int o = 0; o < WAVES; ++o)
            v += red[((i % SUMS * WAVES + o) * 8 + w) * WAVE + lane];
        const int m = m0 + 16 * i + c;
        if (m >= p.M)
            continue;
        const size_t o = static_cast<size_t>(m) * p.K + chunk * 128 + 16 * w + 4 * g;
        if (p.part) {
            *reinterpret_cast<f32x4_t*>(p.part + static_cast<size_t>(blockIdx.y) * p.M * p.K + o) = v;
        } else {
            u32x2_t y;
            y[0] = f32_to_bf16(v[0]) | f32_to_bf16(v[1]) << 16;
            y[1] = f32_to_bf16(v[2]) | f32_to_bf16(v[3]) << 16;
            *reinterpret_cast<u32x2_t*>(p.dx + o) = y;
        }
    }
}

template <int FMT, bool WHOLE>
void launch_few(const FewArgs& a, int mb, hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.M + 16 * mb - 1) / (16 * mb) * (a.K / 128)), static_cast<unsigned>(a.S));
#define FEW(MB_) hipLaunchKernelGGL((k_dx_few<FMT, MB_, WHOLE>), grid, dim3(FEW_THREADS), 0, stream, a)
    if (mb == 1) FEW(1);
    else FEW(4);
#undef FEW
}

template <int FMT>
void launch_few(const FewArgs& a, int mb, hipStream_t stream)
{
    if (a.N % 8 == 0 && is_aligned(a.dy, 16))
        launch_few<FMT, true>(a, mb, stream);
    else
        launch_few<FMT, false>(a, mb, stream);
}

// The splits' sums in order, 4 values a thread, eight splits' loads at a time.
__global__ __launch_bounds__(256) void k_dx_sum(const float* __restrict__ part, uint16_t* __restrict__ dx, int S, size_t quads)
{
    const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
    if (i >= quads)
        return;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < S; s0 += 8) {
        f32x4_t x[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
            x[s] = s0 + s < S ? reinterpret_cast<const f32x4_t*>(part)[(s0 + s) * quads + i] : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < 8; ++s)
            v += x[s];
    }
    u32x2_t o;
    o[0] = f32_to_bf16(v[0]) | f32_to_bf16(v[1]) << 16;
    o[1] = f32_to_bf16(v[2]) | f32_to_bf16(v[3]) << 16;
    reinterpret_cast<u32x2_t*>(dx)[i] = o;
}

// dx = 0: a layer without outputs.
__global__ __launch_bounds__(256) void k_dx_zero(uint16_t* dx, size_t octs)
{
    const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
    if (i < octs)
        reinterpret_cast<u32x4_t*>(dx)[i] = u32x4_t{0u, 0u, 0u, 0u};
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int64_t padded(int64_t N) { return (N + STEP - 1) / STEP * STEP; }

// How a product is run: decoded on the way (few rows), else turned first, in
// 256 x 256 or 128 x 128 tiles, n split where that leaves less to do for the
// longest-working CU; the partial sums are fp32.
struct Shape {
    int few;                 // blocks of 16 rows of a workgroup, 0: turned first
    bool big;
    int64_t tiles;
    int S;
};

Shape dx_shape(int64_t M, int64_t N, int64_t K)
{
    const int64_t steps = padded(N) / STEP;
    Shape s{0, false, 0, 1};
    int64_t least = INT64_MAX;
    if (M <= FEW_M) {
        s.few = M <= 16 ? 1 : 4;
        s.tiles = (M + 16 * s.few - 1) / (16 * s.few) * (K / 128);
        // Of the splits that leave each wave a step, the one with the fewest steps
        // over all rounds of the chip (its LDS holds two workgroups of 16 rows a CU,
        // one of 64), two more a round to start and to add up.  As many workgroups as
        // there are CUs, rounds or not: 64 rows, 4096 x 14336 (112 tiles) 36 us
        // against 25; 16 rows 23 against 19.
        const int64_t most = steps / 8 < 16 ? steps / 8 : 16, room = s.few == 1 ? 512 : 256;
        for (int64_t n = 1; n == 1 || n <= most; ++n) {
            const int64_t time = (s.tiles * n + room - 1) / room * ((steps + 8 * n - 1) / (8 * n) + 2);
            if (time <= least) {
                least = time;
                s.S = static_cast<int>(n);
            }
        }
        return s;
    }
    // Turned first: the time of each choice in units of 10 ns, from what steps were
    // measured to take (a large tile 1.6 us; a small one 0.7, two on a CU 0.95 together;
    // splits 7 us and 0.3 us a MB of partial sums to write, read and add) on the CU with
    // the most tiles.  Splits go up to two workgroups a CU, each at least four steps.
    // A fixed number of workgroups instead (256 large or 512 small, rounded up),
    // whole calls in us: M 2048, 4096 x 4096 91 against 75 here; 1500 83 against 69;
    // 320 44 against 39; 600, 14336 x 4096 152 against 121; 2500 378 against 316; 600,
    // 4096 x 14336 164 against 126; 3000, 2048 x 2048 57 against 40.
    const int64_t tiles[2] = {(M + 127) / 128 * (K / 128), K % 256 ? 0 : (M + 255) / 256 * (K / 256)};
    for (int big = 0; big < 2; ++big)
        for (int64_t n = 1; tiles[big] && n <= 16 && (n == 1 || (tiles[big] * n <= 512 && steps / n >= 4)); ++n) {
            const int64_t on_cu = (tiles[big] * n + 255) / 256, step = big ? 160 * on_cu : on_cu / 2 * 95 + on_cu % 2 * 70;
            const int64_t time = step * ((steps + n - 1) / n) + (n > 1 ? 700 + n * M * K / 8333 : 300);
            if (time < least) {
                least = time;
                s.big = big;
                s.tiles = tiles[big];
                s.S = static_cast<int>(n);
            }
        }
    return s;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

size_t wt_bytes(int64_t N, int64_t K) { return up256(static_cast<size_t>(K) * padded(N) * 2); }

size_t dx_bytes(const Shape& s, int64_t M, int64_t N, int64_t K)
{
    const size_t part = s.S > 1 ? up256(static_cast<size_t>(s.S) * M * K * 4) : 0;
    if (s.few)
        return part + 256;       // never 0 where the call has work
    return wt_bytes(N, K) + up256(static_cast<size_t>(M) * padded(N) * 2) + part;
}

bool dx_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t g)
{
    const int64_t top = static_cast<int64_t>(1) << 31;
    return M >= 0 && M <= 65535 * 64 && N >= 0 && N <= static_cast<int64_t>(1) << 21 && K >= 0 && K < top && g > 0 && g % 128 == 0 &&
           K % g == 0 && N * K < 2 * top && M * K * 2 < top && M * N * 2 < top;
}

any4_status gemm_dx(int fmt, const uint16_t* dy, const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha,
                    const uint16_t* beta, uint16_t* dx, int64_t M, int64_t N, int64_t K, int64_t g, void* workspace,
                    size_t workspace_bytes, hipStream_t stream)
{
    if (!dx_sizes_ok(M, N, K, g))
        return ANY4_E_SHAPE;
    if (M == 0 || K == 0)
        return ANY4_OK;
    if (!dx || (N > 0 && (!dy || !packed || (fmt != FMT_INT4 && !lut) || !alpha || !beta || !workspace)))
        return ANY4_E_NULL;
    if (!is_aligned(dx, 16) || (N > 0 && (!is_aligned(dy, 2) || !is_aligned(packed, 16) || !is_aligned(lut, 2) ||
                                          !is_aligned(alpha, 2) || !is_aligned(beta, 2) || !is_aligned(workspace, 16))))
        return ANY4_E_ALIGN;
    const Shape shape = N > 0 ? dx_shape(M, N, K) : Shape{};
    if (N > 0 && workspace_bytes < dx_bytes(shape, M, N, K))
        return ANY4_E_WORKSPACE;
    (void)hipGetLastError();
    if (N == 0) {
        const size_t octs = static_cast<size_t>(M) * K / 8;
        hipLaunchKernelGGL(k_dx_zero, dim3(static_cast<unsigned>((octs + 255) / 256)), dim3(256), 0, stream, dx, octs);
        return launch_status();
    }
    const int Np = static_cast<int>(padded(N));
    const size_t quads = static_cast<size_t>(M) * K / 4;
    const dim3 sum_grid(static_cast<unsigned>((quads + 255) / 256));
    if (shape.few) {
        float* part = shape.S > 1 ? static_cast<float*>(workspace) : nullptr;
        const FewArgs f{dy, packed, lut, alpha, beta, dx, part, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K),
                        static_cast<int>(g), shape.S};
        if (fmt == FMT_ANY4) launch_few<FMT_ANY4>(f, shape.few, stream);
        else if (fmt == FMT_INT4) launch_few<FMT_INT4>(f, shape.few, stream);
        else if (fmt == FMT_ANY2) launch_few<FMT_ANY2>(f, shape.few, stream);
        else launch_few<FMT_ANY3>(f, shape.few, stream);
        if (part)
            hipLaunchKernelGGL(k_dx_sum, sum_grid, dim3(256), 0, stream, part, dx, shape.S, quads);
        return launch_status();
    }
    char* at = static_cast<char*>(workspace);
    uint16_t* wt = reinterpret_cast<uint16_t*>(at);
    at += wt_bytes(N, K);
    const dim3 grid(static_cast<unsigned>(Np / 64 * (K / 128)));
#define TURN(FMT_) hipLaunchKernelGGL(k_dequant_t<FMT_>, grid, dim3(DT_THREADS), 0, stream, packed, lut, alpha, beta, wt, \
                                      static_cast<int>(N), static_cast<int>(K), static_cast<int>(g), Np)
    if (fmt == FMT_ANY4) TURN(FMT_ANY4);
    else if (fmt == FMT_INT4) TURN(FMT_INT4);
    else if (fmt == FMT_ANY2) TURN(FMT_ANY2);
    else TURN(FMT_ANY3);
#undef TURN
    DxArgs a{dy, wt, dx, nullptr, static_cast<int>(M), static_cast<int>(K), Np, shape.S};
    if (N != Np || !is_aligned(dy, 16)) {
        uint16_t* copy = reinterpret_cast<uint16_t*>(at);
        const size_t pieces = static_cast<size_t>(M) * (Np / 8);
        hipLaunchKernelGGL(k_pad_rows, dim3(static_cast<unsigned>((pieces + 255) / 256)), dim3(256), 0, stream, dy, copy,
                           static_cast<int>(N), Np, pieces);
        a.dy = copy;
    }
    at += up256(static_cast<size_t>(M) * Np * 2);
    if (a.S > 1)
        a.part = reinterpret_cast<float*>(at);
    const dim3 tiles(static_cast<unsigned>(shape.tiles), static_cast<unsigned>(a.S));
    if (shape.big)
        hipLaunchKernelGGL((k_dx<2, 4, 8>), tiles, dim3(512), 0, stream, a);
    else
        hipLaunchKernelGGL((k_dx<2, 2, 4>), tiles, dim3(256), 0, stream, a);
    if (a.S > 1)
        hipLaunchKernelGGL(k_dx_sum, sum_grid, dim3(256), 0, stream, a.part, dx, a.S, quads);
    return launch_status();
}

}  // namespace

extern "C" {

size_t any4_gemm_dx_workspace_size(int64_t M, int64_t N, int64_t K, int64_t g)
{
    if (M <= 0 || N <= 0 || K <= 0 || !dx_sizes_ok(M, N, K, g))
        return 0;
    return dx_bytes(dx_shape(M, N, K), M, N, K);
}

any4_status any4_gemm_dx(const uint16_t* dy, const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha,
                         const uint16_t* beta, uint16_t* dx, int64_t M, int64_t N, int64_t K, int64_t g, void* workspace,
                         size_t workspace_bytes, hipStream_t stream)
{
    return gemm_dx(FMT_ANY4, dy, packed, lut, alpha, beta, dx, M, N, K, g, workspace, workspace_bytes, stream);
}

any4_status any4_gemm_int4_dx(const uint16_t* dy, const uint8_t* packed, const uint16_t* alpha, const uint16_t* beta,
                              uint16_t* dx, int64_t M, int64_t N, int64_t K, int64_t g, void* workspace,
                              size_t workspace_bytes, hipStream_t stream)
{
    return gemm_dx(FMT_INT4, dy, packed, nullptr, alpha, beta, dx, M, N, K, g, workspace, workspace_bytes, stream);
}

any4_status any2_gemm_dx(const uint16_t* dy, const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha,
                         const uint16_t* beta, uint16_t* dx, int64_t M, int64_t N, int64_t K, int64_t g, void* workspace,
                         size_t workspace_bytes, hipStream_t stream)
{
    return gemm_dx(FMT_ANY2, dy, packed, lut, alpha, beta, dx, M, N, K, g, workspace, workspace_bytes, stream);
}

any4_status any3_gemm_dx(const uint16_t* dy, const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha,
                         const uint16_t* beta, uint16_t* dx, int64_t M, int64_t N, int64_t K, int64_t g, void* workspace,
                         size_t workspace_bytes, hipStream_t stream)
{
    return gemm_dx(FMT_ANY3, dy, packed, lut, alpha, beta, dx, M, N, K, g, workspace, workspace_bytes, stream);
}

}  // extern "C"
