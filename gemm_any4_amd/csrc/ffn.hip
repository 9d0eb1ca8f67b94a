// Products of quantised layers with what a feed-forward block puts around them:
// bias, activation, gate and residual, for one layer (any4_gemm_act) or for the
// stacked layers of many experts, each row through the expert that the router
// chose (any4_experts_gemm), the experts' input gradient (any4_experts_gemm_dx)
// and the activation's backward pass (any4_act_backward).  The C ABI is declared
// in include/any4.h.
//
//     z[p] = W_e x[p / div] + bias_e      e = ids[p] (one layer: 0)
//     out[p] = act(z) + residual[p], or with a gate, W_e = [gate; up],
//     out[p] = act(z_gate) * z_up + residual[p]
//
// Rows of one expert are worked on in tiles, from the plan (plan.h) or, for few
// pairs, from ballots over the ids.
#include <cmath>
#include <type_traits>

#include "codes.h"
#include "plan.h"

namespace {

constexpr int MAX_EXPERTS = 1024;
constexpr int STEP = 64;                                  // of the summed dimension, k_tile
constexpr int FMT_BF16 = FMT_ANY3 + 1;                    // of k_tile: a layer that k_rows has laid out as bf16 rows
constexpr int64_t MAX_PAIRS = static_cast<int64_t>(1) << 20;
enum { X_BF16, X_F32, X_PARTS };     // how the rows of x are kept

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// the rows of a product
// ---------------------------------------------------------------------------
struct Rows {
    const int* ids;      // few pairs: their experts; else null
    const int* plan;     // or the pairs by expert; both null: one layer
    int P, E, div;       // pairs, experts, pairs that share a row of x
};

struct Layer {           // of all experts, one after another
    const uint8_t* packed;
    const uint16_t *lut, *alpha, *beta;
    int N, K, g;
    size_t packed_bytes; // of one expert

    __device__ __forceinline__ const uint8_t* codes(int e) const { return packed + e * packed_bytes; }
    __device__ __forceinline__ const uint16_t* table(int e) const { return lut + static_cast<size_t>(e) * N * 16; }
    __device__ __forceinline__ size_t scales(int e) const { return static_cast<size_t>(e) * N * (K / g); }
};

constexpr int FEW_T = 16;            // rows of a tile of k_few
constexpr int FEW_P = WAVE;          // pairs up to which tiles come from ballots

struct Tile {
    int e;          // expert; E: rows without one; -1: no such tile
    int count;
};

__device__ __forceinline__ int expert_of(int id, int E) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(E) ? id : E; }

// Tile t of FEW_T rows, its pairs in own[0 .. count): every wave for itself.
__device__ __forceinline__ Tile find_few(const Rows& r, int t, int* own)
{
    const int lane = threadIdx.x & 63;
    if (r.plan) {
        if (r.plan[2] != r.P || r.plan[3] != r.E)
            return {-1, 0};
        const PlanLayout p(r.P, r.E);
        const int at = t / (TILE_T / FEW_T), from = t % (TILE_T / FEW_T) * FEW_T;
        if (at >= r.plan[0])
            return {-1, 0};
        const int a = r.plan[p.tile + 2 * static_cast<int64_t>(at)], n = r.plan[p.tile + 2 * static_cast<int64_t>(at) + 1];
        if (from >= n)
            return {-1, 0};
        if (lane < FEW_T)
            own[lane] = r.plan[p.rows + TILE_T * static_cast<int64_t>(at) + from + lane];
        wave_sync();
        return {a < 0 ? r.E : a, n - from < FEW_T ? n - from : FEW_T};
    }
    if (!r.ids) {
        const int left = r.P - t * FEW_T;
        if (lane < FEW_T)
            own[lane] = t * FEW_T + lane;
        wave_sync();
        return {left > 0 ? 0 : -1, left < FEW_T ? left : FEW_T};
    }
    const bool live = lane < r.P;
    const int a = live ? expert_of(r.ids[lane], r.E) : -1;
    uint64_t left = __ballot(live);
    while (left) {
        const int v = __builtin_amdgcn_readlane(a, __builtin_ctzll(left));
        const uint64_t m = __ballot(live && a == v);
        const int n = __builtin_popcountll(m), tiles = (n + FEW_T - 1) / FEW_T;
        if (t < tiles) {
            const int rank = __builtin_popcountll(m & ((1ull << lane) - 1));
            if ((m >> lane & 1) && rank / FEW_T == t)
                own[rank % FEW_T] = lane;
            wave_sync();
            return {v, n - t * FEW_T < FEW_T ? n - t * FEW_T : FEW_T};
        }
        t -= tiles;
        left &= ~m;
    }
    return {-1, 0};
}

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------
enum { ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACTS };

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + expf(-z)); }

constexpr float GELU_C = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float GELU_D = 0.044715f;

// The normal distribution's integral up to z; 1 + erf would cancel left of 0 (4% off at -5).
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }

__device__ __forceinline__ float activate(float z, int act)
{
    switch (act) {
    case ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case ACT_SILU: return z * sigmoid(z);
    case ACT_GELU: return z * normal_cdf(z);
    case ACT_GELU_TANH: return z * sigmoid(GELU_C * (z + GELU_D * z * z * z));
    default: return z;
    }
}

// act(z) and its slope
__device__ __forceinline__ void activate_both(float z, int act, float& f, float& slope)
{
    switch (act) {
    case ACT_RELU:
        f = z > 0.0f || z != z ? z : 0.0f;
        slope = z > 0.0f ? 1.0f : z != z ? z : 0.0f;
        break;
    case ACT_SILU: {
        const float p = sigmoid(z);
        f = z * p;
        slope = p * (1.0f + z * (1.0f - p));
        break;
    }
    case ACT_GELU: {
        const float p = normal_cdf(z);
        f = z * p;
        slope = p + z * 0.39894228040143268f * expf(-0.5f * z * z);
        break;
    }
    case ACT_GELU_TANH: {
        const float p = sigmoid(GELU_C * (z + GELU_D * z * z * z));
        f = z * p;
        const float turn = p * (1.0f - p);       // 0 before z * z is no longer finite
        slope = turn > 0.0f ? p + z * turn * GELU_C * (1.0f + 3.0f * GELU_D * z * z) : p;
        break;
    }
    default:
        f = z;
        slope = 1.0f;
    }
}

// ---------------------------------------------------------------------------
// the epilogue: everything in fp32, each result rounded once
// ---------------------------------------------------------------------------
struct Epilogue {
    const uint16_t* bias;        // [E][N] or null
    const uint16_t* residual;    // [P][No] or null
    void* z;                     // [P][N] or null
    void* out;                   // [P][No], in parts [2][P][No]
    float* part;                 // [S][P][N] or null (S = 1)
    int N, No, act, S;           // No = N / 2: gated
    int z32, out32;              // fp32 instead of bf16; out32 ANY4_PARTS: two bf16 parts
    size_t plane;                // in parts: from hi to lo

    __host__ __device__ __forceinline__ bool gated() const { return No != N; }
};

// fp32 as the bf16 parts hi + lo: hi cut off, lo what is left, rounded (2^-16 of the
// value at most).  An infinity has no lo.  (Not contracted: lo is what is left of the
// rounded value that hi was cut from, not of a product behind it.)
__device__ __forceinline__ void split(float v, uint32_t& hi, uint32_t& lo)
{
#pragma clang fp contract(off)
    const uint32_t top = __builtin_bit_cast(uint32_t, v) & 0xffff0000u;
    hi = top >> 16;
    lo = f32_to_bf16(__builtin_isinf(v) ? 0.0f : v - __builtin_bit_cast(float, top));
}

__device__ __forceinline__ void put_parts(uint16_t* to, size_t plane, int valid, const float (&v)[8])
{
    u32x4_t hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2], l[2];
        split(v[2 * i], h[0], l[0]);
        split(v[2 * i + 1], h[1], l[1]);
        hi[i] = h[0] | h[1] << 16;
        lo[i] = l[0] | l[1] << 16;
    }
    store8(to, hi, valid);
    store8(to + plane, lo, valid);
}

__device__ __forceinline__ void put_outs(const Epilogue& q, size_t at, int valid, const float (&v)[8])
{
    if (q.out32 != ANY4_PARTS) {
        put_values(q.out, q.out32, at, valid, v);
        return;
    }
    put_parts(static_cast<uint16_t*>(q.out) + at, q.plane, valid, v);
}

__device__ __forceinline__ void put_out(const Epilogue& q, size_t at, float v)
{
    if (q.out32 != ANY4_PARTS) {
        put_value(q.out, q.out32, at, v);
        return;
    }
    uint32_t hi, lo;
    split(v, hi, lo);
    uint16_t* out = static_cast<uint16_t*>(q.out) + at;
    out[0] = static_cast<uint16_t>(hi);
    out[q.plane] = static_cast<uint16_t>(lo);
}

// Columns col .. col + 7 of pair p: v the (gate's) sums, u the up rows' where there
// is a gate.
__device__ __forceinline__ void finish8(const Epilogue& q, int e, int p, int col, float (&v)[8], float (&u)[8])
{
    const int valid = q.No - col;
    if (valid <= 0)
        return;
    const bool gate = q.gated();
    if (q.bias) {
        const size_t at = static_cast<size_t>(e) * q.N + col;
        float b[8];
        get_values(q.bias, 0, at, valid, b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += b[i];
        if (gate) {
            get_values(q.bias, 0, at + q.No, valid, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                u[i] += b[i];
        }
    }
    if (q.z) {
        const size_t at = static_cast<size_t>(p) * q.N + col;
        put_values(q.z, q.z32, at, valid, v);
        if (gate)
            put_values(q.z, q.z32, at + q.No, valid, u);
    }
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        o[i] = activate(v[i], q.act);
        if (gate)
            o[i] *= u[i];
    }
    const size_t at = static_cast<size_t>(p) * q.No + col;
    if (q.residual) {
        float r[8];
        get_values(q.residual, 0, at, valid, r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] += r[i];
    }
    put_outs(q, at, valid, o);
}

// Where part i of n starts among `all` (below 2^25, n at most 64); the same for all
// lanes, which the compiler does not see of a division.
__device__ __forceinline__ int share(int all, int i, int n) { return __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(all) * i / n)); }

// ---------------------------------------------------------------------------
// few rows: packed weights read once, decoded in registers
// ---------------------------------------------------------------------------
constexpr int FEW_ROWS = 64;         // rows of W of a workgroup

struct FewArgs {
    Rows r;
    Layer w;
    const void* x;
    Epilogue q;
    size_t plane;            // X_PARTS: from hi to lo
};

template <int I, int N, typename F>
__device__ __forceinline__ void static_for(F&& f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        static_for<I + 1, N>(f);
    }
}

// D[i][lane] += sum over four k of A[i] B[lane]: A's block ABID for all lanes.
template <int ABID>
__device__ __forceinline__ f32x4_t mfma4(s16x4_t a, s16x4_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(a, b, c, 4, ABID, 0);
}

// A row's next 128 weights and their scales.
template <int FMT>
struct RowChunk {
    uint32_t code[4][4], alpha, beta;

    __device__ __forceinline__ void fetch(const uint8_t* packed, const uint16_t* a, const uint16_t* b, int row, int Kc, int chunk, int g)
    {
        const size_t grp = static_cast<size_t>(row) * (Kc * 128 / g) + chunk * 128 / g;
        alpha = a[grp];
        beta = b[grp];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            fetch_codes<FMT>(packed, row, Kc, chunk, q, code[q]);
    }
};

__device__ __forceinline__ void split4(f32x4_t v, s16x4_t& hi, s16x4_t& lo)
{
    u32x2_t h, l;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t top[2], rest[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            split(v[2 * i + j], top[j], rest[j]);
        h[i] = top[0] | top[1] << 16;
        l[i] = rest[0] | rest[1] << 16;
    }
    hi = __builtin_bit_cast(s16x4_t, h);
    lo = __builtin_bit_cast(s16x4_t, l);
}

// The product of 4 * NB rows of x with the lane's row of W over chunks s0 .. s1.  Rows
// of fp32 or in parts are two of bf16.
template <int FMT, int NB, int X>
__device__ __forceinline__ void few_product(const FewArgs& p, int e, int wr, const int* own, int count, int s0, int s1,
                                            f32x4_t (&acc)[4])
{
    if (s0 >= s1)
        return;
    const int lane = threadIdx.x & 63, Kc = p.w.K / 128;
    const uint8_t* packed = p.w.codes(e);
    const uint16_t *alpha = p.w.alpha + p.w.scales(e), *beta = p.w.beta + p.w.scales(e);
    typedef std::conditional_t<X == X_F32, float, uint16_t> Element;
    typedef std::conditional_t<X == X_F32, f32x4_t, s16x4_t> Four;
    uint32_t at[NB];                 // bytes to the lane's four k of a row, of each 64 (below 2^32)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int i = 4 * b + (lane & 3);
        at[b] = static_cast<uint32_t>(sizeof(Element)) *
                (static_cast<uint32_t>(own[i < count ? i : count - 1] / p.r.div) * static_cast<uint32_t>(p.w.K) + 4u * (lane >> 2));
    }
    RowChunk<FMT> next;
    next.fetch(packed, alpha, beta, wr, Kc, s0, p.w.g);
    RowTable row = fetch_table<FMT>(FMT == FMT_INT4 ? nullptr : p.w.table(e), alpha, beta, wr, Kc, s0, p.w.g);
    for (int s = s0; s < s1; ++s) {
        Four in[NB][2], rest[NB][2];
        const char *hi = reinterpret_cast<const char*>(static_cast<const Element*>(p.x) + s * 128),
                   *lo_part = reinterpret_cast<const char*>(static_cast<const Element*>(p.x) + p.plane + s * 128);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                in[b][j] = *reinterpret_cast<const Four*>(hi + at[b] + 64 * j * sizeof(Element));
                if constexpr (X == X_PARTS)
                    rest[b][j] = *reinterpret_cast<const Four*>(lo_part + at[b] + 64 * j * sizeof(Element));
            }
        const RowChunk<FMT> now = next;
        if (s + 1 < s1)
            next.fetch(packed, alpha, beta, wr, Kc, s + 1, p.w.g);
        __builtin_amdgcn_sched_barrier(0);      // asked for here, not where they are used
        row.alpha = now.alpha;
        row.beta = now.beta;
        const ByteTable<FMT> t(row);
        s16x4_t a[NB], lo[NB];
        static_for<0, 4>([&](auto q_) __attribute__((always_inline)) {
            constexpr int q = decltype(q_)::value;
            if constexpr (q % 2 == 0)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (X == X_F32)
                        split4(in[b][q / 2], a[b], lo[b]);
                    else
                        a[b] = in[b][q / 2];
                    if constexpr (X == X_PARTS)
                        lo[b] = rest[b][q / 2];
                }
            uint32_t v[16];
            decode_in_order(t, now.code[q], v);
            static_for<0, 8>([&](auto i_) __attribute__((always_inline)) {
                constexpr int i = decltype(i_)::value;
                const u32x2_t w = {v[2 * i], v[2 * i + 1]};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    acc[b] = mfma4<8 * (q & 1) + i>(a[b], __builtin_bit_cast(s16x4_t, w), acc[b]);
                    if constexpr (X != X_BF16)
                        acc[b] = mfma4<8 * (q & 1) + i>(lo[b], __builtin_bit_cast(s16x4_t, w), acc[b]);
                }
            });
        });
    }
}

// A lane has one row of W, so that its table and scales serve 128 weights at a
// time, which the matrix cores multiply as they stand: the 16 blocks of a 4 x 4 x 4
// product hold 64 rows of W, four k each, and four rows of x go to all of them.
// WAVES share the chunks out.
//
// Bound by the vector ALU: of some 550 instructions for a lane's 128 weights 416 look
// them up.  One row with 28672 x 4096 takes 21 us (63 MB, 3.0 TB/s): 13.5 of these
// instructions, where the bytes alone would take 12.5; half its layer takes 12.5 us, twice
// as much 43.  448 workgroups are 1.75 to a CU and take the time of two: 16 rows of W a
// wave, four quarters of k side by side, fill the CUs evenly and gained less than 10% (not
// kept).  any2 and any3 have half the lookups: 14336 x 4096 in 10.4 us for any4's 12.5.
// Rows of fp32: one token through two experts' 4096 x 14336 27.7 us for 24.7, rows in parts
// 25.4 (they need no splitting).
template <int FMT, int WAVES, int X>
__global__ __launch_bounds__(WAVE * WAVES, 4) void k_few(const FewArgs p)
{
    __shared__ int own[WAVES][FEW_T];
    __shared__ float red[WAVES][FEW_T][WAVE];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tile t = find_few(p.r, blockIdx.y, own[w]);
    if (t.e < 0)
        return;
    const bool gate = p.q.gated();
    const int half = gate ? lane >> 5 : 0;
    const int col = gate ? blockIdx.x * (FEW_ROWS / 2) + (lane & 31) : blockIdx.x * FEW_ROWS + lane;
    const bool live = col < p.q.No;
    const int wr = live ? col + half * p.q.No : 0;
    if (t.e == p.r.E) {              // no expert: zeros
        if (blockIdx.z == 0 && live)
            for (int i = w; i < t.count; i += WAVES) {
                if (half == 0)
                    put_out(p.q, static_cast<size_t>(own[w][i]) * p.q.No + col, 0.0f);
                if (p.q.z)
                    put_value(p.q.z, p.q.z32, static_cast<size_t>(own[w][i]) * p.q.N + wr, 0.0f);
            }
        return;
    }
    const int Kc = p.w.K / 128, parts = p.q.S * WAVES, at = blockIdx.z * WAVES + w;
    const int s0 = share(Kc, at, parts), s1 = share(Kc, at + 1, parts);
    f32x4_t acc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
        acc[b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    static_for<0, 3>([&](auto n_) __attribute__((always_inline)) {
        constexpr int NB = 1 << decltype(n_)::value;
        if (t.count <= 4 * NB && (NB == 1 || t.count > 2 * NB))
            few_product<FMT, NB, X>(p, t.e, wr, own[w], t.count, s0, s1, acc);
    });
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (4 * b < t.count)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[w][4 * b + i][lane] = acc[b][i];
    __syncthreads();
    for (int i = w; i < t.count; i += WAVES) {
        const int pair = own[w][i];
        float v = 0.0f;
#pragma unroll
        for (int o = 0; o < WAVES; ++o)
            v += red[o][i][lane];
        if (p.q.part) {
            if (live)
                p.q.part[(static_cast<size_t>(blockIdx.z) * p.r.P + pair) * p.q.N + wr] = v;
            continue;
        }
        if (p.q.bias && live)
            v += bf16_to_f32(p.q.bias[static_cast<size_t>(t.e) * p.q.N + wr]);
        if (p.q.z && live)
            put_value(p.q.z, p.q.z32, static_cast<size_t>(pair) * p.q.N + wr, v);
        const float up = __shfl(v, lane | 32);
        if (half || !live)
            continue;
        v = activate(v, p.q.act);
        if (gate)
            v *= up;
        const size_t to = static_cast<size_t>(pair) * p.q.No + col;
        if (p.q.residual)
            v += bf16_to_f32(p.q.residual[to]);
        put_out(p.q, to, v);
    }
}

// The splits' sums in order, then the epilogue; 8 columns a thread.  Bound by its bytes
// (2062 rows of 4096 in four splits to fp32, 169 MB: 33 us), for few rows by its launch (4 us).
__global__ __launch_bounds__(256) void k_join(const Epilogue q, const int* __restrict__ ids, const int* __restrict__ plan, int P, int E,
                                              size_t pieces)
{
    const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
    if (i >= pieces || (plan && (plan[2] != P || plan[3] != E)))
        return;
    const int per = (q.No + 7) / 8, p = static_cast<int>(i / per), col = static_cast<int>(i % per) * 8;
    const int e = ids ? expert_of(ids[p], E) : 0;
    if (ids && e == E)
        return;                      // zeros are there already
    float v[8], u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = u[k] = 0.0f;
    const int valid = q.No - col;
    for (int s = 0; s < q.S; ++s) {
        const float* f = q.part + (static_cast<size_t>(s) * P + p) * q.N + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h && !q.gated())
                break;
            float (&to)[8] = h ? u : v;
            const float* from = f + h * q.No;
            if (valid >= 8) {
                const f32x4_t a = *reinterpret_cast<const f32x4_a4_t*>(from), b = *reinterpret_cast<const f32x4_a4_t*>(from + 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    to[k] += a[k];
                    to[4 + k] += b[k];
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < valid)
                        to[k] += from[k];
            }
        }
    }
    finish8(q, e, p, col, v, u);
}

// ---------------------------------------------------------------------------
// more rows: tiles for the matrix cores, weights decoded into LDS
// ---------------------------------------------------------------------------
struct TileArgs {
    Rows r;
    Layer w;
    const uint16_t* x;       // [rows][D], D the summed dimension (padded to 8); in parts [2][rows][D]
    Epilogue q;
    int rows, D, steps;
    int tiles_m, tiles_n;
};

// The tile's expert, its pairs among the plan's rows and their number.  Every
// wave sums the experts' tiles for itself.
__device__ __forceinline__ Tile find_tile(const Rows& r, int t, int BM, int64_t& first)
{
    const int lane = threadIdx.x & 63;
    if (!r.plan) {
        const int left = r.P - t * BM;
        return {left > 0 ? 0 : -1, left < BM ? left : BM};
    }
    if (r.plan[2] != r.P || r.plan[3] != r.E)
        return {-1, 0};
    const PlanLayout p(r.P, r.E);
    for (int e0 = 0; e0 <= r.E; e0 += WAVE) {
        const int e = e0 + lane;
        const int n = e <= r.E ? r.plan[p.count + e] : 0, at = e <= r.E ? r.plan[p.first + e] : 0;
        const int tiles = (n + BM - 1) / BM;
        int sum = tiles;
        for (int d = 1; d < WAVE; d <<= 1) {
            const int o = __shfl_up(sum, d);
            sum += lane >= d ? o : 0;
        }
        const uint64_t hit = __ballot(t < sum);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int before = __builtin_amdgcn_readlane(sum - tiles, l), rows = __builtin_amdgcn_readlane(n, l);
            const int from = (t - before) * BM;
            first = p.rows + static_cast<int64_t>(__builtin_amdgcn_readlane(at, l)) * TILE_T + from;
            return {e0 + l, rows - from < BM ? rows - from : BM};
        }
        t -= __builtin_amdgcn_readlane(sum, WAVE - 1);
    }
    return {-1, 0};
}

// Columns of the products of a wave: place 16 t + rho of its 64 holds column
// 16 (rho / 4) + 4 t + rho % 4, so that a lane's results are 16 adjacent columns.
__device__ __forceinline__ int column_of(int place) { return 16 * (place >> 2 & 3) + 4 * (place >> 4 & 3) + (place & 3); }

// Rows of 64 values in LDS, eight pieces of 16 bytes; piece q stands at q ^ key(row):
// 16 rows of an operand read, and 16 rows that lanes write, touch all 64 banks once.
__device__ __forceinline__ int key(int row) { return row >> 1 & 7; }
__device__ __forceinline__ void put8(float* to, f32x4_t a, f32x4_t b, int valid)
{
    if (valid >= 8) {
        *reinterpret_cast<f32x4_a4_t*>(to) = a;
        *reinterpret_cast<f32x4_a4_t*>(to + 4) = b;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < valid)
            to[i] = a[i];
        if (4 + i < valid)
            to[4 + i] = b[i];
    }
}

constexpr int slot_bytes(int fmt) { return fmt == FMT_ANY2 ? 8 : fmt == FMT_ANY3 ? 12 : 16; }    // of 32 codes

template <int FMT>
__device__ __forceinline__ void load_slot(__amdgpu_buffer_rsrc_t codes, int at, int from, uint32_t (&c)[4])
{
    c[0] = c[1] = c[2] = c[3] = 0u;
    if constexpr (FMT == FMT_ANY2) {
        const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(codes, at, from, 0);
        c[0] = v[0];
        c[1] = v[1];
    } else if constexpr (FMT == FMT_ANY3) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b96(codes, at, from, 0);
        c[0] = v[0];
        c[1] = v[1];
        c[2] = v[2];
    } else {
        const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(codes, at, from, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = v[i];
    }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, size_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), static_cast<int>(bytes), 0x00020000);
}

// A chunk of 128 k of a row, of which a thread decodes a quarter a step, by buffer
// loads: the row's place is the lane's offset, the chunk's the wave's.
struct RowPart {
    uint32_t code[2][4], alpha, beta;
};

template <int FMT>
struct RowReader {
    static constexpr int BYTES = slot_bytes(FMT), LOADS = 4;
    __amdgpu_buffer_rsrc_t codes, alpha, beta;
    int at, scale_at, g;

    __device__ __forceinline__ RowReader(const Layer& w, int e, int row, int h) : g(w.g)
    {
        const size_t scales = static_cast<size_t>(w.N) * (w.K / w.g) * 2;
        codes = buffer_of(w.codes(e), w.packed_bytes);
        alpha = buffer_of(w.alpha + w.scales(e), scales);
        beta = buffer_of(w.beta + w.scales(e), scales);
        at = (row / 16 * (w.K / 128) * 64 + 16 * h + row % 16) * BYTES;
        scale_at = row * (w.K / w.g) * 2;
    }
    // LOADS instructions
    __device__ __forceinline__ void fetch(RowPart& c, int chunk) const
    {
        const int from = chunk * 64 * BYTES, scale = chunk * 128 / g * 2;
        load_slot<FMT>(codes, at, from, c.code[0]);
        load_slot<FMT>(codes, at + 32 * BYTES, from, c.code[1]);
        c.alpha = __builtin_amdgcn_raw_buffer_load_b16(alpha, scale_at, scale, 0);
        c.beta = __builtin_amdgcn_raw_buffer_load_b16(beta, scale_at, scale, 0);
    }
};

constexpr int parts_of(int blocks) { return blocks >= 2 ? 4 : 2; }

// 2 x WN waves of RM x 4 blocks of 16 x 16.  TURN: the sum runs over the rows of W
// and the results are its columns (the input's gradient).  SPLIT: of every 64 rows of the
// tile the first 32 are the hi parts of 32 pairs, the others their lo parts; a wave has both,
// and adds their sums at the end.  (2062 pairs through 8 experts of 4096 x 14336 686 us for
// 444 in bf16, 8192 through 16 of 2048 x 1024 115 for 89: what is decoded serves as many
// products, of half as many pairs.  TURN: 2062 pairs back through 28672 x 4096 1800 for 1029, 8192
// through 2048 x 2048 271 for 179.)
//
// The matrix cores take a 16 x 16 x 32 product in 7.8 ns and let two vector instructions
// in for nothing; every further one costs its 1.9 ns.  Decoding is 4.2 instructions a
// product in tiles of 128 rows and 2.1 in tiles of 256, so those are the faster where
// there are rows for them (a step of 64 of 256 x 256: 1.9 us; four tiles of 128 x 128:
// 2.8): 1024 rows with 28672 x 4096 253 us, 950 TFLOP/s, for 300.  With one barrier a
// step and one workgroup a CU of 256 x 256, and 192 KB a step through LDS, half the
// time the matrix cores wait.  TURN pairs two rows' values before they are written: 1.0 us
// a step of 128 x 128 for 0.7.
//
// Tried and not kept: the weights decoded into the operands' registers, every wave with
// 32 columns and all rows of a tile, and x alone in LDS: 4096 rows with 28672 x 4096 in
// tiles of 128 x 128 1168 us for 1203, and 64 rows 44 for 46, since the lookups bound both;
// four waves of 128 x 128 each (accumulators moved between register files).
template <int FMT, int WN, int RM, bool TURN, bool SPLIT>
__global__ __launch_bounds__(128 * WN, WN == 2 ? 2 : 1) void k_tile(const TileArgs p)
{
    constexpr int THREADS = 128 * WN, BM = 32 * RM, BN = WN * 64, WAVES = 2 * WN, LA = BM / 8 / WAVES;
    constexpr int BP = SPLIT ? BM / 2 : BM, RP = SPLIT ? RM / 2 : RM;       // pairs of a tile, their blocks of a wave
    static_assert(LA >= 1, "every wave loads rows of x");
    static_assert(!SPLIT || (RM >= 2 && 4 % LA == 0), "what a wave loads are hi parts or lo parts");
    __shared__ __attribute__((aligned(16))) uint16_t sa0[BM * STEP], sb0[BN * STEP], sa1[BM * STEP], sb1[BN * STEP];
    __shared__ int pairs[BP];
    // forward: the tables of the rows at the places; TURN: byte tables of the next steps' rows
    __shared__ u32x4_t tables[TURN || FMT == FMT_INT4 || FMT == FMT_BF16 ? 1 : BN][FMT == FMT_ANY4 ? 2 : 1];
    __shared__ uint32_t turned[TURN ? 2 : 1][TURN ? BN / 128 : 1][TURN ? 2 * ByteTable<FMT>::ENTRIES / 4 : 1][STEP];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, g = lane >> 4;
    // Workgroups go to the eight XCDs in turn: each XCD gets a run of tiles whose
    // operands its L2 then shares, four rows of tiles high, or with experts all rows (some
    // of the last have no rows of x: every XCD gets its share of them).
    const int id = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8, HIGH = p.r.plan ? p.tiles_m : 4;
    if (id >= p.tiles_m * p.tiles_n)
        return;
    const int band = id / (HIGH * p.tiles_n), high = p.tiles_m - band * HIGH < HIGH ? p.tiles_m - band * HIGH : HIGH;
    const int in_band = id - band * HIGH * p.tiles_n;
    const int tm = __builtin_amdgcn_readfirstlane(band * HIGH + in_band % high), tn = __builtin_amdgcn_readfirstlane(in_band / high);
    int64_t first = 0;
    const Tile t = find_tile(p.r, tm, BP, first);
    if (t.e < 0)
        return;
    for (int i = tid; i < BP; i += THREADS)
        pairs[i] = i >= t.count ? -1 : p.r.plan ? p.r.plan[first + i] : tm * BP + i;
    __syncthreads();
    const bool gate = p.q.gated();
    const int col0 = gate ? tn * (BN / 2) : tn * BN;       // of out
    if (t.e == p.r.E) {              // no expert: zeros
        if (blockIdx.y == 0)
            for (int i = w; i < t.count; i += WAVES)
                for (int o = lane; o < (gate ? BN / 2 : BN); o += WAVE)
                    if (col0 + o < p.q.No) {
                        put_out(p.q, static_cast<size_t>(pairs[i]) * p.q.No + col0 + o, 0.0f);
                        if (p.q.z) {
                            const size_t z = static_cast<size_t>(pairs[i]) * p.q.N + col0 + o;
                            put_value(p.q.z, p.q.z32, z, 0.0f);
                            if (gate)
                                put_value(p.q.z, p.q.z32, z + p.q.No, 0.0f);
                        }
                    }
        return;
    }

    // x: a wave's load instruction fills 8 rows of a tile; lane: row lane / 8, place lane % 8
    const size_t plane = static_cast<size_t>(p.rows) * p.D;
    const __amdgpu_buffer_rsrc_t ra = buffer_of(p.x + (SPLIT && w * LA / 4 % 2 ? plane : 0), plane * 2);
    uint32_t ga[LA];
    int na[LA];                      // TURN: where the piece stands in the sum
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int r = (w * LA + i) * 8 + lane / 8, piece = (lane & 7) ^ key(r);
        const int pair = pairs[SPLIT ? r / 64 * 32 + r % 32 : r];
        ga[i] = pair < 0 ? OOR : static_cast<uint32_t>(pair / p.r.div) * (static_cast<uint32_t>(p.D) * 2u) + piece * 16u;
        na[i] = 8 * piece;
    }
    auto fetch = [&](int st, uint16_t* sa) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LA; ++i)
            load_lds(ra, sa + (w * LA + i) * 8 * STEP, static_cast<int>(TURN && st * STEP + na[i] >= p.D ? OOR : ga[i]), st * STEP * 2);
    };
    const int Kc = p.w.K / 128;

    f32x4_t acc[RM][4];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    // of every 32 rows of the tile a wave takes the first or the second 16
    const int wm = w / WN * 16, wn = (w % WN) * 64;
    const int blocks = __builtin_amdgcn_readfirstlane(t.count > wm ? (t.count - wm + 31) / 32 * (SPLIT ? 2 : 1) : 0);
    // operand reads: 16 or 32 rows on the key is the same, so one place each and
    // constant distances; the second half of a step is four pieces on.  (Kept from the
    // compiler, which would hold row and piece apart and add them every time.)
    int oa = (wm + c) * STEP + (g ^ key(wm + c)) * 8, ob = (wn + c) * STEP + (g ^ key(wn + c)) * 8;
    asm("" : "+v"(oa), "+v"(ob));
    auto operand_a = [&](const uint16_t* sa, int i, int kk) __attribute__((always_inline)) {
        return *reinterpret_cast<const bf16x8_t*>(sa + (oa ^ 32 * kk) + 32 * i * STEP);
    };
    auto operand_b = [&](const uint16_t* sb, int j, int kk) __attribute__((always_inline)) {
        return *reinterpret_cast<const bf16x8_t*>(sb + (ob ^ 32 * kk) + 16 * j * STEP);
    };
    // A step's products in parts, each with a share of the decoding, aside(part),
    // between them: a product leaves the vector ALU three issues in four, and what a
    // part decodes is written before the next begins, or the compiler keeps all of it
    // in registers.
    // Blocks: of 16 rows of the tile that the wave works on.
    auto multiply = [&](auto blocks_, const uint16_t* sa, const uint16_t* sb, auto aside) __attribute__((always_inline)) {
        constexpr int BLOCKS = decltype(blocks_)::value, PARTS = parts_of(BLOCKS), PER = 2 * BLOCKS / PARTS;
        bf16x8_t b[4];
        static_for<0, PARTS>([&](auto part_) __attribute__((always_inline)) {
            constexpr int part = decltype(part_)::value, kk = part * PER / BLOCKS;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (part * PER % BLOCKS == 0)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b[j] = operand_b(sb, j, kk);
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const int i = part * PER % BLOCKS + q;
                const bf16x8_t a = operand_a(sa, i, kk);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = mfma(b[j], a, acc[i][j]);
            }
            aside(part_);
        });
        __builtin_amdgcn_sched_barrier(0);
    };
    // this step's tiles are in, all but the wave's last n loads, and every wave has
    // read the other buffers
    auto meet = [&](auto n) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(decltype(n)::value) : "memory");
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    };
    typedef std::integral_constant<int, 0> All;
    typedef std::integral_constant<int, RowReader<FMT>::LOADS> AllButChunk;
    // the column of out and the row of W at a place
    auto row_of = [&](int place) __attribute__((always_inline)) {
        const int b = column_of(place), half = gate ? b >> 3 & 1 : 0;
        const int col = gate ? col0 + (place & ~63) / 2 + 8 * (b >> 4) + (b & 7) : col0 + (place & ~63) + b;
        return col < p.q.No ? col + half * p.q.No : 0;
    };
    auto run = [&](auto blocks_) __attribute__((always_inline)) {
        constexpr int PARTS = parts_of(decltype(blocks_)::value);
        auto product = [&](const uint16_t* sa, const uint16_t* sb, auto aside) __attribute__((always_inline)) {
            multiply(blocks_, sa, sb, aside);
        };
        if constexpr (TURN) {
            // A wave decodes 32 k of 64 rows (any 32 where the tile reaches past the last).
            // A row's byte table serves 128 k, four waves: four threads make a quarter each, two
            // steps ahead, and it lies in LDS.
            constexpr int QUARTERS = ByteTable<FMT>::ENTRIES / 4;
            const int s0 = share(p.steps, blockIdx.y, p.q.S), s1 = share(p.steps, blockIdx.y + 1, p.q.S);
            const int slot = col0 + 32 * w < p.w.K ? (col0 >> 5) + w : 0, chunk = slot >> 2, part = w & 3;
            const size_t scales = static_cast<size_t>(p.w.N) * (p.w.K / p.w.g) * 2;
            const __amdgpu_buffer_rsrc_t codes = buffer_of(p.w.codes(t.e), p.w.packed_bytes),
                                         alpha = buffer_of(p.w.alpha + p.w.scales(t.e), scales),
                                         beta = buffer_of(p.w.beta + p.w.scales(t.e), scales);
            const uint16_t* lut = FMT == FMT_INT4 ? nullptr : p.w.table(t.e);
            const int tile_pitch = Kc * 64 * slot_bytes(FMT);
            const int at = (lane >> 4) * tile_pitch + ((slot & 3) * 16 + (lane & 15)) * slot_bytes(FMT);
            uint32_t code[4];
            struct {
                u32x2_t entries;
                uint32_t alpha, beta;
            } row;
            auto fetch_row = [&](int st) __attribute__((always_inline)) {     // for a quarter of a table
                const int n = st * STEP + lane < p.w.N ? st * STEP + lane : 0, at_scale = n * (p.w.K / p.w.g) * 2;
                row.alpha = __builtin_amdgcn_raw_buffer_load_b16(alpha, at_scale, chunk * 128 / p.w.g * 2, 0);
                row.beta = __builtin_amdgcn_raw_buffer_load_b16(beta, at_scale, chunk * 128 / p.w.g * 2, 0);
                typedef u32x2_t __attribute__((aligned(2))) entries_t;
                if constexpr (FMT != FMT_INT4)
                    row.entries = *reinterpret_cast<const entries_t*>(lut + static_cast<size_t>(n) * 16 + 4 * part);
            };
            auto make_table = [&](int st, int buffer) __attribute__((always_inline)) {
                const float fa = bf16_to_f32(row.alpha), fb = bf16_to_f32(row.beta);
                uint32_t v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float x = FMT == FMT_INT4 ? static_cast<float>(4 * part + 2 * i) : __uint_as_float(row.entries[i] << 16);
                    const float y = FMT == FMT_INT4 ? static_cast<float>(4 * part + 2 * i + 1) : __uint_as_float(row.entries[i] & 0xffff0000u);
                    v[i] = f32_to_bf16(fmaf(fa, x, fb)) | f32_to_bf16(fmaf(fa, y, fb)) << 16;
                }
                const bool in = st * STEP + lane < p.w.N;                  // rows behind the last: weights of 0
                if (part < QUARTERS) {
                    turned[buffer][w >> 2][part][lane] = in ? __builtin_amdgcn_perm(v[1], v[0], 0x06040200u) : 0u;
                    turned[buffer][w >> 2][QUARTERS + part][lane] = in ? __builtin_amdgcn_perm(v[1], v[0], 0x07050301u) : 0u;
                }
            };
            auto fetch_weights = [&](int st) __attribute__((always_inline)) {
                load_slot<FMT>(codes, at, (st * (STEP / 16) * Kc + chunk) * 64 * slot_bytes(FMT), code);
            };
            ByteTable<FMT> table;
            auto read_table = [&](int buffer) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < QUARTERS; ++i) {
                    table.lo[i] = turned[buffer][w >> 2][i][lane];
                    table.hi[i] = turned[buffer][w >> 2][QUARTERS + i][lane];
                }
            };
            auto unpack = [&](int i, uint16_t* sb) __attribute__((always_inline)) {
                uint32_t v[4];
                decode8(table, code, i, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int b = 32 * (w & 1) + 8 * i + 2 * j + (lane & 1);         // of the 64 k of two waves
                    const int to = 64 * (w >> 1) + 16 * (b >> 2 & 3) + 4 * (b >> 4) + (b & 3);
                    reinterpret_cast<uint32_t*>(sb)[to * (STEP / 2) + ((lane >> 3) ^ key(to)) * 4 + (lane >> 1 & 3)] = pair_rows(v[j], lane & 1);
                }
            };
            // what lies past the last step is fetched and decoded for nothing: there is no
            // branch between the products
            auto near = [&](int st) __attribute__((always_inline)) { return st < s1 ? st : s1 - 1; };
            auto step = [&](int st, uint16_t* sa, uint16_t* sb, uint16_t* sa_next, uint16_t* sb_next) __attribute__((always_inline)) {
                meet(All{});
                fetch(near(st + 1), sa_next);
                make_table(near(st + 2), st - s0 & 1);
                fetch_row(near(st + 3));
                read_table(st + 1 - s0 & 1);
                product(sa, sb, [&](auto n) __attribute__((always_inline)) {
#pragma unroll
                    for (int i = 0; i < 4 / PARTS; ++i)
                        unpack(4 / PARTS * decltype(n)::value + i, sb_next);
                });
                fetch_weights(near(st + 2));
            };
            fetch_row(s0);
            make_table(s0, 0);
            fetch_row(near(s0 + 1));
            make_table(near(s0 + 1), 1);
            fetch(s0, sa0);
            fetch_weights(s0);
            fetch_row(near(s0 + 2));
            __syncthreads();
            read_table(0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                unpack(i, sb0);
            fetch_weights(near(s0 + 1));
            int st = s0;
            for (; st + 1 < s1; st += 2) {
                step(st, sa0, sb0, sa1, sb1);
                step(st + 1, sa1, sb1, sa0, sb0);
            }
            if (st < s1)
                step(st, sa0, sb0, sa1, sb1);
        } else if constexpr (FMT == FMT_BF16) {
            constexpr int LB = BN / 8 / WAVES;
            const int s0 = share(p.steps, blockIdx.y, p.q.S), s1 = share(p.steps, blockIdx.y + 1, p.q.S);
            const __amdgpu_buffer_rsrc_t rb = buffer_of(p.w.packed, static_cast<size_t>(p.w.N) * p.w.K * 2);
            uint32_t gb[LB];
#pragma unroll
            for (int i = 0; i < LB; ++i) {
                const int r = (w * LB + i) * 8 + lane / 8;
                gb[i] = static_cast<uint32_t>(row_of(r)) * (static_cast<uint32_t>(p.w.K) * 2u) + ((lane & 7) ^ key(r)) * 16u;
            }
            auto fetch_both = [&](int st, uint16_t* sa, uint16_t* sb) __attribute__((always_inline)) {
                fetch(st, sa);
#pragma unroll
                for (int i = 0; i < LB; ++i)
                    load_lds(rb, sb + (w * LB + i) * 8 * STEP, static_cast<int>(gb[i]), st * STEP * 2);
            };
            fetch_both(s0, sa0, sb0);
            int st = s0;
            for (; st + 1 < s1; st += 2) {
                meet(All{});
                fetch_both(st + 1, sa1, sb1);
                product(sa0, sb0, [](auto) {});
                meet(All{});
                fetch_both(st + 2 < s1 ? st + 2 : s0, sa0, sb0);
                product(sa1, sb1, [](auto) {});
            }
            meet(All{});
            if (st < s1)
                product(sa0, sb0, [](auto) {});
        } else {
            // chunks of two steps; thread h of the row at a place has half h of each step's k
            const int c0 = share(Kc, blockIdx.y, p.q.S), c1 = share(Kc, blockIdx.y + 1, p.q.S);
            const int place = tid % BN, h = tid / BN;
            const int wr = row_of(place);
            const RowReader<FMT> reader(p.w, t.e, wr, h);
            int ow = place * STEP + (4 * h ^ key(place)) * 8;        // where the first goes; the i-th at ow ^ 8 i
            asm("" : "+v"(ow));
            if constexpr (FMT != FMT_INT4) {
                if (h == 0) {
                    const RowTable row = fetch_table<FMT>(p.w.table(t.e), p.w.alpha + p.w.scales(t.e), p.w.beta + p.w.scales(t.e), wr, Kc, c0, p.w.g);
#pragma unroll
                    for (int i = 0; i < (FMT == FMT_ANY4 ? 2 : 1); ++i)
                        tables[place][i] = row.table[i];
                }
                __syncthreads();
            }
            RowPart A, B;
            ByteTable<FMT> table;
            // a chunk's table serves both its steps
            auto tabulate = [&](const RowPart& from) __attribute__((always_inline)) {
                RowTable row;
                row.table[0] = row.table[1] = u32x4_t{0u, 0u, 0u, 0u};
                if constexpr (FMT != FMT_INT4)
#pragma unroll
                    for (int i = 0; i < (FMT == FMT_ANY4 ? 2 : 1); ++i)
                        row.table[i] = tables[place][i];
                row.alpha = from.alpha;
                row.beta = from.beta;
                return ByteTable<FMT>(row);
            };
            auto unpack = [&](const RowPart& from, int which, int i, uint16_t* sb) __attribute__((always_inline)) {
                uint32_t v[4];
                decode8(table, from.code[which], i, v);
                *reinterpret_cast<u32x4_t*>(sb + (ow ^ 8 * i)) = u32x4_t{v[0], v[1], v[2], v[3]};
            };
            // The first step of a chunk: its second half is decoded, and the chunk after
            // the next asked for; the second step decodes the next chunk's first half.
            // (Past the last chunk both do so for nothing: a branch would keep the decoding
            // from standing between the products.)
            auto first_step = [&](int ch, RowPart& mine) __attribute__((always_inline)) {
                fetch(2 * ch + 1, sa1);
                product(sa0, sb0, [&](auto part) __attribute__((always_inline)) {
                    constexpr int n = decltype(part)::value, share = 4 / PARTS;
#pragma unroll
                    for (int i = 0; i < share; ++i)
                        unpack(mine, 1, share * n + i, sb1);
                });
                reader.fetch(mine, ch + 2 < c1 ? ch + 2 : c0);
            };
            auto second_step = [&](int ch, const RowPart& other) __attribute__((always_inline)) {
                fetch(ch + 1 < c1 ? 2 * ch + 2 : 2 * c0, sa0);
                product(sa1, sb1, [&](auto part) __attribute__((always_inline)) {
                    constexpr int n = decltype(part)::value;
                    if constexpr (n == 0)
                        table = tabulate(other);
                    // four parts: the table, then one, one and two eighths of 32 weights
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (PARTS == 4 ? n == (i < 2 ? i + 1 : 3) : n == i / 2)
                            unpack(other, 0, i, sb0);
                });
            };
            reader.fetch(A, c0);
            reader.fetch(B, c0 + 1 < c1 ? c0 + 1 : c0);
            fetch(2 * c0, sa0);
            table = tabulate(A);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                unpack(A, 0, i, sb0);
            int ch = c0;
            for (; ch + 1 < c1; ch += 2) {
                meet(All{});
                first_step(ch, A);
                meet(AllButChunk{});
                second_step(ch, B);
                meet(All{});
                first_step(ch + 1, B);
                meet(AllButChunk{});
                second_step(ch + 1, A);
            }
            if (ch < c1) {
                meet(All{});
                first_step(ch, A);
                meet(All{});         // no chunk is asked for here: the last loads are the tile's own
                second_step(ch, B);
            }
        }
    };
    // rows behind the last are zeros; where they fill half of the wave's blocks, those
    // are left out
    if (RM > 1 && blocks <= RM / 2)
        run(std::integral_constant<int, (RM > 1 ? RM / 2 : 1)>{});
    else
        run(std::integral_constant<int, RM>{});
    if constexpr (SPLIT)
#pragma unroll
        for (int i = 0; i < RP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = acc[2 * i][j] + acc[2 * i + 1][j];
    // The sums leave through LDS of the wave's own, so that lanes next to one another
    // write columns next to one another: 16 pieces of four floats a row, piece q at
    // q ^ row.  With a gate its columns come first, those of the up rows behind.
    meet(All{});
    constexpr int ROOM = (BM < BN ? BM : BN) * STEP * 2 / (WAVES / 4);          // bytes of a wave
    constexpr int HALVES = 16 * RP * 256 > ROOM ? 2 : 1, ROWS = 16 * RP / HALVES;
    static_assert(ROWS * 256 <= ROOM, "the waves' rooms lie in the four buffers");
    const int room = w * 4 / WAVES;       // a wave's, or two waves', of the four buffers
    uint16_t* const in = room == 0 ? sa0 : room == 1 ? sb0 : room == 2 ? sa1 : sb1;
    f32x4_t* stage = reinterpret_cast<f32x4_t*>(in) + w % (WAVES / 4) * (ROWS * 16);
    const int lane2 = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)), c2 = lane2 & 15, g2 = lane2 >> 4;   // no register for them until here
    const int pieces = gate ? 4 : 8;       // of eight columns of out a row
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
        wave_sync();
#pragma unroll
        for (int i = 0; i < RP / HALVES; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int to = gate ? 8 * (j >> 1) + 2 * g2 + (j & 1) : 4 * g2 + j;
                stage[(16 * i + c2) * 16 + (to ^ c2)] = acc[half * (RP / HALVES) + i][j];
            }
        wave_sync();
        for (int o = lane2; o < ROWS * pieces; o += WAVE) {
            const int row = o / pieces, q = o % pieces;
            const int pair = pairs[32 * (half * (RP / HALVES) + row / 16) + wm + row % 16];
            const int col = col0 + (gate ? wn / 2 : wn) + 8 * q;
            if (pair < 0 || col >= p.q.No)
                continue;
            f32x4_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = stage[row * 16 + ((2 * q + (e & 1) + (gate ? 8 * (e >> 1) : 0)) ^ (row & 15))];
            if (p.q.part) {
                float* to = p.q.part + (static_cast<size_t>(blockIdx.y) * p.r.P + pair) * p.q.N + col;
                put8(to, f[0], f[1], p.q.No - col);
                if (gate)
                    put8(to + p.q.No, f[2], f[3], p.q.No - col);
                continue;
            }
            float v[8], u[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = f[0][e];
                v[4 + e] = f[1][e];
                u[e] = f[2][e];
                u[4 + e] = f[3][e];
            }
            finish8(p.q, t.e, pair, col, v, u);
        }
    }
}

// ---------------------------------------------------------------------------
// many rows: the layer laid out as bf16 once, for k_tile<FMT_BF16>
// ---------------------------------------------------------------------------
// A wave decodes a packed tile of 16 rows x 128 k and turns it in LDS of its own,
// so that it leaves in whole pieces of rows.  Bound by its bytes (28672 x 4096, 298 MB:
// 53 us, 5.6 TB/s).  A call of 4096 rows takes 864 to 885 us with it, a library's product alone 722.
constexpr int ROWS_WAVES = 4;

template <int FMT>
__global__ __launch_bounds__(64 * ROWS_WAVES) void k_rows(const Layer layer, uint16_t* __restrict__ to)
{
    __shared__ u32x4_t room[ROWS_WAVES][16 * 16];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int Kc = layer.K / 128, per = (Kc + ROWS_WAVES - 1) / ROWS_WAVES;
    const int chunk = blockIdx.x % per * ROWS_WAVES + w, block = blockIdx.x / per;
    if (chunk >= Kc)
        return;
    const int n = block * 16 + c < layer.N ? block * 16 + c : layer.N - 1;
    uint32_t code[4], v[16];
    fetch_codes<FMT>(layer.packed, n, Kc, chunk, g, code);
    decode_in_order(ByteTable<FMT>(fetch_table<FMT>(layer.lut, layer.alpha, layer.beta, n, Kc, chunk, layer.g)), code, v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        room[w][c * 16 + ((4 * g + i) ^ c)] = u32x4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    wave_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + g;
        if (block * 16 + r < layer.N)
            *reinterpret_cast<u32x4_t*>(to + static_cast<size_t>(block * 16 + r) * layer.K + chunk * 128 + 8 * c) = room[w][r * 16 + (c ^ r)];
    }
}

// ---------------------------------------------------------------------------
// the activation's backward pass
// ---------------------------------------------------------------------------
struct BwdArgs {
    const void *dy, *z;
    uint16_t* dz;            // [M][N], in parts [2][M][N]
    float* part;             // [slabs][N] or null: no bias
    int M, N, No, act, slab; // rows of a workgroup
};

// Of eight columns: a what dz is, or with a gate its half of the gate's rows, b the up rows'.
template <bool GATE>
__device__ __forceinline__ void gradients(const float (&d)[8], const float (&zg)[8], const float (&zu)[8], int act, float (&a)[8], float (&b)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f, slope;
        activate_both(zg[i], act, f, slope);
        a[i] = d[i] * slope;
        if constexpr (GATE) {
            a[i] *= zu[i];
            b[i] = d[i] * f;
        }
    }
}

constexpr int BWD_COLS = 8 * WAVE;           // columns of out of a workgroup

constexpr int BWD_FEW = 128;                 // rows of the one slab of few

// LANES of a wave take eight columns each, its other lanes other rows: 512 columns of
// every fourth row of a slab, two rows at a time (LANES 64, four waves), or 64 columns of
// 64 rows at a time (LANES 8, eight waves).  The column sums meet in LDS.  Bound by its bytes.  What the loads depend
// on is known to the compiler, and a row past the last is the last again: a branch
// between them would make each wait for the one before.  4096 x 28672, gated, 587 MB:
// 117 us, 5.0 TB/s, a copy's rate.
template <bool DY32, bool Z32, bool GATE, bool WHOLE, bool SPLIT, int WAVES, int LANES>
__global__ __launch_bounds__(WAVE * WAVES) void k_act_bwd(const BwdArgs p)
{
    constexpr int COLS = 8 * LANES, AT_ONCE = WAVES * (WAVE / LANES), ROWS = WAVES == 4 ? 2 : 1;
    __shared__ float red[AT_ONCE][GATE ? 2 : 1][8][LANES];
    const int lane = threadIdx.x % LANES, w = threadIdx.x / LANES, col = blockIdx.x * COLS + 8 * lane;
    const int m0 = blockIdx.y * p.slab, m1 = m0 + p.slab < p.M ? m0 + p.slab : p.M;
    const int left = p.No - col, valid = WHOLE ? 8 : left;
    float sum[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sum[0][i] = sum[1][i] = 0.0f;
    for (int m = m0 + w; m < m1; m += AT_ONCE * ROWS) {
        if (left <= 0)
            break;
        float d[ROWS][8], zg[ROWS][8], zu[ROWS][8];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const size_t row = m + AT_ONCE * r < m1 ? m + AT_ONCE * r : m;
            get_values(p.dy, DY32, row * p.No + col, valid, d[r]);
            get_values(p.z, Z32, row * p.N + col, valid, zg[r]);
            if constexpr (GATE)
                get_values(p.z, Z32, row * p.N + p.No + col, valid, zu[r]);
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (m + AT_ONCE * r >= m1)
                break;
            float a[8], b[8];
            gradients<GATE>(d[r], zg[r], zu[r], p.act, a, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0][i] += a[i];
                if constexpr (GATE)
                    sum[1][i] += b[i];
            }
            const size_t at = static_cast<size_t>(m + AT_ONCE * r) * p.N + col;
            auto put = [&](size_t to, const float (&v)[8]) __attribute__((always_inline)) {
                if constexpr (SPLIT)
                    put_parts(p.dz + to, static_cast<size_t>(p.M) * p.N, valid, v);
                else
                    put_values(p.dz, 0, to, valid, v);
            };
            put(at, a);
            if constexpr (GATE)
                put(at + p.No, b);
        }
    }
    if (!p.part)
        return;
#pragma unroll
    for (int h = 0; h < (GATE ? 2 : 1); ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            red[w][h][i][lane] = sum[h][i];
    __syncthreads();
    for (int i = threadIdx.x; i < (GATE ? 2 : 1) * COLS; i += WAVE * WAVES) {
        const int h = i / COLS, o = i % COLS, c = blockIdx.x * COLS + o;
        if (c >= p.No)
            continue;
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            v += red[j][h][o & 7][o >> 3];
        p.part[static_cast<size_t>(blockIdx.y) * p.N + h * p.No + c] = v;
    }
}

// The slabs' sums: 64 columns a workgroup, every wave a quarter of the slabs, eight
// loads at a time (one thread a column: 18.6 us for 74 slabs of 28672).
__global__ __launch_bounds__(256) void k_bias_sum(const float* __restrict__ part, float* __restrict__ dbias, int N, int slabs)
{
    __shared__ float red[4][WAVE];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = blockIdx.x * WAVE + lane;
    float v = 0.0f;
    if (n < N)
        for (int s0 = w; s0 < slabs; s0 += 32) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = s0 + 4 * i < slabs ? part[static_cast<size_t>(s0 + 4 * i) * N + n] : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v += x[i];
        }
    red[w][lane] = v;
    __syncthreads();
    if (w == 0 && n < N)
        dbias[n] = red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane];
}

// ---------------------------------------------------------------------------
// the gradient of the experts' bias
// ---------------------------------------------------------------------------
struct ExpertBiasArgs {
    const void *dy, *z;
    const int* plan;         // null: no pairs
    float *dbias, *part;     // [E][N], [slots][N]
    int P, E, N, No, act;

    __device__ __forceinline__ bool fits() const { return !plan || (plan[2] == P && plan[3] == E); }
};

// The sums over one expert's pairs, 64 columns and a chunk of the plan (up to 512 pairs) a
// workgroup: eight lanes have a pair's columns, 64 pairs at a time, whose sums meet in LDS.  In
// the plan's order, so that they are the same each time.  Bound by its bytes: 2062 pairs of 28672
// columns in fp32, gated, 355 MB: 69 us, 5.1 TB/s; 8192 of 2048 through 16 experts 24 us.
template <bool DY32, bool Z32, bool GATE, bool WHOLE>
__global__ __launch_bounds__(8 * WAVE) void k_expert_bias(const ExpertBiasArgs p)
{
    constexpr int LANES = 8, COLS = 8 * LANES, AT_ONCE = 8 * WAVE / LANES;
    __shared__ float red[AT_ONCE][GATE ? 2 : 1][8][LANES];
    if (!p.fits() || static_cast<int>(blockIdx.y) >= p.plan[1])
        return;
    const PlanLayout l(p.P, p.E);
    const int* chunk = p.plan + l.chunk + 4 * static_cast<int64_t>(blockIdx.y);
    const int* pairs = p.plan + l.rows + chunk[1];
    const int count = chunk[2], slot = chunk[3];
    const int lane = threadIdx.x % LANES, w = threadIdx.x / LANES, col = blockIdx.x * COLS + 8 * lane;
    const int left = p.No - col, valid = WHOLE ? 8 : left;
    float sum[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sum[0][i] = sum[1][i] = 0.0f;
    for (int m = w; m < count && left > 0; m += AT_ONCE) {
        const size_t row = pairs[m];
        float d[8], zg[8], zu[8], a[8], b[8];
        get_values(p.dy, DY32, row * p.No + col, valid, d);
        get_values(p.z, Z32, row * p.N + col, valid, zg);
        if constexpr (GATE)
            get_values(p.z, Z32, row * p.N + p.No + col, valid, zu);
        gradients<GATE>(d, zg, zu, p.act, a, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum[0][i] += a[i];
            if constexpr (GATE)
                sum[1][i] += b[i];
        }
    }
#pragma unroll
    for (int h = 0; h < (GATE ? 2 : 1); ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            red[w][h][i][lane] = sum[h][i];
    __syncthreads();
    float* to = slot < 0 ? p.dbias + static_cast<size_t>(chunk[0]) * p.N : p.part + static_cast<size_t>(slot) * p.N;
    for (int i = threadIdx.x; i < (GATE ? 2 : 1) * COLS; i += 8 * WAVE) {
        const int h = i / COLS, o = i % COLS, c = blockIdx.x * COLS + o;
        if (c >= p.No)
            continue;
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            v += red[j][h][o & 7][o >> 3];
        to[h * p.No + c] = v;
    }
}

// Experts of several chunks: their sums in order; those without a pair: zeros.
__global__ __launch_bounds__(256) void k_expert_bias_sum(const ExpertBiasArgs p)
{
    const int e = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
    if (n >= p.N || !p.fits())
        return;
    const PlanLayout l(p.P, p.E);
    const int chunks = p.plan ? (p.plan[l.count + e] + CHUNK - 1) / CHUNK : 0;
    if (chunks == 1)                 // there already
        return;
    const float* part = chunks ? p.part + static_cast<size_t>(p.plan[l.slot + e]) * p.N + n : nullptr;
    float v = 0.0f;
    for (int i0 = 0; i0 < chunks; i0 += 8) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = i0 + i < chunks ? part[static_cast<size_t>(i0 + i) * p.N] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v += x[i];
    }
    p.dbias[static_cast<size_t>(e) * p.N + n] = v;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int64_t GIB2 = static_cast<int64_t>(1) << 31;

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

size_t layer_bytes(int fmt, int64_t N, int64_t K)
{
    return static_cast<size_t>((N + 15) / 16 * 16) * (K / 8) * (fmt == FMT_ANY2 ? 2 : fmt == FMT_ANY3 ? 3 : 4);
}

// How a product is run: the tile of k_tile (rm 0: k_few of 2 wn waves), its number and
// the splits.
struct Shape {
    int rm, wn, S;
    int64_t tiles_m, tiles_n;
    bool rows;               // the layer is laid out first
};

int64_t few_tiles(int64_t P, int64_t E, bool experts)
{
    if (!experts)
        return (P + FEW_T - 1) / FEW_T;
    if (P <= FEW_P)
        return P / FEW_T + (P < E + 1 ? P : E + 1);
    return PlanLayout(P, E).TB * (TILE_T / FEW_T);
}

// What a step of 64 was measured to take, in units of 10 ns, of one workgroup that
// has its CU to itself and for each of several (28672 x 4096, 4096 x 14336 and
// 2048 x 2048, one layer of 16 to 4096 rows and 8 to 64 experts; forward, and turned).
struct Form {
    int rm, wn, one[2], more[2];
};
constexpr Form FORMS[] = {{8, 4, {190, 0}, {200, 0}}, {4, 2, {120, 140}, {71, 100}}, {2, 2, {88, 110}, {48, 63}}, {1, 2, {75, 100}, {38, 52}}};
constexpr Form ROWS_FORM = {8, 4, {168, 0}, {180, 0}};
// the same for a chunk of 128 of a wave of k_few, by its rows of x (up to 4, 8, 16), in bf16 and
// in parts (through 8 experts of 4096 x 14336 8 pairs 54 and 56 us, 64 pairs 76 and 107)
constexpr int FEW_TIME[2][3] = {{195, 215, 300}, {205, 290, 430}};

// pairs of a tile of rm blocks
int64_t tile_pairs(int rm, bool parts) { return parts ? 16 * rm : 32 * rm; }

// P rows through E experts (experts = false: one layer), D summed, C columns of the
// product (both halves of a gate).  Of the forms and splits the one with the least
// time for the CU with the most workgroups, splits with their partial sums' bytes
// and a launch.  Rows fall on experts at random: the last tile of each is half empty.
Shape shape_of(int64_t P, int64_t E, bool experts, int64_t D, int64_t C, bool turn, bool parts = false)
{
    Shape s{0, 2, 1, 0, 0, false};
    const int64_t each = (P + E - 1) / E;        // rows of an expert, on average
    // experts that some pair names: 5.3 of 8 for 8 pairs (4096 x 14336: two splits, 49 us for 60)
    const double named = experts ? E * (1.0 - std::pow(1.0 - 1.0 / E, static_cast<double>(P))) : 1.0;
    int64_t least = INT64_MAX;
    auto better = [&](int64_t time, int rm, int wn, int64_t n, bool rows) {
        time += n > 1 ? 400 + n * P * C / 8000 : 0;
        if (time >= least)
            return;
        least = time;
        s.rm = rm;
        s.wn = wn;
        s.S = static_cast<int>(n);
        s.rows = rows;
    };
    // Eight waves a workgroup where they are few (28672 x 4096 in 448: the same; 4096 x 4096
    // in 64: 11.9 us for 13.6), four where there are many or a wave had less than four
    // chunks (64 experts of 2048 x 2048, 1 token 8.2 us for 11.8, 8 tokens 28 for 40; two
    // of eight 28672 x 4096, 896 workgroups: the same).
    if (!turn && (!experts || P <= FEW_P || each <= 64)) {
        const int64_t chunks = D / 128;
        const int rows = each <= 4 ? 0 : each <= 8 ? 1 : 2;
        const double row_tiles = experts ? named * (each < 8 ? 4 : each / 4 + 2) / 4 : static_cast<double>((P + FEW_T - 1) / FEW_T);
        const int64_t tiles = static_cast<int64_t>((C + FEW_ROWS - 1) / FEW_ROWS * row_tiles + 0.5);
        for (int64_t n = 1; n <= 8 && (n == 1 || chunks / n >= 8); n *= 2)
            better((tiles * n + 255) / 256 * FEW_TIME[parts][rows] * ((chunks + 8 * n - 1) / (8 * n)) + (n > 1 ? 250 : 0), 0,
                   tiles * n >= 1024 || chunks < 32 ? 2 : 4, n, false);
    }
    const int64_t steps = (D + STEP - 1) / STEP;
    auto weigh = [&](const Form& f, int64_t before, bool rows) {
        const int64_t bm = tile_pairs(f.rm, parts), bn = 64 * f.wn, tiles_n = (C + bn - 1) / bn;
        // in quarters
        const int64_t a_tile = 4 * each < bm ? 4 : 4 * each < 3 * bm ? 5 : 4 * each / bm + 2;
        const int64_t tiles_m = experts ? static_cast<int64_t>(named * a_tile + 0.5) : 4 * ((P + bm - 1) / bm);
        for (int64_t n = 1; n <= 8 && (n == 1 || steps / n >= 8); ++n) {
            const int64_t tiles = tiles_m * tiles_n * n, on_cu = (tiles + 1023) / 1024 * 1024;
            const int64_t all = (on_cu < (turn ? 2 : 3) * 1024 ? on_cu : tiles + 512) * f.more[turn] / 1024;
            better(before + 300 + (all > f.one[turn] ? all : f.one[turn]) * ((steps + n - 1) / n), f.rm, f.wn, n, rows);
        }
    };
    if (turn || !experts || P > FEW_P)           // fewer pairs have no plan forward
        for (const Form& f : FORMS)
            if (f.one[turn] && !(parts && f.rm == 1))
                weigh(f, 0, false);
    if (!experts && !turn && C * D < GIB2 / 2)
        weigh(ROWS_FORM, 300 + C * D / 22000, true);       // 2.5 bytes a weight at 5.5 TB/s
    if (s.rm == 0) {
        s.tiles_m = few_tiles(P, E, experts);
        s.tiles_n = (C + FEW_ROWS - 1) / FEW_ROWS;
        return s;
    }
    const int64_t bm = tile_pairs(s.rm, parts), bn = 64 * s.wn;
    s.tiles_m = experts ? P / bm + (P < E + 1 ? P : E + 1) : (P + bm - 1) / bm;
    s.tiles_n = (C + bn - 1) / bn;
    return s;
}

size_t part_bytes(const Shape& s, int64_t P, int64_t C, int64_t D)
{
    return (s.S > 1 ? up256(static_cast<size_t>(s.S) * P * C * 4) : 0) + (s.rows ? up256(static_cast<size_t>(C) * D * 2) : 0);
}

template <int FMT, bool TURN, bool SPLIT>
void launch_tile(const Shape& s, const TileArgs& a, hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((s.tiles_m * s.tiles_n + 7) / 8 * 8), static_cast<unsigned>(s.S));
#define TILE(WN_, RM_) hipLaunchKernelGGL((k_tile<FMT, WN_, RM_, TURN, SPLIT>), grid, dim3(128 * WN_), 0, stream, a)
    if constexpr (FMT == FMT_BF16) {
        TILE(4, 8);
    } else {
        if (s.rm == 4) TILE(2, 4);
        else if (s.rm == 2) TILE(2, 2);
        else if (s.rm == 8) {
            if constexpr (!TURN) TILE(4, 8);
        } else {
            if constexpr (!SPLIT) TILE(2, 1);
        }
    }
#undef TILE
}

template <bool TURN, bool SPLIT>
void launch_tile(int fmt, const Shape& s, const TileArgs& a, hipStream_t stream)
{
    if (fmt == FMT_ANY4) launch_tile<FMT_ANY4, TURN, SPLIT>(s, a, stream);
    else if (fmt == FMT_INT4) launch_tile<FMT_INT4, TURN, SPLIT>(s, a, stream);
    else if (fmt == FMT_ANY2) launch_tile<FMT_ANY2, TURN, SPLIT>(s, a, stream);
    else launch_tile<FMT_ANY3, TURN, SPLIT>(s, a, stream);
}

template <int FMT, int X>
void launch_few(const Shape& s, const FewArgs& a, hipStream_t stream)
{
    const int per = a.q.gated() ? FEW_ROWS / 2 : FEW_ROWS;
    const dim3 grid(static_cast<unsigned>((a.q.No + per - 1) / per), static_cast<unsigned>(s.tiles_m), static_cast<unsigned>(s.S));
    if (s.wn == 2)
        hipLaunchKernelGGL((k_few<FMT, 4, X>), grid, dim3(4 * WAVE), 0, stream, a);
    else
        hipLaunchKernelGGL((k_few<FMT, 8, X>), grid, dim3(8 * WAVE), 0, stream, a);
}

template <int X>
void launch_few(int fmt, const Shape& s, const FewArgs& a, hipStream_t stream)
{
    if (fmt == FMT_ANY4) launch_few<FMT_ANY4, X>(s, a, stream);
    else if (fmt == FMT_INT4) launch_few<FMT_INT4, X>(s, a, stream);
    else if (fmt == FMT_ANY2) launch_few<FMT_ANY2, X>(s, a, stream);
    else launch_few<FMT_ANY3, X>(s, a, stream);
}

bool act_ok(int act) { return act >= 0 && act < ACTS; }
bool fmt_ok(int fmt) { return fmt >= FMT_ANY4 && fmt <= FMT_ANY3; }

// P rows of out [P][No], x [X][K], a layer [N][K] of each of E experts
bool sizes_ok(int64_t P, int64_t X, int64_t E, int64_t N, int64_t K, int64_t g)
{
    return P >= 0 && P <= MAX_PAIRS && X >= 0 && E >= 1 && E <= MAX_EXPERTS && N >= 0 && N < GIB2 / 2 && K > 0 && K < GIB2 / 2 &&
           g > 0 && g % 128 == 0 && K % g == 0 && (N + 15) / 16 * 16 * K < 2 * GIB2 && (P == 0 || N < GIB2 / 2 / P) && (X == 0 || K < GIB2 / 2 / X);
}

// kind: of x's rows
any4_status product(int fmt, const Rows& rows, int64_t X, const void* x, int kind, const Layer& w, const Epilogue& q, const int32_t* ids,
                    void* workspace, size_t workspace_bytes, bool experts, hipStream_t stream)
{
    const Shape s = shape_of(rows.P, rows.E, experts, w.K, w.N, false, kind == X_PARTS);
    char* at = static_cast<char*>(workspace);
    Rows r = rows;
    Epilogue e = q;
    e.S = s.S;
    const size_t need = part_bytes(s, r.P, w.N, w.K);
    if (experts && r.P <= FEW_P) {
        r.plan = nullptr;
        r.ids = ids;
    } else if (experts && !r.plan) {
        const size_t bytes = any4_lora_plan_bytes(r.P, r.E);
        if (workspace_bytes < need + bytes || !workspace)
            return workspace ? ANY4_E_WORKSPACE : ANY4_E_NULL;
        const any4_status st = any4_lora_plan(ids, at, bytes, r.P, r.E, stream);
        if (st != ANY4_OK)
            return st;
        r.plan = reinterpret_cast<const int*>(at);
        at += up256(bytes);
        workspace_bytes -= bytes;
    }
    if (need && (workspace_bytes < need || !workspace))
        return workspace ? ANY4_E_WORKSPACE : ANY4_E_NULL;
    if (s.S > 1)
        e.part = reinterpret_cast<float*>(at);
    if (s.rm == 0) {
        const FewArgs a{r, w, x, e, static_cast<size_t>(X) * w.K};
        if (kind == X_F32) launch_few<X_F32>(fmt, s, a, stream);
        else if (kind == X_PARTS) launch_few<X_PARTS>(fmt, s, a, stream);
        else launch_few<X_BF16>(fmt, s, a, stream);
    } else if (s.rows) {
        uint16_t* rows = reinterpret_cast<uint16_t*>(at + (s.S > 1 ? up256(static_cast<size_t>(s.S) * r.P * w.N * 4) : 0));
        const int Kc = w.K / 128;
        const dim3 grid(static_cast<unsigned>((w.N + 15) / 16) * ((Kc + ROWS_WAVES - 1) / ROWS_WAVES));
#define LAY_OUT(FMT_) hipLaunchKernelGGL(k_rows<FMT_>, grid, dim3(64 * ROWS_WAVES), 0, stream, w, rows)
        if (fmt == FMT_ANY4) LAY_OUT(FMT_ANY4);
        else if (fmt == FMT_INT4) LAY_OUT(FMT_INT4);
        else if (fmt == FMT_ANY2) LAY_OUT(FMT_ANY2);
        else LAY_OUT(FMT_ANY3);
#undef LAY_OUT
        Layer laid = w;
        laid.packed = reinterpret_cast<const uint8_t*>(rows);
        launch_tile<FMT_BF16, false, false>(s, TileArgs{r, laid, static_cast<const uint16_t*>(x), e, static_cast<int>(X), w.K, w.K / STEP, static_cast<int>(s.tiles_m), static_cast<int>(s.tiles_n)},
                                     stream);
    } else {
        r.ids = nullptr;
        const TileArgs a{r, w, static_cast<const uint16_t*>(x), e, static_cast<int>(X), w.K, w.K / STEP, static_cast<int>(s.tiles_m), static_cast<int>(s.tiles_n)};
        if (kind == X_PARTS) launch_tile<false, true>(fmt, s, a, stream);
        else launch_tile<false, false>(fmt, s, a, stream);
    }
    if (s.S > 1) {
        const size_t pieces = static_cast<size_t>(r.P) * ((e.No + 7) / 8);
        hipLaunchKernelGGL(k_join, dim3(static_cast<unsigned>((pieces + 255) / 256)), dim3(256), 0, stream, e, experts ? ids : nullptr, r.plan, r.P, r.E,
                           pieces);
    }
    return launch_status();
}

int64_t bwd_slab(int64_t M, int64_t No, bool bias)
{
    // Few rows are one slab, whose sums are dbias itself: no second launch, no workspace.
    // 64 x 512: a call 9.7 us for 13.9, captured in a graph 3.2 for 5.1; 128 x 28672, gated,
    // 9.6 for 13.7, and 6.0 for 9.3.  (256 x 2048 in a graph: 7.6 for 6.4.)
    if (bias && M <= BWD_FEW)
        return M;
    // about eight workgroups a CU, at least four rows each
    const int64_t across = (No + BWD_COLS - 1) / BWD_COLS, want = (2048 + across - 1) / across;
    const int64_t slab = (M + want - 1) / want;
    return (slab + 3) / 4 * 4;
}

template <bool SPLIT>
any4_status act_backward(const void* dy, int dy_f32, const void* z, int z_f32, uint16_t* dz, float* dbias, any4_activation act,
                         int gate, int64_t M, int64_t N, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!act_ok(act) || M < 0 || M > MAX_PAIRS || N < 0 || N > GIB2 / 4 || (M > 0 && N >= GIB2 / 2 / M) || (gate && N % 2))
        return ANY4_E_SHAPE;
    if (N == 0 || (M == 0 && !dbias))
        return ANY4_OK;
    const size_t need = dbias ? any4_act_backward_workspace_size(M, N, gate) : 0;
    if (M > 0 && (!dy || !z || !dz || (need && !workspace)))
        return ANY4_E_NULL;
    if (!is_aligned(dbias, 4) || (M > 0 && (!is_aligned(dy, dy_f32 ? 4 : 2) || !is_aligned(z, z_f32 ? 4 : 2) || !is_aligned(dz, 2) || !is_aligned(workspace, 16))))
        return ANY4_E_ALIGN;
    const int n = static_cast<int>(N), no = static_cast<int>(gate ? N / 2 : N);
    const int slab = M > 0 ? static_cast<int>(bwd_slab(M, no, dbias != nullptr)) : 1, slabs = static_cast<int>((M + slab - 1) / slab);
    if (need && workspace_bytes < need)
        return ANY4_E_WORKSPACE;
    (void)hipGetLastError();
    float* part = need ? static_cast<float*>(workspace) : dbias;
    if (M > 0) {
        const BwdArgs a{dy, z, dz, part, static_cast<int>(M), n, no, static_cast<int>(act), slab};
        // a grid has less than 2^32 threads, eight of these for each column
        const bool few = slabs == 1 && dbias && no <= GIB2 / 8;
        const int cols = few ? 64 : BWD_COLS;
        const dim3 grid(static_cast<unsigned>((no + cols - 1) / cols), static_cast<unsigned>(slabs));
        auto launch = [&](auto dy32, auto z32) {
#define BWD(GATE_, WHOLE_)                                                                                                     \
    do {                                                                                                                       \
        constexpr bool D = decltype(dy32)::value, Z = decltype(z32)::value;                                                    \
        if (few)                                                                                                               \
            hipLaunchKernelGGL((k_act_bwd<D, Z, GATE_, WHOLE_, SPLIT, 8, 8>), grid, dim3(8 * WAVE), 0, stream, a);                    \
        else                                                                                                                   \
            hipLaunchKernelGGL((k_act_bwd<D, Z, GATE_, WHOLE_, SPLIT, 4, WAVE>), grid, dim3(4 * WAVE), 0, stream, a);                 \
    } while (0)
            if (gate && no % 8 == 0) BWD(true, true);
            else if (gate) BWD(true, false);
            else if (no % 8 == 0) BWD(false, true);
            else BWD(false, false);
#undef BWD
        };
        if (dy_f32 && z_f32) launch(std::true_type{}, std::true_type{});
        else if (dy_f32) launch(std::true_type{}, std::false_type{});
        else if (z_f32) launch(std::false_type{}, std::true_type{});
        else launch(std::false_type{}, std::false_type{});
    }
    if (dbias && slabs != 1)         // none: zeros
        hipLaunchKernelGGL(k_bias_sum, dim3(static_cast<unsigned>((n + WAVE - 1) / WAVE)), dim3(256), 0, stream, part, dbias, n, slabs);
    return launch_status();
}

bool bias_ok(int64_t T, int64_t k, int64_t E, int64_t N)
{
    return T >= 0 && T <= MAX_PAIRS && k >= 1 && k <= MAX_PAIRS && T * k <= MAX_PAIRS && E >= 1 && E <= MAX_EXPERTS && N >= 0 &&
           N <= GIB2 / 8 && (T == 0 || N < GIB2 / 2 / (T * k));
}

// partial sums: of the chunks of experts with more than one
size_t bias_part_bytes(int64_t P, int64_t N) { return P > CHUNK ? up256(static_cast<size_t>(2 * (P / CHUNK)) * N * 4) : 0; }

size_t experts_dx_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g, bool parts)
{
    if (T <= 0 || k <= 0 || N <= 0 || T > MAX_PAIRS || k > MAX_PAIRS || !sizes_ok(T * k, T * k, E, (N + 7) / 8 * 8, K, g))
        return 0;
    const int64_t P = T * k;
    return part_bytes(shape_of(P, E, true, N, K, true, parts), P, K, N) + any4_lora_plan_bytes(P, E) +
           up256(static_cast<size_t>(P) * ((N + 7) / 8 * 8) * (parts ? 4 : 2));
}

// parts: dy in two parts
any4_status experts_dx(any4_format format, const uint16_t* dy, bool parts, const uint8_t* packed, const uint16_t* lut,
                       const uint16_t* alpha, const uint16_t* beta, const int32_t* ids, const void* plan, void* dx,
                       int dx_f32, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g, void* workspace,
                       size_t workspace_bytes, hipStream_t stream)
{
    const int fmt = static_cast<int>(format);
    if (!fmt_ok(fmt) || T < 0 || k < 1 || T > MAX_PAIRS || k > MAX_PAIRS || N < 1 ||
        !sizes_ok(T * k, T * k, E, (N + 7) / 8 * 8, K, g))
        return ANY4_E_SHAPE;
    if (T == 0)
        return ANY4_OK;
    if (!dy || !packed || (fmt != FMT_INT4 && !lut) || !alpha || !beta || !ids || !dx || !workspace)
        return ANY4_E_NULL;
    if (!is_aligned(dy, 2) || !is_aligned(packed, 16) || !is_aligned(lut, 2) || !is_aligned(alpha, 2) || !is_aligned(beta, 2) ||
        !is_aligned(ids, 4) || !is_aligned(plan, 16) || !is_aligned(dx, dx_f32 ? 4 : 2) || !is_aligned(workspace, 16))
        return ANY4_E_ALIGN;
    if (workspace_bytes < experts_dx_bytes(T, k, E, N, K, g, parts))
        return ANY4_E_WORKSPACE;
    (void)hipGetLastError();
    const int P = static_cast<int>(T * k), Np = static_cast<int>((N + 7) / 8 * 8);
    const Shape s = shape_of(P, E, true, N, K, true, parts);
    char* at = static_cast<char*>(workspace);
    if (!plan) {
        const any4_status st = any4_lora_plan(ids, at, any4_lora_plan_bytes(P, E), P, E, stream);
        if (st != ANY4_OK)
            return st;
        plan = at;
    }
    at += any4_lora_plan_bytes(P, E);
    if (N != Np || !is_aligned(dy, 16)) {
        uint16_t* copy = reinterpret_cast<uint16_t*>(at);
        const size_t pieces = static_cast<size_t>(P) * (Np / 8) * (parts ? 2 : 1);
        hipLaunchKernelGGL(k_pad_rows, dim3(static_cast<unsigned>((pieces + 255) / 256)), dim3(256), 0, stream, dy, copy,
                           static_cast<int>(N), Np, pieces);
        dy = copy;
    }
    at += up256(static_cast<size_t>(P) * Np * (parts ? 4 : 2));
    const Layer w{packed, lut, alpha, beta, static_cast<int>(N), static_cast<int>(K), static_cast<int>(g), layer_bytes(fmt, N, K)};
    const Epilogue q{nullptr, nullptr, nullptr, dx, s.S > 1 ? reinterpret_cast<float*>(at) : nullptr, static_cast<int>(K),
                     static_cast<int>(K), ACT_NONE, s.S, 0, dx_f32 != 0, 0};
    const Rows r{nullptr, static_cast<const int*>(plan), P, static_cast<int>(E), 1};
    const TileArgs a{r, w, dy, q, P, Np, (Np + STEP - 1) / STEP, static_cast<int>(s.tiles_m), static_cast<int>(s.tiles_n)};
    if (parts) launch_tile<true, true>(fmt, s, a, stream);
    else launch_tile<true, false>(fmt, s, a, stream);
    if (s.S > 1) {
        const size_t pieces = static_cast<size_t>(P) * (K / 8);
        hipLaunchKernelGGL(k_join, dim3(static_cast<unsigned>((pieces + 255) / 256)), dim3(256), 0, stream, q, ids, r.plan, P, static_cast<int>(E),
                           pieces);
    }
    return launch_status();
}

}  // namespace

extern "C" {

any4_status any4_ffn_form(int64_t P, int64_t E, int64_t N, int64_t K, int back, int parts, int32_t* form)
{
    if (!sizes_ok(P, P, E > 0 ? E : 1, N, K, K) || P == 0 || N == 0 || E < 0 || (E == 0 && (back || parts)))
        return ANY4_E_SHAPE;
    if (!form)
        return ANY4_E_NULL;
    const Shape s = shape_of(P, E > 0 ? E : 1, E > 0, back ? N : K, back ? K : N, back != 0, parts != 0);
    form[0] = 32 * s.rm;
    form[1] = 2 * s.wn;
    form[2] = s.S;
    form[3] = s.rows;
    return ANY4_OK;
}

size_t any4_gemm_act_workspace_size(int64_t M, int64_t N, int64_t K, int64_t g)
{
    if (M <= 0 || N <= 0 || !sizes_ok(M, M, 1, N, K, g))
        return 0;
    return part_bytes(shape_of(M, 1, false, K, N, false), M, N, K);
}

any4_status any4_gemm_act(any4_format format, const uint16_t* x, const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha,
                          const uint16_t* beta, const uint16_t* bias, const uint16_t* residual, void* z, int z_f32, void* out, int out_f32,
                          any4_activation act, int gate, int64_t M, int64_t N, int64_t K, int64_t g, void* workspace,
                          size_t workspace_bytes, hipStream_t stream)
{
    const int fmt = static_cast<int>(format);
    if (!fmt_ok(fmt) || !act_ok(act) || !sizes_ok(M, M, 1, N, K, g) || (gate && N % 2))
        return ANY4_E_SHAPE;
    if (M == 0 || N == 0)
        return ANY4_OK;
    if (!x || !packed || (fmt != FMT_INT4 && !lut) || !alpha || !beta || !out)
        return ANY4_E_NULL;
    if (!is_aligned(x, 16) || !is_aligned(packed, 16) || !is_aligned(lut, 2) || !is_aligned(alpha, 2) || !is_aligned(beta, 2) ||
        !is_aligned(bias, 2) || !is_aligned(residual, 2) || !is_aligned(z, z_f32 ? 4 : 2) || !is_aligned(out, out_f32 ? 4 : 2) || !is_aligned(workspace, 16))
        return ANY4_E_ALIGN;
    (void)hipGetLastError();
    const Layer w{packed, lut, alpha, beta, static_cast<int>(N), static_cast<int>(K), static_cast<int>(g), layer_bytes(fmt, N, K)};
    const Epilogue q{bias, residual, z, out, nullptr, static_cast<int>(N), static_cast<int>(gate ? N / 2 : N), static_cast<int>(act), 1,
                     z_f32 != 0, out_f32 != 0, 0};
    return product(fmt, Rows{nullptr, nullptr, static_cast<int>(M), 1, 1}, M, x, X_BF16, w, q, nullptr, workspace, workspace_bytes, false, stream);
}

size_t any4_act_backward_workspace_size(int64_t M, int64_t N, int gate)
{
    if (M <= 0 || N <= 0 || M > MAX_PAIRS || N > GIB2 / 4 || N >= GIB2 / 2 / M || (gate && N % 2))
        return 0;
    const int64_t slab = bwd_slab(M, gate ? N / 2 : N, true), slabs = (M + slab - 1) / slab;
    return slabs == 1 ? 0 : up256(static_cast<size_t>(slabs) * N * 4);
}

any4_status any4_act_backward(const void* dy, int dy_f32, const void* z, int z_f32, uint16_t* dz, float* dbias, any4_activation act,
                              int gate, int64_t M, int64_t N, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return act_backward<false>(dy, dy_f32, z, z_f32, dz, dbias, act, gate, M, N, workspace, workspace_bytes, stream);
}

any4_status any4_act_backward_parts(const void* dy, int dy_f32, const void* z, int z_f32, uint16_t* dz, float* dbias, any4_activation act,
                                    int gate, int64_t M, int64_t N, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return act_backward<true>(dy, dy_f32, z, z_f32, dz, dbias, act, gate, M, N, workspace, workspace_bytes, stream);
}

size_t any4_experts_bias_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N)
{
    if (T <= 0 || N <= 0 || !bias_ok(T, k, E, N))
        return 0;
    return bias_part_bytes(T * k, N) + any4_lora_plan_bytes(T * k, E);
}

any4_status any4_experts_bias_backward(const void* dy, int dy_f32, const void* z, int z_f32, const int32_t* ids, const void* plan,
                                       float* dbias, any4_activation act, int gate, int64_t T, int64_t k, int64_t E, int64_t N,
                                       void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!act_ok(act) || !bias_ok(T, k, E, N) || (gate && N % 2))
        return ANY4_E_SHAPE;
    if (N == 0)
        return ANY4_OK;
    const int64_t P = T * k;
    const size_t parts = bias_part_bytes(P, N), need = P == 0 ? 0 : parts + (plan ? 0 : any4_lora_plan_bytes(P, E));
    if (!dbias || (P > 0 && (!dy || !z || !ids || (need && !workspace))))
        return ANY4_E_NULL;
    if (!is_aligned(dbias, 4) || (P > 0 && (!is_aligned(dy, dy_f32 ? 4 : 2) || !is_aligned(z, z_f32 ? 4 : 2) || !is_aligned(ids, 4) ||
                                            !is_aligned(plan, 16) || !is_aligned(workspace, 16))))
        return ANY4_E_ALIGN;
    if (need && workspace_bytes < need)
        return ANY4_E_WORKSPACE;
    (void)hipGetLastError();
    char* at = static_cast<char*>(workspace);
    if (P > 0 && !plan) {
        const any4_status st = any4_lora_plan(ids, at + parts, any4_lora_plan_bytes(P, E), P, E, stream);
        if (st != ANY4_OK)
            return st;
        plan = at + parts;
    }
    const ExpertBiasArgs a{dy, z, P > 0 ? static_cast<const int*>(plan) : nullptr, dbias, reinterpret_cast<float*>(at), static_cast<int>(P),
                           static_cast<int>(E), static_cast<int>(N), static_cast<int>(gate ? N / 2 : N), static_cast<int>(act)};
    if (P > 0) {
        const dim3 grid(static_cast<unsigned>((a.No + 63) / 64), static_cast<unsigned>(PlanLayout(P, E).CB));
        auto launch = [&](auto dy32, auto z32) {
            constexpr bool D = decltype(dy32)::value, Z = decltype(z32)::value;
#define EXPERT_BIAS(GATE_, WHOLE_) hipLaunchKernelGGL((k_expert_bias<D, Z, GATE_, WHOLE_>), grid, dim3(8 * WAVE), 0, stream, a)
            if (gate && a.No % 8 == 0) EXPERT_BIAS(true, true);
            else if (gate) EXPERT_BIAS(true, false);
            else if (a.No % 8 == 0) EXPERT_BIAS(false, true);
            else EXPERT_BIAS(false, false);
#undef EXPERT_BIAS
        };
        if (dy_f32 && z_f32) launch(std::true_type{}, std::true_type{});
        else if (dy_f32) launch(std::true_type{}, std::false_type{});
        else if (z_f32) launch(std::false_type{}, std::true_type{});
        else launch(std::false_type{}, std::false_type{});
    }
    hipLaunchKernelGGL(k_expert_bias_sum, dim3(static_cast<unsigned>((N + 255) / 256), static_cast<unsigned>(E)), dim3(256), 0, stream, a);
    return launch_status();
}

size_t any4_experts_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g)
{
    if (T <= 0 || k <= 0 || N <= 0 || T > MAX_PAIRS || k > MAX_PAIRS || !sizes_ok(T * k, T, E, N, K, g))
        return 0;
    const int64_t P = T * k;
    return part_bytes(shape_of(P, E, true, K, N, false), P, N, K) + (P <= FEW_P ? 0 : any4_lora_plan_bytes(P, E));
}

size_t any4_experts_parts_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g)
{
    if (T <= 0 || k <= 0 || N <= 0 || T > MAX_PAIRS || k > MAX_PAIRS || !sizes_ok(T * k, T * k, E, N, K, g))
        return 0;
    const int64_t P = T * k;
    return part_bytes(shape_of(P, E, true, K, N, false, true), P, N, K) + (P <= FEW_P ? 0 : any4_lora_plan_bytes(P, E));
}

any4_status any4_experts_gemm(any4_format format, const void* x, int x_f32, int per_pair, const uint8_t* packed, const uint16_t* lut,
                              const uint16_t* alpha, const uint16_t* beta, const uint16_t* bias, const int32_t* ids, const void* plan,
                              void* z, int z_f32, void* out, int out_f32, any4_activation act, int gate, int64_t T, int64_t k, int64_t E, int64_t N,
                              int64_t K, int64_t g, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    const int fmt = static_cast<int>(format);
    if (!fmt_ok(fmt) || !act_ok(act) || T < 0 || k < 1 || T > MAX_PAIRS || k > MAX_PAIRS ||
        !sizes_ok(T * k, per_pair ? T * k : T, E, N, K, g) || (gate && N % 2))
        return ANY4_E_SHAPE;
    const int kind = !x_f32 ? X_BF16 : x_f32 == ANY4_PARTS ? X_PARTS : X_F32;
    if ((kind == X_F32 && T * k > FEW_P) || (kind == X_PARTS && !per_pair))
        return ANY4_E_SHAPE;
    if (T == 0 || N == 0)
        return ANY4_OK;
    if (!x || !packed || (fmt != FMT_INT4 && !lut) || !alpha || !beta || !ids || !out)
        return ANY4_E_NULL;
    if (!is_aligned(x, 16) || !is_aligned(packed, 16) || !is_aligned(lut, 2) || !is_aligned(alpha, 2) || !is_aligned(beta, 2) ||
        !is_aligned(bias, 2) || !is_aligned(ids, 4) || !is_aligned(plan, 16) || !is_aligned(z, z_f32 ? 4 : 2) ||
        !is_aligned(out, out_f32 && out_f32 != ANY4_PARTS ? 4 : 2) || !is_aligned(workspace, 16))
        return ANY4_E_ALIGN;
    (void)hipGetLastError();
    const Layer w{packed, lut, alpha, beta, static_cast<int>(N), static_cast<int>(K), static_cast<int>(g), layer_bytes(fmt, N, K)};
    const int64_t No = gate ? N / 2 : N;
    const Epilogue q{bias, nullptr, z, out, nullptr, static_cast<int>(N), static_cast<int>(No), static_cast<int>(act), 1,
                     z_f32 != 0, out_f32 == ANY4_PARTS ? ANY4_PARTS : out_f32 != 0, static_cast<size_t>(T * k * No)};
    const Rows r{nullptr, static_cast<const int*>(plan), static_cast<int>(T * k), static_cast<int>(E), per_pair ? 1 : static_cast<int>(k)};
    return product(fmt, r, per_pair ? T * k : T, x, kind, w, q, ids, workspace, workspace_bytes, true, stream);
}

size_t any4_experts_dx_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g)
{
    return experts_dx_bytes(T, k, E, N, K, g, false);
}

size_t any4_experts_dx_parts_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g)
{
    return experts_dx_bytes(T, k, E, N, K, g, true);
}

any4_status any4_experts_gemm_dx(any4_format format, const uint16_t* dy, const uint8_t* packed, const uint16_t* lut,
                                 const uint16_t* alpha, const uint16_t* beta, const int32_t* ids, const void* plan, void* dx,
                                 int dx_f32, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream)
{
    return experts_dx(format, dy, false, packed, lut, alpha, beta, ids, plan, dx, dx_f32, T, k, E, N, K, g, workspace, workspace_bytes, stream);
}

any4_status any4_experts_gemm_dx_parts(any4_format format, const uint16_t* dy, const uint8_t* packed, const uint16_t* lut,
                                       const uint16_t* alpha, const uint16_t* beta, const int32_t* ids, const void* plan, void* dx,
                                       int dx_f32, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream)
{
    return experts_dx(format, dy, true, packed, lut, alpha, beta, ids, plan, dx, dx_f32, T, k, E, N, K, g, workspace, workspace_bytes, stream);
}

}  // extern "C"
