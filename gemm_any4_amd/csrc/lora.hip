// Low-rank adapters beside a frozen any4 layer, served for many requests at
// once and trained, and activations kept in 8 bits.  The C ABI is declared in
// include/any4.h.
//
// The mathematics.  Row m of the batch uses adapter a = ids[m]:
//     h[m]   = A_a x[m]                       y'[m]  = y[m]  + s_a sum_j h[m][j] B_a[j]
//     dh[m]  = s_a B_a dy[m]                  dx'[m] = dx[m] + sum_j dh[m][j] A_a[j]
//     dA_a   = sum_m dh[m]^T x[m]             dB_a   = s_a sum_m h[m]^T dy[m]
// A is [L][r][K] and B [L][r][N] (rank-major), so a pass is made of three
// products, each used twice:
//     shrink   part[m][j] = sum_d in[m][d] W_a[j][d]       (x with A, dy with B)
//     expand   out[m][d]  = base[m][d] + sum_j c[m][j] W_a[j][d]
//     wgrad    G_a[j][d]  = sum_m c[m][j] in[m][d]
// The fp32 factors (h, dh) enter the matrix cores as three bf16 parts
// (split3), which together are the fp32 value: with r <= 128 the products are
// never what bounds a kernel, so nothing is rounded that need not be.
//
// Rows of one adapter are worked on in tiles.  For few rows a wave finds
// its tile from the ids alone (ballots); beyond that the plan (rows sorted by
// adapter, tables of tiles and chunks) is made by k_plan* once, in the
// workspace or, for callers that keep it, in a buffer of theirs.
#include <type_traits>

#include "frag.h"

namespace {

constexpr int SMALL_M = 64;          // up to here tiles come from ballots over the ids,
constexpr int SMALL_M_FORWARD = 256; // and in the forward pass up to here with few adapters
constexpr int SMALL_L_FORWARD = 8;
constexpr int SMALL_T = 16;          // rows of a tile there
constexpr int TILE_T = 32;           // rows of a tile of the plan
constexpr int CHUNK = 512;           // rows of a chunk of the weight gradient
constexpr int MAX_RANK = 128;
constexpr int MAX_ADAPTERS = 4096;
constexpr int64_t MAX_M = static_cast<int64_t>(1) << 20;   // tiles fit a grid's second dimension
constexpr int64_t ACT8_MAX_M = 65535 * 64;

// ---------------------------------------------------------------------------
// the plan: rows sorted by adapter (stable), tiles and chunks of equal adapter
// ---------------------------------------------------------------------------
// int32 words: [0] tiles, [1] chunks, [2] M, [3] L, then
//   first [L+1]  first tile of each adapter (entry L: of the rows without one)
//   count [L+1]  its rows
//   slot  [L+1]  its first partial-sum slot (adapters of one chunk or none have
//                no slot)
//   chunk [CB][4]  adapter, first place, rows, slot (-1: the only chunk)
//   tile  [TB][2]  adapter (-1: none), rows
//   rows  [TB][TILE_T]  the rows of each tile; places behind the last repeat it
// A place is TILE_T * tile + position: the rows of one adapter stand together, and
// a kernel that knows its tile's number knows where they are.
struct PlanLayout {
    int64_t first, count, slot, chunk, tile, rows, words;
    int64_t TB, CB;

    __host__ __device__ PlanLayout(int64_t M, int64_t L)
    {
        const int64_t segs = M < L + 1 ? M : L + 1;
        TB = M / TILE_T + segs;
        CB = M / CHUNK + segs;
        first = 4;
        count = first + L + 1;
        slot = count + L + 1;
        chunk = (slot + L + 1 + 3) / 4 * 4;
        tile = chunk + 4 * CB;
        rows = tile + (2 * TB + 3) / 4 * 4;
        words = rows + TILE_T * TB;
    }
};

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_WAVES = PLAN_THREADS / WAVE;
constexpr int PLAN_ONE_M = 16384;    // up to here (and PLAN_ONE_L) one workgroup does it all
constexpr int PLAN_ONE_L = 512;
constexpr int PLAN_PARTS = 256;      // beyond: waves of their own, with counts in memory

__device__ __forceinline__ int adapter_of(int id, int L) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(L) ? id : L; }

// This lane's place among the rows of its adapter that the wave has counted so
// far in n[]; the wave's rows in order.  Lanes of equal adapter find each other
// by ballots, and the first of them adds them all.
__device__ __forceinline__ int count_rows(int a, bool live, int* n)
{
    const int lane = threadIdx.x & 63;
    uint64_t left = __ballot(live), mine = 0;
    while (left) {
        const int v = __builtin_amdgcn_readlane(a, __builtin_ctzll(left));
        const uint64_t m = __ballot(live && a == v);
        if (a == v)
            mine = m;
        left &= ~m;
    }
    const int lead = mine ? __builtin_ctzll(mine) : lane;
    int at = 0;
    if (live && lane == lead)
        at = atomicAdd(&n[a], __builtin_popcountll(mine));
    return __shfl(at, lead) + __builtin_popcountll(mine & ((1ull << lane) - 1));
}

// Row m is number `at` of the n rows of an adapter whose first place is given;
// the last one also fills the tile's empty places.
__device__ __forceinline__ void place_row(int m, int at, int n, int64_t first, int* rows)
{
    rows[first + at] = m;
    if (at == n - 1)
        for (int i = n; i % TILE_T; ++i)
            rows[first + i] = m;
}

struct Three {
    int v[3];
};

// Exclusive sums over the block's threads (one_wave: only the first 64 threads'
// values count, and only they ask).
__device__ __forceinline__ Three block_scan(Three x, int (*wave_sum)[3], bool one_wave)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    Three s = x;
    if (!one_wave || w == 0)
        for (int d = 1; d < WAVE; d <<= 1) {
            int o[3];
#pragma unroll
            for (int q = 0; q < 3; ++q)
                o[q] = __shfl_up(s.v[q], d);
#pragma unroll
            for (int q = 0; q < 3; ++q)
                s.v[q] += lane >= d ? o[q] : 0;
        }
    if (!one_wave) {
#pragma unroll
        for (int q = 0; q < 3; ++q)
            if (lane == 63)
                wave_sum[w][q] = s.v[q];
        __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        int before = 0;
        if (!one_wave)
            for (int i = 0; i < PLAN_WAVES; ++i)
                before += i < w ? wave_sum[i][q] : 0;
        s.v[q] += before - x.v[q];
    }
    return s;
}

__device__ __forceinline__ int tiles_of(int rows) { return (rows + TILE_T - 1) / TILE_T; }
__device__ __forceinline__ int chunks_of(int rows) { return (rows + CHUNK - 1) / CHUNK; }

// From cnt[part][L+1] (rows of each adapter in each of the batch's 16 n parts): the
// plan's tables, s_rows and s_tile (rows and first tile of each adapter), and
// cnt turned into the number of the adapter's rows in earlier parts.
__device__ __forceinline__ void plan_tables(int* cnt, int parts, int M, int L, int* plan, int* s_rows,
                                            int* s_tile, int* s_chunk, int* s_slot, int (*wave_sum)[3])
{
    const PlanLayout p(M, L);
    const int tid = threadIdx.x, per = (L + 1 + PLAN_THREADS - 1) / PLAN_THREADS;
    for (int a = tid; a <= L; a += PLAN_THREADS) {
        int n = 0;
        for (int q0 = 0; q0 < parts; q0 += 16) {     // sixteen reads, then the writes
            int c[16];
#pragma unroll
            for (int q = 0; q < 16; ++q)
                c[q] = cnt[static_cast<size_t>(q0 + q) * (L + 1) + a];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                cnt[static_cast<size_t>(q0 + q) * (L + 1) + a] = n;
                n += c[q];
            }
        }
        s_rows[a] = n;
    }
    __syncthreads();
    Three sum = {{0, 0, 0}};
    for (int e = 0; e < per; ++e) {
        const int a = tid * per + e;
        if (a > L)
            break;
        const int n = s_rows[a], ch = a < L ? chunks_of(n) : 0;
        sum.v[0] += tiles_of(n);
        sum.v[1] += ch;
        sum.v[2] += ch > 1 ? ch : 0;
    }
    Three at = block_scan(sum, wave_sum, L < WAVE);
    for (int e = 0; e < per; ++e) {
        const int a = tid * per + e;
        if (a > L)
            break;
        const int n = s_rows[a], ch = a < L ? chunks_of(n) : 0;
        s_tile[a] = at.v[0];
        s_chunk[a] = at.v[1];
        s_slot[a] = at.v[2];
        plan[p.first + a] = at.v[0];
        plan[p.count + a] = n;
        plan[p.slot + a] = at.v[2];
        at.v[0] += tiles_of(n);
        at.v[1] += ch;
        at.v[2] += ch > 1 ? ch : 0;
        if (a == L) {
            s_tile[L + 1] = at.v[0];
            s_chunk[L + 1] = at.v[1];
            plan[0] = at.v[0];
            plan[1] = at.v[1];
            plan[2] = M;
            plan[3] = L;
        }
    }
    __syncthreads();
    for (int kind = 0; kind < 2; ++kind) {
        const int* start = kind ? s_chunk : s_tile;
        const int total = start[L + 1], size = kind ? CHUNK : TILE_T;
        for (int t = tid; t < total; t += PLAN_THREADS) {
            int lo = 0, hi = L + 1;      // the last adapter that starts at or before t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            const int before = (t - start[lo]) * size, left = s_rows[lo] - before, rows = left < size ? left : size;
            if (kind == 0) {
                int* o = plan + p.tile + 2 * static_cast<int64_t>(t);
                o[0] = lo < L ? lo : -1;
                o[1] = rows;
            } else {
                int* o = plan + p.chunk + 4 * static_cast<int64_t>(t);
                o[0] = lo;
                o[1] = s_tile[lo] * TILE_T + before;
                o[2] = rows;
                o[3] = start[lo + 1] - start[lo] > 1 ? s_slot[lo] + t - start[lo] : -1;
            }
        }
    }
}

// Up to STEPS x 64 rows a wave, their ids in registers from the first load on.
// A chain of waits, not of work: 4.0 us for 1031 rows, 4.9 us for 4096, 11.7 us for
// 16384 (1.5 us more with the sums over all waves where the first holds all the
// adapters); half a microsecond more between a batch's other kernels.
template <int STEPS>
__global__ __launch_bounds__(PLAN_THREADS) void k_plan(const int* __restrict__ ids, int* plan, int M, int L)
{
    __shared__ int cnt[PLAN_WAVES * (PLAN_ONE_L + 1)];
    __shared__ int s_rows[PLAN_ONE_L + 2], s_tile[PLAN_ONE_L + 2], s_chunk[PLAN_ONE_L + 2], s_slot[PLAN_ONE_L + 2];
    __shared__ int wave_sum[PLAN_WAVES][3];
    const int w = threadIdx.x >> 6, per = (M + PLAN_THREADS - 1) / PLAN_THREADS;      // at most STEPS
    const int m0 = w * (per * WAVE) + (threadIdx.x & 63);
    int a[STEPS], at[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        a[i] = i < per && m0 + i * WAVE < M ? ids[m0 + i * WAVE] : -1;
    for (int i = threadIdx.x; i < PLAN_WAVES * (L + 1); i += PLAN_THREADS)
        cnt[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (i >= per)
            break;
        a[i] = adapter_of(a[i], L);
        at[i] = count_rows(a[i], m0 + i * WAVE < M, cnt + w * (L + 1));
    }
    __syncthreads();
    plan_tables(cnt, PLAN_WAVES, M, L, plan, s_rows, s_tile, s_chunk, s_slot, wave_sum);
    int* rows = plan + PlanLayout(M, L).rows;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (i < per && m0 + i * WAVE < M)
            place_row(m0 + i * WAVE, cnt[w * (L + 1) + a[i]] + at[i], s_rows[a[i]],
                      static_cast<int64_t>(s_tile[a[i]]) * TILE_T, rows);
}

// Larger batches or many adapters: the same in three launches, one wave for
// each part of the batch, the counts in memory (PLAN_PARTS x (L + 1) words).
__global__ __launch_bounds__(WAVE) void k_plan_count(const int* __restrict__ ids, int* cnt, int M, int L, int per)
{
    int* mine = cnt + static_cast<size_t>(blockIdx.x) * (L + 1);
    for (int i = threadIdx.x; i <= L; i += WAVE)
        mine[i] = 0;
    __threadfence();     // the zeros are in place before the atomics below
    __syncthreads();
    const int m0 = blockIdx.x * per, m1 = m0 + per < M ? m0 + per : M;     // parts * per < 2^21
    for (int b = m0; b < m1; b += WAVE) {
        const int m = b + threadIdx.x;
        count_rows(m < m1 ? adapter_of(ids[m], L) : -1, m < m1, mine);
    }
}

__global__ __launch_bounds__(PLAN_THREADS) void k_plan_tables(int* cnt, int* plan, int M, int L, int parts)
{
    __shared__ int s_rows[MAX_ADAPTERS + 2], s_tile[MAX_ADAPTERS + 2], s_chunk[MAX_ADAPTERS + 2],
        s_slot[MAX_ADAPTERS + 2];
    __shared__ int wave_sum[PLAN_WAVES][3];
    plan_tables(cnt, parts, M, L, plan, s_rows, s_tile, s_chunk, s_slot, wave_sum);
}

__global__ __launch_bounds__(WAVE) void k_plan_place(const int* __restrict__ ids, int* cnt, int* plan, int M, int L, int per)
{
    const PlanLayout p(M, L);
    const int m0 = blockIdx.x * per, m1 = m0 + per < M ? m0 + per : M;
    for (int b = m0; b < m1; b += WAVE) {
        const int m = b + threadIdx.x;
        const bool live = m < m1;
        const int a = live ? adapter_of(ids[m], L) : -1;
        const int at = count_rows(a, live, cnt + static_cast<size_t>(blockIdx.x) * (L + 1));
        if (live)
            place_row(m, at, plan[p.count + a], static_cast<int64_t>(plan[p.first + a]) * TILE_T, plan + p.rows);
    }
}

bool plan_in_one(int64_t M, int64_t L) { return M <= PLAN_ONE_M && L <= PLAN_ONE_L; }

// words of the plan, and of the counts behind it
int64_t plan_words(int64_t M, int64_t L)
{
    return PlanLayout(M, L).words + (plan_in_one(M, L) ? 0 : PLAN_PARTS * (L + 1));
}

void launch_plan(const int32_t* ids, int32_t* plan, int64_t M, int64_t L, hipStream_t stream)
{
    const int m = static_cast<int>(M), l = static_cast<int>(L);
    if (plan_in_one(M, L)) {
        if (M <= 2 * PLAN_THREADS)
            hipLaunchKernelGGL(k_plan<2>, dim3(1), dim3(PLAN_THREADS), 0, stream, ids, plan, m, l);
        else if (M <= 8 * PLAN_THREADS)
            hipLaunchKernelGGL(k_plan<8>, dim3(1), dim3(PLAN_THREADS), 0, stream, ids, plan, m, l);
        else
            hipLaunchKernelGGL(k_plan<PLAN_ONE_M / PLAN_THREADS>, dim3(1), dim3(PLAN_THREADS), 0, stream, ids, plan, m, l);
        return;
    }
    int* cnt = plan + PlanLayout(M, L).words;
    const int steps = (m + WAVE - 1) / WAVE, parts = steps < PLAN_PARTS ? (steps + 15) / 16 * 16 : PLAN_PARTS;
    const int per = (steps + parts - 1) / parts * WAVE;
    hipLaunchKernelGGL(k_plan_count, dim3(parts), dim3(WAVE), 0, stream, ids, cnt, m, l, per);
    hipLaunchKernelGGL(k_plan_tables, dim3(1), dim3(PLAN_THREADS), 0, stream, cnt, plan, m, l, parts);
    hipLaunchKernelGGL(k_plan_place, dim3(parts), dim3(WAVE), 0, stream, ids, cnt, plan, m, l, per);
}

// ---------------------------------------------------------------------------
// the rows of a tile
// ---------------------------------------------------------------------------
struct Batch {
    const int* ids;     // [M]
    const int* plan;    // null: tiles of SMALL_T rows by ballots
    int M, L;
    bool given;         // the plan is the caller's, not of this call
};

// Whether the plan is one of this M and L.  A given one may be of others, and
// its buffer smaller: nothing else of it is read before its first words agree.
// That wait costs calls with a kept plan up to 1% (4096 rows, 4096 to 14336, rank
// 16, 49.2 against 49.7 us).  A plan of this call fits, and nobody waits for them.
__device__ __forceinline__ bool fits(const Batch& b)
{
    if (!b.given)
        return true;
    const int m = b.plan[2], l = b.plan[3];       // both loads before the comparisons: one wait
    return (m == b.M) & (l == b.L);
}

struct Tile {
    int a;              // adapter, -1: rows without one, -2: no such tile
    int count;
    const int* rows;    // its T rows; places behind the last repeat it
};

// Every wave finds tile t of SMALL_T rows for itself, the batch's ids in WORDS
// of 64: adapters in the order of their first rows, by ballots.
template <int WORDS>
__device__ __forceinline__ Tile search_tile(const Batch& b, int t, int* own)
{
    constexpr int T = SMALL_T;
    const int lane = threadIdx.x & 63;
    int id[WORDS];
    uint64_t left[WORDS], any = 0;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        const int m = lane + i * WAVE;
        id[i] = m < b.M ? adapter_of(b.ids[m], b.L) : -1;
        left[i] = __ballot(m < b.M);
        any |= left[i];
    }
    while (any) {
        int a = 0;          // the adapter of the first row left
#pragma unroll
        for (int i = WORDS - 1; i >= 0; --i)
            if (WORDS == 1 || left[i])
                a = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(left[i]));
        uint64_t mask[WORDS];
        int n = 0;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            mask[i] = __ballot(id[i] == a);
            n += __builtin_popcountll(mask[i]);
        }
        const int tiles = (n + T - 1) / T;
        if (t < tiles) {
            const int count = n - t * T < T ? n - t * T : T;
            int before = -t * T;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const int at = before + __builtin_popcountll(mask[i] & ((1ull << lane) - 1));
                if ((mask[i] >> lane & 1) && at >= 0 && at < T) {
                    own[at] = lane + i * WAVE;
                    if (at == count - 1)
                        for (int e = count; e < T; ++e)
                            own[e] = lane + i * WAVE;
                }
                before += __builtin_popcountll(mask[i]);
            }
            wave_sync();
            return {a < b.L ? a : -1, count, own};
        }
        t -= tiles;
        any = 0;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            left[i] &= ~mask[i];
            any |= left[i];
        }
    }
    return {-2, 0, own};
}

// Tile t.  own: SMALL_T ints of LDS of this wave (the small form keeps the rows
// there).
template <int T>
__device__ __forceinline__ Tile find_tile(const Batch& b, int t, int* own)
{
    if constexpr (T == SMALL_T) {
        return b.M <= WAVE ? search_tile<1>(b, t, own) : search_tile<SMALL_M_FORWARD / WAVE>(b, t, own);
    } else {
        if (!fits(b))
            return {-2, 0, nullptr};
        const PlanLayout p(b.M, b.L);
        const int* e = b.plan + p.tile + 2 * static_cast<int64_t>(t);     // in the plan's bounds for every t of the grid
        const int a = e[0], count = e[1];
        if (t >= b.plan[0])
            return {-2, 0, nullptr};
        return {a, count, b.plan + p.rows + TILE_T * static_cast<int64_t>(t)};
    }
}

// Whether the forward pass finds its tiles by ballots, without a plan.  The
// search takes 0.2 us for each adapter that a wave passes over, a plan 6 us and a
// launch: 250 rows of 4 adapters, 4096 x 14336, rank 64, 15 us against 22; 256 rows of
// 64 adapters, 34 us against 20.  (The backward pass reads the factors of its weight
// gradients faster by place: beyond SMALL_M rows it always has a plan.)
bool by_ballots(int64_t M, int64_t L) { return M <= SMALL_M || (M <= SMALL_M_FORWARD && L <= SMALL_L_FORWARD); }

int64_t tile_bound(int64_t M, int64_t L, bool ballots)
{
    if (ballots)       // each adapter's rows in tiles of SMALL_T
        return M / SMALL_T + (M < L + 1 ? M : L + 1);
    return PlanLayout(M, L).TB;
}

// ---------------------------------------------------------------------------
// activations in 8 bits: s = fp32(amax / 127) over GROUP8 channels,
// q = rint(fp32(x * fp32(127 / amax)))
// ---------------------------------------------------------------------------
constexpr int GROUP8 = 128;

__device__ __forceinline__ uint32_t abs_max(u32x4_t v)
{
    // magnitudes of bf16 values order as their bits, a NaN above an infinity
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = v[i] & 0x7fffu, hi = v[i] >> 16 & 0x7fffu;
        m = max(m, max(lo, hi));
    }
    return m;
}

struct Scale8 {
    float unit, inv;
};

__device__ __forceinline__ Scale8 scale8(uint32_t top)
{
    const float amax = bf16_to_f32(top);
    // below 2^-100 the inverse would overflow: such a group is kept as zeros
    const bool dead = amax < 0x1p-100f;
    return {dead ? 0.0f : amax / 127.0f, dead ? 0.0f : 127.0f / amax};
}

__device__ __forceinline__ u32x2_t quantise8(u32x4_t v, float inv)
{
    // the product is rounded to fp32 first (no fma), then adding 1.5 * 2^23 rounds
    // it to a whole number, ties to even, and leaves that in the low byte (0 for
    // a NaN: its group's scale is NaN or inf)
#pragma clang fp contract(off)
    uint32_t k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16) * inv;
        k[i] = __float_as_uint(f + 0x1.8p23f);
    }
    u32x2_t q;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        q[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(k[4 * i + 3], k[4 * i + 2], 0x0c0c0400u),
                                     __builtin_amdgcn_perm(k[4 * i + 1], k[4 * i], 0x0c0c0400u), 0x05040100u);
    return q;
}

// The 128 channels of a row that four lanes (g = 0 .. 3, 16 apart) hold, 8 at
// 32 i + 8 g each: q and scale are where the first of them go.  The lanes trade
// their 8-byte pieces (a 4 x 4 transposition in two rounds of swaps between
// rows of 16 lanes), so that each stores 32 bytes in one place.
__device__ __forceinline__ void store_row8(const u32x4_t (&v)[4], uint8_t* q, float* scale, int g, bool live)
{
    uint32_t top = max(max(abs_max(v[0]), abs_max(v[1])), max(abs_max(v[2]), abs_max(v[3])));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
    const Scale8 e = scale8(top);
    u32x2_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = quantise8(v[i], e.inv);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto s = __builtin_amdgcn_permlane32_swap(o[i][b], o[i + 2][b], false, false);
            o[i][b] = s[0];
            o[i + 2][b] = s[1];
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const auto s = __builtin_amdgcn_permlane16_swap(o[i][b], o[i + 1][b], false, false);
            o[i][b] = s[0];
            o[i + 1][b] = s[1];
        }
    }
    if (!live)
        return;
    u32x4_t* to = reinterpret_cast<u32x4_t*>(q + 32 * g);
    to[0] = u32x4_t{o[0][0], o[0][1], o[1][0], o[1][1]};
    to[1] = u32x4_t{o[2][0], o[2][1], o[3][0], o[3][1]};
    if (g == 0)
        *scale = e.unit;
}

// Signed byte i of v as fp32.
__device__ __forceinline__ float byte_to_f32(uint32_t v, int i)
{
    return static_cast<float>(static_cast<int>(v << (24 - 8 * i)) >> 24);
}

constexpr int ACT8_THREADS = 256;

// One 16-lane group per GROUP8 channels, 16 bytes of x a lane; one pass, bound by
// its bytes: 8192 x 14336 71 us to keep and 58 us to read back (5.0 and 6.1 TB/s).
__global__ __launch_bounds__(ACT8_THREADS) void k_act8_save(const uint16_t* __restrict__ x, uint8_t* __restrict__ q,
                                                            float* __restrict__ s, uint32_t slots)
{
    const uint32_t i = blockIdx.x * ACT8_THREADS + threadIdx.x;
    if (i >= slots)      // slots is a multiple of 16: a group is live as a whole
        return;
    const u32x4_t v = reinterpret_cast<const u32x4_t*>(x)[i];
    uint32_t top = abs_max(v);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1)
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
    const Scale8 g = scale8(top);
    reinterpret_cast<u32x2_t*>(q)[i] = quantise8(v, g.inv);
    if ((i & 15) == 0)
        s[i >> 4] = g.unit;
}

__global__ __launch_bounds__(ACT8_THREADS) void k_act8_load(const uint8_t* __restrict__ q, const float* __restrict__ s,
                                                            uint16_t* __restrict__ x, uint32_t slots)
{
    const uint32_t i = blockIdx.x * ACT8_THREADS + threadIdx.x;
    if (i >= slots)
        return;
    const u32x2_t v = reinterpret_cast<const u32x2_t*>(q)[i];
    const float unit = s[i >> 4];
    u32x4_t o;
#pragma unroll
    for (int p = 0; p < 4; ++p)
        o[p] = f32_to_bf16(byte_to_f32(v[p / 2], (2 * p) & 3) * unit) |
               f32_to_bf16(byte_to_f32(v[p / 2], (2 * p + 1) & 3) * unit) << 16;
    reinterpret_cast<u32x4_t*>(x)[i] = o;
}

// ---------------------------------------------------------------------------
// shrink: part[sk][place][j] = sum over this split's d of in[row][d] W_a[j][d]
// ---------------------------------------------------------------------------
// A workgroup takes a tile of rows, 16*RB ranks and one of SK ranges of d,
// which its eight waves share out again in steps of 128; the matrix cores sum
// 16 rows x 16 ranks x 32 d at a time.  The eight waves' sums meet in LDS, the
// splits' in the expand kernel, both in a fixed order.
// Bound by the bytes of `in`: 4096 x 14336, rank 16, 30 us (3.9 TB/s); 4096 x 4096
// 12 us, of which six are the launch and its chain of waits (plan, rows, data),
// and 17 us with the 8-bit copy; rank 64 adds W from the caches, 2048 x 4096 12
// us.  A step ahead in registers gained a quarter while rows were loaded as
// operands and nothing since they are turned (fewer workgroups fit a CU), so
// there is none.  Tiles of 64 rows and four waves: 42 us at 4096 x 14336.
struct ShrinkArgs {
    Batch b;
    const uint16_t* in;    // [M][D]
    const uint16_t* w;     // [L][r][D]
    float* part;           // [SK][tiles * T][r16]: by place, not by row
    uint8_t* q;            // [M][D] int8 and its scales, or null (D % 128 == 0)
    float* qs;
    int D, r, r16, SK;
};

constexpr int SHRINK_THREADS = 512;
constexpr int SHRINK_WAVES = SHRINK_THREADS / WAVE;

template <int T, int RB, bool Q8, bool WHOLE>
__global__ __launch_bounds__(SHRINK_THREADS) void k_shrink(const ShrinkArgs p)
{
    constexpr int MS = T / 16;
    __shared__ int own[SHRINK_WAVES][SMALL_T];
    // the waves' blocks on their way into operands, and afterwards their sums
    constexpr int PIECES = TURN_PIECES > MS * RB * WAVE ? TURN_PIECES : MS * RB * WAVE;
    __shared__ u32x4_t room[SHRINK_WAVES * PIECES];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const Tile tile = find_tile<T>(p.b, blockIdx.x, own[w]);
    if (tile.a == -2 || (tile.a < 0 && !Q8))
        return;
    u32x4_t* turn = room + w * TURN_PIECES;
    const int steps = (p.D + 127) / 128, parts = p.SK * SHRINK_WAVES;
    const int at = blockIdx.y * SHRINK_WAVES + w, j0 = blockIdx.z * (16 * RB);
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * at / parts);
    const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (at + 1) / parts);

    const Matrix<WHOLE> in(p.in, static_cast<size_t>(p.b.M) * p.D);
    const Matrix<WHOLE> wt(p.w, static_cast<size_t>(p.b.L) * p.r * p.D);
    uint32_t row[MS][4];               // where the lane's columns of row 16 s + 4 i + g start
#pragma unroll
    for (int s = 0; s < MS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            row[s][i] = static_cast<uint32_t>(tile.rows[16 * s + 4 * i + g]) * p.D + 8 * c;
    const uint32_t wrow = static_cast<uint32_t>((tile.a < 0 ? 0 : tile.a) * p.r + j0 + g) * p.D + 8 * c;
    f32x4_t acc[MS][RB];
#pragma unroll
    for (int s = 0; s < MS; ++s)
#pragma unroll
        for (int t = 0; t < RB; ++t)
            acc[s][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    typedef typename Matrix<WHOLE>::Piece Piece;
    auto fetch = [&](int st, Piece (&v)[MS][4], Piece (&wv)[RB][4]) {
        const int d0 = st * 128, valid = p.D - (d0 + 8 * c);
        const bool edge = d0 + 128 > p.D;
#pragma unroll
        for (int t = 0; t < RB; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)      // ranks behind the last are zeros
                wv[t][i] = wt.fetch(wrow + (16 * t + 4 * i) * p.D + d0, j0 + 16 * t + 4 * i + g < p.r ? valid : 0, edge);
#pragma unroll
        for (int s = 0; s < MS; ++s)
            if (16 * s < tile.count)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[s][i] = in.fetch(row[s][i] + d0, 16 * s + 4 * i < tile.count ? valid : 0, edge);
    };
    auto use = [&](int st, const Piece (&vp)[MS][4], const Piece (&wp)[RB][4]) {
        const int d0 = st * 128, valid = p.D - (d0 + 8 * c);
        const bool edge = d0 + 128 > p.D;
        u32x4_t wv[RB][4];
#pragma unroll
        for (int t = 0; t < RB; ++t) {
            u32x4_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = wt.finish(wp[t][i], wrow + (16 * t + 4 * i) * p.D + d0, valid, edge);
            turn16(turn, x, wv[t]);
        }
#pragma unroll
        for (int s = 0; s < MS; ++s) {
            if (16 * s >= tile.count)
                break;
            u32x4_t x[4], v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = in.finish(vp[s][i], row[s][i] + d0, valid, edge);
            turn16(turn, x, v);
            if constexpr (Q8) {
                if (blockIdx.z == 0) {
                    const bool live = 16 * s + c < tile.count;
                    const size_t r = static_cast<size_t>(tile.rows[16 * s + c]);
                    store_row8(v, p.q + r * p.D + d0, p.qs + r * (p.D / GROUP8) + st, g, live);
                }
            }
#pragma unroll
            for (int t = 0; t < RB; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[s][t] = mfma(__builtin_bit_cast(bf16x8_t, v[i]), __builtin_bit_cast(bf16x8_t, wv[t][i]), acc[s][t]);
        }
    };
    for (int st = s0; st < s1; ++st) {
        Piece v[MS][4], wv[RB][4];
        fetch(st, v, wv);
        use(st, v, wv);
    }
    if (tile.a < 0)
        return;
    f32x4_t* red = reinterpret_cast<f32x4_t*>(room);        // [SHRINK_WAVES][MS * RB][WAVE]
    __syncthreads();      // every wave has its operands
#pragma unroll
    for (int e = 0; e < MS * RB; ++e)
        red[(w * MS * RB + e) * WAVE + lane] = acc[e / RB][e % RB];
    __syncthreads();
    const size_t places = static_cast<size_t>(gridDim.x) * T;
    for (int e = w; e < MS * RB; e += SHRINK_WAVES) {     // a 16 x 16 block a wave
        f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int o = 0; o < SHRINK_WAVES; ++o)
            v += red[(o * MS * RB + e) * WAVE + lane];
        const int s = e / RB, j = j0 + 16 * (e % RB) + c;
        if (j < p.r16)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p.part[(blockIdx.y * places + blockIdx.x * T + 16 * s + 4 * g + i) * p.r16 + j] = v[i];
    }
}

// ---------------------------------------------------------------------------
// expand: out[m][d] = base[m][d] + f sum_j c[m][j] W_a[j][d]
// ---------------------------------------------------------------------------
// c is the sum of shrink's SK parts; with SCALED it takes the adapter's scale
// here (dh), else the scale multiplies the sum over j (y).  A wave holds the
// 128 columns of W it works on as matrix-core operands (8 x 8 blocks turned in
// registers, all loads 16 bytes) and goes over the tile's rows, 16 at a time.
// Bound by the bytes of base and out: 4096 x 14336, rank 16, 45 us (5.2 TB/s);
// 2048 x 4096, rank 64, 18 us, where W and the parts come to twice those bytes
// from the caches.  Tiles of 64 rows: 52 us at the first (a third as many waves
// fit a CU); the base rows loaded 16 at a time: 84 us.

// The factors of the weight gradients, in the order their operands take them:
// of each tile (32 places) and 16 ranks, four places of a rank for each lane
// (16 g + c: rank c, places 8 g + 0 .. 3), then the next four.
__host__ __device__ constexpr size_t factor_at(size_t tile, int tiles16, int t) { return (tile * tiles16 + t) * (2 * WAVE); }

struct ExpandArgs {
    Batch b;
    const float* part;        // [SK][tiles * T][r16]
    const uint16_t* w;        // [L][r][D]
    const float* scale;       // [L]
    const uint16_t* base;     // [M][D] or null (0)
    uint16_t* out;            // [M][D] or null (only c is wanted)
    float* c;                 // [M][r] or null
    const float* h;           // [M][r] and
    float* turned;            // c and h as wgrad's operands (factor_at), or null
    int D, r, r16, SK;
};

constexpr int EXPAND_THREADS = 256;
constexpr int EXPAND_COLS = 128 * EXPAND_THREADS / WAVE;

template <int t>
__device__ __forceinline__ void mul_column(f32x4_t (&acc)[8], const Split3& a, const u32x4_t (&R)[8])
{
    const bf16x8_t b = column<t>(R);
#pragma unroll
    for (int q = 0; q < 3; ++q)
        acc[t] = mfma(a.part[q], b, acc[t]);
}

__device__ __forceinline__ void mul_columns(f32x4_t (&acc)[8], const Split3& a, const u32x4_t (&R)[8])
{
    mul_column<0>(acc, a, R);
    mul_column<1>(acc, a, R);
    mul_column<2>(acc, a, R);
    mul_column<3>(acc, a, R);
    mul_column<4>(acc, a, R);
    mul_column<5>(acc, a, R);
    mul_column<6>(acc, a, R);
    mul_column<7>(acc, a, R);
}

// 16 rows x the wave's 128 columns: c from LDS ([16][32 * RK + 4]), W and the
// base rows in registers.
template <int RK, bool WHOLE>
__device__ __forceinline__ void expand16(const float* cs, const u32x4_t (&W)[RK][8],
                                         const typename Matrix<WHOLE>::Piece (&yp)[4], const int* rows, int count, float after,
                                         const Matrix<WHOLE>& base, const Matrix<WHOLE>& out, int D, int d, bool edge)
{
    constexpr int STRIDE = 32 * RK + 4;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    f32x4_t acc[8];
#pragma unroll
    for (int t = 0; t < 8; ++t)
        acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < RK; ++k) {
        float f[8];
        const f32x4_t* src = reinterpret_cast<const f32x4_t*>(cs + c * STRIDE + 32 * k + 8 * g);
        const f32x4_t f0 = src[0], f1 = src[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = f0[e];
            f[4 + e] = f1[e];
        }
        mul_columns(acc, split3(f), W[k]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = 4 * g + i;
        const uint32_t at = static_cast<uint32_t>(rows[m]) * D + d;
        const u32x4_t y = base.finish(yp[i], at, D - d, edge);
        u32x4_t o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = f32_to_bf16(fmaf(after, acc[2 * e][i], bf16_to_f32(y[e] & 0xffffu))) |
                   f32_to_bf16(fmaf(after, acc[2 * e + 1][i], bf16_to_f32(y[e] >> 16))) << 16;
        out.store(at, o, m < count ? D - d : 0, edge);
    }
}

template <int T, int RK, bool SCALED, bool WHOLE>
__global__ __launch_bounds__(EXPAND_THREADS) void k_expand(const ExpandArgs p)
{
    constexpr int MS = T / 16, STRIDE = 32 * RK + 4;   // 4: rows of a quarter wave in other banks
    constexpr int PARTS = 8;                           // parts whose loads go out together
    __shared__ int own[EXPAND_THREADS / WAVE][SMALL_T], rows[T];
    __shared__ __attribute__((aligned(16))) float cs[T * STRIDE];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const Tile tile = find_tile<T>(p.b, blockIdx.y, own[tid >> 6]);
    if (tile.a == -2)
        return;
    const int d0 = blockIdx.x * EXPAND_COLS + (tid >> 6) * 128, d = d0 + 8 * c;     // this lane's 8 columns
    const bool first = blockIdx.x == 0, edge = __builtin_amdgcn_readfirstlane(d0) + 128 > p.D;
    const Matrix<WHOLE> base(p.base, static_cast<size_t>(p.b.M) * p.D), out(p.out, static_cast<size_t>(p.b.M) * p.D);
    const Matrix<WHOLE> wt(p.w, static_cast<size_t>(p.b.L) * p.r * p.D);
    if (tile.a < 0) {     // rows without an adapter: the base as it is
        if (p.c && first)
            for (int i = tid; i < tile.count * p.r; i += EXPAND_THREADS)
                p.c[static_cast<size_t>(tile.rows[i / p.r]) * p.r + i % p.r] = 0.0f;
        if (p.out && p.out != p.base)
            for (int m = g; m < tile.count; m += 4) {
                const uint32_t at = static_cast<uint32_t>(tile.rows[m]) * p.D + d;
                out.store(at, base.finish(base.fetch(at, p.base ? p.D - d : 0, edge), at, p.D - d, edge), p.D - d, edge);
            }
        return;
    }
    // the parts of c (by place: they wait for no row), W and the rows' numbers
    // come in together, then all the base rows
    constexpr int QUADS = 8 * RK, PER = (T * QUADS + EXPAND_THREADS - 1) / EXPAND_THREADS;
    const float scale = p.scale[tile.a];
    const size_t next = static_cast<size_t>(gridDim.y) * T * p.r16;
    typename Matrix<WHOLE>::Piece wp[RK][8], yp[MS][4];
    const uint32_t w0 = static_cast<uint32_t>(tile.a * p.r) * p.D + d;
#pragma unroll
    for (int k = 0; k < RK; ++k)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int j = 32 * k + 8 * g + u;
            wp[k][u] = wt.fetch(w0 + j * p.D, p.out && j < p.r ? p.D - d : 0, edge);
        }
    if (tid < T)
        rows[tid] = tile.rows[tid];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int i = tid + e * EXPAND_THREADS, m = i / QUADS, j = i % QUADS * 4;
        if (i < T * QUADS) {
            f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
            if (m < tile.count && j < p.r16) {
                const float* src = p.part + (static_cast<size_t>(blockIdx.y) * T + m) * p.r16 + j;
                for (int s0 = 0; s0 < p.SK; s0 += PARTS) {
                    f32x4_t x[PARTS];
#pragma unroll
                    for (int s = 0; s < PARTS; ++s)
                        x[s] = s0 + s < p.SK ? *reinterpret_cast<const f32x4_t*>(src + (s0 + s) * next)
                                             : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < PARTS; ++s)
                        v += x[s];
                }
                if (SCALED)
                    v *= scale;
#pragma unroll
                for (int q = 0; q < 4; ++q)      // ranks behind the last: zero weights times an infinity are NaN
                    v[q] = j + q < p.r ? v[q] : 0.0f;
                if (p.c && first) {
                    float* o = p.c + static_cast<size_t>(tile.rows[m]) * p.r + j;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (j + q < p.r)
                            o[q] = v[q];
                }
            }
            *reinterpret_cast<f32x4_t*>(&cs[m * STRIDE + j]) = v;
        }
    }
    __syncthreads();
    if constexpr (T == TILE_T) {
        if (p.turned && first) {     // places behind the last count for nothing
            const int tiles16 = p.r16 / 16;
            f32x4_t* o = reinterpret_cast<f32x4_t*>(p.turned) + factor_at(blockIdx.y, tiles16, 0);
            f32x4_t* oh = o + factor_at(gridDim.y, tiles16, 0);
            for (int i = tid; i < tiles16 * 2 * WAVE; i += EXPAND_THREADS) {
                const int j = i / (2 * WAVE) * 16 + (i & 15), m = (i >> 4 & 3) * 8 + (i / WAVE & 1) * 4;
                f32x4_t v, vh;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = cs[(m + e) * STRIDE + j];
                    vh[e] = p.h && m + e < tile.count && j < p.r ? p.h[static_cast<size_t>(rows[m + e]) * p.r + j] : 0.0f;
                }
                o[i] = v;
                oh[i] = vh;
            }
        }
    }
    if (!p.out || d0 >= p.D)     // waves leave whole: every lane holds matrix-core operands
        return;
#pragma unroll
    for (int s = 0; s < MS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = 16 * s + 4 * g + i;
            yp[s][i] = base.fetch(static_cast<uint32_t>(rows[m]) * p.D + d, p.base && m < tile.count ? p.D - d : 0, edge);
        }
    u32x4_t W[RK][8];
#pragma unroll
    for (int k = 0; k < RK; ++k)
#pragma unroll
        for (int u = 0; u < 8; ++u)
            W[k][u] = wt.finish(wp[k][u], w0 + (32 * k + 8 * g + u) * p.D, p.D - d, edge);
#pragma unroll
    for (int s = 0; s < MS; ++s) {
        if (16 * s >= tile.count)
            break;
        expand16<RK, WHOLE>(cs + 16 * s * STRIDE, W, yp[s], rows + 16 * s, tile.count - 16 * s, SCALED ? 1.0f : scale, base, out,
                            p.D, d, edge);
    }
}

// ---------------------------------------------------------------------------
// both at once, for batches of a few rows
// ---------------------------------------------------------------------------
// Each workgroup works out its tile's c for itself (its eight waves share the
// first product's d out, their sums meet in LDS) and goes on to 1024 columns of
// the second, whose W and base rows it asked for at the start.  The first
// product is repeated for every 1024 columns, from the caches; that is cheaper
// than a second launch while its W is small (one_launch() has the rule).
struct SmallArgs {
    Batch b;
    const uint16_t* in;       // [M][D1]
    const uint16_t* w1;       // [L][r][D1]
    const uint16_t* w2;       // [L][r][D2]
    const float* scale;
    const uint16_t* base;     // [M][D2] or null (0)
    uint16_t* out;            // [M][D2] or null (only c is wanted)
    float* c;                 // [M][r] or null
    uint8_t* q;               // as in ShrinkArgs (D1 % 128 == 0)
    float* qs;
    int D1, D2, r;
    bool scaled;              // c takes the scale (dh), else the sum over j does (y)
};

constexpr int SMALL_THREADS = 512;
constexpr int SMALL_WAVES = SMALL_THREADS / WAVE;
constexpr int SMALL_COLS = 128 * SMALL_WAVES;

template <int RB, bool WHOLE1, bool WHOLE2>
__global__ __launch_bounds__(SMALL_THREADS) void k_small(const SmallArgs p)
{
    constexpr int RK = (RB + 1) / 2, STRIDE = 32 * RK + 4;
    __shared__ int own[SMALL_WAVES][SMALL_T];
    constexpr int PIECES = TURN_PIECES > RB * WAVE ? TURN_PIECES : RB * WAVE;
    __shared__ u32x4_t room[SMALL_WAVES * PIECES];       // as in k_shrink
    __shared__ __attribute__((aligned(16))) float cs[SMALL_T * STRIDE];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, g = lane >> 4;
    const Tile tile = search_tile<1>(p.b, blockIdx.y, own[w]);
    const bool first = blockIdx.x == 0;
    if (tile.a == -2)
        return;
    const int d0 = blockIdx.x * SMALL_COLS + w * 128, d = d0 + 8 * c;
    const bool edge2 = d0 + 128 > p.D2;
    const Matrix<WHOLE2> base(p.base, static_cast<size_t>(p.b.M) * p.D2), out(p.out, static_cast<size_t>(p.b.M) * p.D2);
    const Matrix<WHOLE2> w2(p.w2, static_cast<size_t>(p.b.L) * p.r * p.D2);
    typename Matrix<WHOLE2>::Piece wp[RK][8], yp[4];
    const int a = tile.a < 0 ? 0 : tile.a;
    const uint32_t at2 = static_cast<uint32_t>(a * p.r) * p.D2 + d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = 4 * g + i;
        yp[i] = base.fetch(static_cast<uint32_t>(tile.rows[m]) * p.D2 + d, p.base && m < tile.count ? p.D2 - d : 0, edge2);
    }
#pragma unroll
    for (int k = 0; k < RK; ++k)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int j = 32 * k + 8 * g + u;
            wp[k][u] = w2.fetch(at2 + j * p.D2, p.out && tile.a >= 0 && j < p.r ? p.D2 - d : 0, edge2);
        }
    const float scale = p.scale[a];

    f32x4_t acc[RB];
#pragma unroll
    for (int t = 0; t < RB; ++t)
        acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const bool quant = p.q && first;
    if (tile.a >= 0 || quant) {
        const Matrix<WHOLE1> in(p.in, static_cast<size_t>(p.b.M) * p.D1);
        const Matrix<WHOLE1> w1(p.w1, static_cast<size_t>(p.b.L) * p.r * p.D1);
        typedef typename Matrix<WHOLE1>::Piece Piece;
        u32x4_t* turn = room + w * TURN_PIECES;
        uint32_t row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            row[i] = static_cast<uint32_t>(tile.rows[4 * i + g]) * p.D1 + 8 * c;
        const uint32_t wrow = static_cast<uint32_t>(a * p.r + g) * p.D1 + 8 * c;
        const int steps = (p.D1 + 127) / 128;
        auto fetch = [&](int st, Piece (&x)[4], Piece (&v)[RB][4]) {
            const int o = st * 128, valid = p.D1 - (o + 8 * c);
            const bool edge = o + 128 > p.D1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = in.fetch(row[i] + o, 4 * i < tile.count ? valid : 0, edge);
#pragma unroll
                for (int t = 0; t < RB; ++t)      // ranks behind the last are zeros
                    v[t][i] = w1.fetch(wrow + (16 * t + 4 * i) * p.D1 + o, 16 * t + 4 * i + g < p.r ? valid : 0, edge);
            }
        };
        auto use = [&](int st, const Piece (&xp)[4], const Piece (&vp)[RB][4]) {
            const int o = st * 128, valid = p.D1 - (o + 8 * c);
            const bool edge = o + 128 > p.D1;
            u32x4_t y[4], x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = in.finish(xp[i], row[i] + o, valid, edge);
            turn16(turn, y, x);
            if (quant) {
                const size_t r = static_cast<size_t>(tile.rows[c]);
                store_row8(x, p.q + r * p.D1 + o, p.qs + r * (p.D1 / GROUP8) + st, g, c < tile.count);
            }
#pragma unroll
            for (int t = 0; t < RB; ++t) {
                u32x4_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = w1.finish(vp[t][i], wrow + (16 * t + 4 * i) * p.D1 + o, valid, edge);
                turn16(turn, y, v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[t] = mfma(__builtin_bit_cast(bf16x8_t, x[i]), __builtin_bit_cast(bf16x8_t, v[i]), acc[t]);
            }
        };
        // as many steps' loads at once as fit the registers (K = 4096, rank 16: all)
        constexpr int DEPTH = RB == 1 ? 4 : RB == 2 ? 2 : 1;
        Piece x[DEPTH][4], v[DEPTH][RB][4];
        for (int st = w; st < steps; st += DEPTH * SMALL_WAVES) {
#pragma unroll
            for (int e = 0; e < DEPTH; ++e)
                if (st + e * SMALL_WAVES < steps)
                    fetch(st + e * SMALL_WAVES, x[e], v[e]);
#pragma unroll
            for (int e = 0; e < DEPTH; ++e)
                if (st + e * SMALL_WAVES < steps)
                    use(st + e * SMALL_WAVES, x[e], v[e]);
        }
    }
    f32x4_t* red = reinterpret_cast<f32x4_t*>(room);        // [SMALL_WAVES][RB][WAVE]
    __syncthreads();      // every wave has its operands
#pragma unroll
    for (int t = 0; t < RB; ++t)
        red[(w * RB + t) * WAVE + lane] = acc[t];
    __syncthreads();
    if (w < 2 * RK) {          // 16 ranks a wave; zeros where there are none
        f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
        if (w < RB)
#pragma unroll
            for (int o = 0; o < SMALL_WAVES; ++o)
                v += red[(o * RB + (w < RB ? w : 0)) * WAVE + lane];
        const int j = 16 * w + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = 4 * g + i;
            float f = p.scaled ? v[i] * scale : v[i];
            f = j < p.r && m < tile.count && tile.a >= 0 ? f : 0.0f;
            cs[m * STRIDE + j] = f;
            if (p.c && first && j < p.r && m < tile.count)
                p.c[static_cast<size_t>(tile.rows[m]) * p.r + j] = f;
        }
    }
    __syncthreads();
    if (!p.out || d0 >= p.D2)     // waves leave whole: every lane holds matrix-core operands
        return;
    if (tile.a < 0) {             // rows without an adapter: the base as it is
        if (p.out != p.base)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = 4 * g + i;
                const uint32_t at = static_cast<uint32_t>(tile.rows[m]) * p.D2 + d;
                out.store(at, base.finish(yp[i], at, p.D2 - d, edge2), m < tile.count ? p.D2 - d : 0, edge2);
            }
        return;
    }
    u32x4_t W[RK][8];
#pragma unroll
    for (int k = 0; k < RK; ++k)
#pragma unroll
        for (int u = 0; u < 8; ++u)
            W[k][u] = w2.finish(wp[k][u], at2 + (32 * k + 8 * g + u) * p.D2, p.D2 - d, edge2);
    expand16<RK, WHOLE2>(cs, W, yp, tile.rows, tile.count, p.scaled ? 1.0f : scale, base, out, p.D2, d, edge2);
}

// ---------------------------------------------------------------------------
// wgrad: G_a[j][d] = f sum_m c[m][j] in[m][d]
// ---------------------------------------------------------------------------
// A workgroup takes 128 columns and the rows of one adapter (or one chunk of
// them); its eight waves take 32 rows each in turn, and their sums meet in
// LDS (WIDE: each wave 128 columns and all the rows).  Chunks of one adapter leave partial sums, which k_wgrad_sum adds in
// order.  In 8 bits, the row's scale of these 128 channels goes into c, whose
// three bf16 parts hold it, and the whole numbers are exact bf16 values.
// Bound by the bytes of `in`: 4096 rows of 4096 columns in 8 bits and 14336 in
// bf16, rank 16, 26 us (5.1 TB/s); rank 64, 2048 x 8192, 22 us, where the factors
// come to as many bytes again.  Factors by row instead of operand order: 46 and
// 47 us.  Chunks of 1024 rows: 28 and 19 us there, but 17 against 12 us at 4096 x
// 1024, rank 64, where they leave half the CUs idle; of 256: 27 and 27 us.
struct WgradJob {
    const uint16_t* in;      // [M][D] bf16, or null:
    const uint8_t* q;        // [M][D] int8 and
    const float* qs;         // [M][D/128] its scales
    const float* c;          // up to SMALL_M rows [M][r], else as factor_at() says
    float* out;              // [L][r][D] or null
    float* part;             // [slots][r][cols * 128]
    int D, cols;             // columns, and blocks of 128 of them
    bool scaled;             // multiply by the adapter's scale
};

struct WgradArgs {
    Batch b;
    const float* scale;
    WgradJob job[2];
    int r, r16;
    bool chunked;            // blockIdx.y is a chunk of the plan; else an adapter
};

constexpr int WGRAD_THREADS = 512;
constexpr int WGRAD_WAVES = WGRAD_THREADS / WAVE;

template <int RT, bool WHOLE, bool SMALL, bool WIDE>
__global__ __launch_bounds__(WGRAD_THREADS) void k_wgrad(const WgradArgs p)
{
    constexpr int STRIDE = 128 + 4;      // 4: rows of a quarter wave in other banks
    __shared__ __attribute__((aligned(16))) float red[WGRAD_WAVES][16 * STRIDE];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, g = lane >> 4;
    constexpr int SHARE = WIDE ? 1 : WGRAD_WAVES;          // waves that share the rows out
    const int block = WIDE ? static_cast<int>(blockIdx.x) * WGRAD_WAVES + w : static_cast<int>(blockIdx.x);
    if (WIDE && block >= p.job[0].cols + p.job[1].cols)    // no barriers then
        return;
    const int at_row = WIDE ? 0 : 32 * w;
    const bool second = block >= p.job[0].cols;
    const WgradJob job = second ? p.job[1] : p.job[0];
    const int cb = block - (second ? p.job[0].cols : 0), j0 = blockIdx.z * (16 * RT);
    int a = blockIdx.y, count = 0, slot = -1, first = 0;
    const int* rows;
    if constexpr (!SMALL) {
        if (!fits(p.b))
            return;
        const PlanLayout l(p.b.M, p.b.L);
        if (p.chunked) {
            const int* e = p.b.plan + l.chunk + 4 * static_cast<int64_t>(a);
            if (a >= p.b.plan[1])
                return;
            a = e[0];
            first = e[1];
            count = e[2];
            slot = e[3];
        } else {
            first = p.b.plan[l.first + a] * TILE_T;
            count = p.b.plan[l.count + a];
        }
        rows = p.b.plan + l.rows + first;
    } else {
        // every wave lists the rows for itself, where its sums go afterwards
        int* own = reinterpret_cast<int*>(red[w]);
        const bool mine = lane < p.b.M && p.b.ids[lane < p.b.M ? lane : 0] == a;
        const uint64_t m = __ballot(mine);
        count = __builtin_popcountll(m);
        if (count && lane >= count)
            own[lane] = 63 - __builtin_clzll(m);      // places behind the last repeat it
        if (mine)
            own[__builtin_popcountll(m & ((1ull << lane) - 1))] = lane;
        wave_sync();
        rows = own;
    }
    const int d = cb * 128 + 8 * c;
    const bool edge = cb * 128 + 128 > job.D;
    const Matrix<WHOLE> in(job.in, static_cast<size_t>(p.b.M) * job.D);
    f32x4_t acc[RT][8];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int t = 0; t < 8; ++t)
            acc[rt][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    // 32 rows: their numbers, 8 x 8 blocks of their columns and their factors
    auto step = [&](int m0, auto in8) {
        constexpr bool Q8 = decltype(in8)::value;
        uint32_t row[8];
        typename Matrix<WHOLE>::Piece x[8];
        u32x2_t q[8];
        float unit[8], f[RT][8];
#pragma unroll
        for (int u = 0; u < 8; ++u)      // m0 + 31 lies in the last row's tile
            row[u] = static_cast<uint32_t>(rows[m0 + 8 * g + u]);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if constexpr (Q8) {
                q[u] = *reinterpret_cast<const u32x2_t*>(job.q + row[u] * job.D + d);
                unit[u] = job.qs[row[u] * (job.D / GROUP8) + cb];
            } else {
                x[u] = in.fetch(row[u] * job.D + d, job.D - d, edge);
            }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int j = j0 + 16 * rt + c;
            if constexpr (SMALL) {
#pragma unroll
                for (int u = 0; u < 8; ++u)     // places behind the last count for nothing
                    f[rt][u] = m0 + 8 * g + u < count && j < p.r ? job.c[row[u] * p.r + j] : 0.0f;
            } else if (j0 + 16 * rt < p.r16) {
                const f32x4_t* src = reinterpret_cast<const f32x4_t*>(job.c) +
                                     factor_at((first + m0) / TILE_T, p.r16 / 16, j0 / 16 + rt) + lane;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[rt][e] = src[e / 4 * WAVE][e % 4];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[rt][e] = 0.0f;
            }
        }
        u32x4_t R[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if constexpr (Q8) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    R[u][e] = __builtin_amdgcn_perm(__float_as_uint(byte_to_f32(q[u][e / 2], (2 * e + 1) & 3)),
                                                    __float_as_uint(byte_to_f32(q[u][e / 2], (2 * e) & 3)), 0x07060302u);
            } else {
                R[u] = in.finish(x[u], row[u] * job.D + d, job.D - d, edge);
            }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            if constexpr (Q8)
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    f[rt][u] *= unit[u];
            mul_columns(acc[rt], split3(f[rt]), R);
        }
    };
    if (job.in)
        for (int m0 = at_row; m0 < count; m0 += 32 * SHARE)
            step(m0, std::false_type{});
    else
        for (int m0 = at_row; m0 < count; m0 += 32 * SHARE)
            step(m0, std::true_type{});
    const float f = slot < 0 && job.scaled && count ? p.scale[a] : 1.0f;
    const size_t width = slot < 0 ? job.D : static_cast<size_t>(job.cols) * 128;
    float* out = slot < 0 ? job.out + static_cast<size_t>(a) * p.r * width : job.part + static_cast<size_t>(slot) * p.r * width;
    auto store = [&](float* o, f32x4_t v, int at) {       // columns at .. at + 3 of this job
        v *= f;
        if (WHOLE || slot >= 0 || at + 4 <= job.D) {
            if (slot >= 0 || at < job.D)
                *reinterpret_cast<f32x4_a4_t*>(o) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at + i < job.D)
                    o[i] = v[i];
        }
    };
    if (WIDE || count <= 32) {   // a wave, the first, has it all
        if (!WIDE && w > 0)
            return;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = j0 + 16 * rt + 4 * g + i;
                if (j < p.r)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        store(out + j * width + d + 4 * h,
                              f32x4_t{acc[rt][4 * h][i], acc[rt][4 * h + 1][i], acc[rt][4 * h + 2][i], acc[rt][4 * h + 3][i]}, d + 4 * h);
            }
        return;
    }
    // 16 ranks at a time, the eight waves' sums side by side, then added in
    // order by all threads: 4 columns of one rank each
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<f32x4_t*>(&red[w][(4 * g + i) * STRIDE + 8 * c + 4 * h]) =
                    f32x4_t{acc[rt][4 * h][i], acc[rt][4 * h + 1][i], acc[rt][4 * h + 2][i], acc[rt][4 * h + 3][i]};
        __syncthreads();
        const int q = tid >> 5, e = (tid & 31) * 4, j = j0 + 16 * rt + q, at = cb * 128 + e;
        f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int o = 0; o < WGRAD_WAVES; ++o)
            v += *reinterpret_cast<const f32x4_t*>(&red[o][q * STRIDE + e]);
        if (j < p.r)
            store(out + j * width + at, v, at);
    }
}

// Adapters of several chunks: their partial sums in order, 4 columns a thread and
// four chunks' loads at a time (2048 rows of 4 adapters, rank 64, 4096 + 4099
// columns 4.9 us; one column a thread 3 us more).  Adapters without
// rows: zeros.  (An adapter of one chunk is done.)
__global__ __launch_bounds__(256) void k_wgrad_sum(const WgradArgs p)
{
    const int a = blockIdx.y, j = blockIdx.z;
    if (!fits(p.b))
        return;
    const PlanLayout l(p.b.M, p.b.L);
    const int n = chunks_of(p.b.plan[l.count + a]);
    if (n == 1)
        return;
    int d = (blockIdx.x * 256 + threadIdx.x) * 4;
    const int first = p.job[0].cols * 128;
    const bool second = d >= first;
    const WgradJob job = second ? p.job[1] : p.job[0];
    d -= second ? first : 0;
    if (d >= job.D || !job.out)
        return;
    const size_t width = static_cast<size_t>(job.cols) * 128;
    const float* src = job.part + (static_cast<size_t>(p.b.plan[l.slot + a]) * p.r + j) * width + d;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i0 = 0; i0 < n; i0 += 4) {
        f32x4_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = i0 + i < n ? *reinterpret_cast<const f32x4_t*>(src + static_cast<size_t>(i0 + i) * p.r * width)
                              : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v += x[i];
    }
    v *= job.scaled && n ? p.scale[a] : 1.0f;
    float* o = job.out + (static_cast<size_t>(a) * p.r + j) * job.D + d;
    if (d + 4 <= job.D) {
        *reinterpret_cast<f32x4_a4_t*>(o) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < job.D)
                o[e] = v[e];
    }
}

// Gradients of an empty batch.
__global__ __launch_bounds__(256) void k_lora_zero(float* __restrict__ p, size_t n)
{
    const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
    if (i < n)
        p[i] = 0.0f;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int round16(int64_t r) { return static_cast<int>((r + 15) / 16 * 16); }

// Ranges that a shrink's D is split into: enough workgroups for the chip, at
// most as many as leave a wave no more than one step of 128 d (some of the last
// one's waves may have none), and few enough that the parts stay small beside
// the rows (the expand kernel reads them all).  One split fewer where the steps
// are no multiple of eight, so that each wave has a step, takes longer: whole
// calls of 64 rows, rank 64, 1152 to 4096 11.2 us against 10.3 here; 1000 rows of
// 2176, rank 8, 15.8 against 15.1; 1000 of 1152, rank 128, 28.2 and 28.4.
// Beyond rank 32 the registers leave a CU one workgroup: the split with the
// fewest steps over all rounds of the 256 CUs, two more a round to start and to
// add up.  (Two a CU and up to four parts there too, whole calls in us: 1000 x
// 14336 to 4096, rank 128, 48 against 43; 2048 x 4096, rank 128, 48 against 42;
// 8000 x 4096, rank 64, 77 against 71.)
int split_of(int64_t M, int64_t L, int64_t D, int64_t r, bool ballots)
{
    const int64_t steps = (D + 127) / 128, most = (steps + SHRINK_WAVES - 1) / SHRINK_WAVES;
    const int64_t groups = tile_bound(M, L, ballots) * ((r + 63) / 64);
    const int64_t cap = M <= SMALL_M ? 16 : ballots || r > 32 ? 8 : 4;
    int64_t want = ballots ? cap : (512 + groups - 1) / groups;
    if (!ballots && r > 32) {
        int64_t least = INT64_MAX;
        for (int64_t n = 1; n <= cap; ++n) {
            const int64_t time = (groups * n + 255) / 256 * ((steps + SHRINK_WAVES * n - 1) / (SHRINK_WAVES * n) + 2);
            if (time < least) {
                least = time;
                want = n;
            }
        }
    }
    want = want < cap ? want : cap;
    return static_cast<int>(want < most ? want : most);
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

size_t part_bytes(int64_t M, int64_t L, int64_t D, int64_t r, bool ballots)
{
    const int64_t places = tile_bound(M, L, ballots) * (ballots ? SMALL_T : TILE_T);
    return up256(static_cast<size_t>(split_of(M, L, D, r, ballots)) * places * round16(r) * 4);
}

size_t plan_bytes(int64_t M, int64_t L) { return up256(static_cast<size_t>(plan_words(M, L)) * 4); }

// partial-sum slots: chunks of adapters with more than one
int64_t slot_bound(int64_t M) { return M > CHUNK ? 2 * (M / CHUNK) : 0; }

size_t wgrad_bytes(int64_t M, int64_t D, int64_t r)
{
    return up256(static_cast<size_t>(slot_bound(M)) * r * ((D + 127) / 128 * 128) * 4);
}

// what the weight gradients multiply with: dh by row, or dh and h by place
size_t factor_bytes(int64_t M, int64_t L, int64_t r)
{
    return up256(static_cast<size_t>(M <= SMALL_M ? M * r : 2 * round16(r) * tile_bound(M, L, false) * TILE_T) * 4);
}

bool sizes_ok(int64_t M, int64_t N, int64_t K, int64_t r, int64_t L)
{
    const int64_t top = static_cast<int64_t>(1) << 31, widest = static_cast<int64_t>(1) << 24;   // grids: 512 columns a workgroup
    return M >= 0 && M <= MAX_M && N >= 0 && N <= widest && K >= 128 && K % 128 == 0 && K <= widest && r >= 1 &&
           r <= MAX_RANK && L >= 1 && L <= MAX_ADAPTERS && M * K * 2 < top && M * N * 2 < top &&
           L * r * K < top / 2 && L * r * N < top / 2;
}

template <bool Q8, bool WHOLE>
void launch_shrink_as(const ShrinkArgs& s, int64_t tiles, hipStream_t stream)
{
    const int rb = s.r <= 16 ? 1 : s.r <= 32 ? 2 : 4;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(s.SK), static_cast<unsigned>((s.r + 16 * rb - 1) / (16 * rb)));
#define SHRINK(T_, RB_) hipLaunchKernelGGL((k_shrink<T_, RB_, Q8, WHOLE>), grid, dim3(SHRINK_THREADS), 0, stream, s)
    if (!s.b.plan) {
        if (rb == 1) SHRINK(SMALL_T, 1);
        else if (rb == 2) SHRINK(SMALL_T, 2);
        else SHRINK(SMALL_T, 4);
    } else {
        if (rb == 1) SHRINK(TILE_T, 1);
        else if (rb == 2) SHRINK(TILE_T, 2);
        else SHRINK(TILE_T, 4);
    }
#undef SHRINK
}

void launch_shrink(const ShrinkArgs& s, int64_t tiles, hipStream_t stream)
{
    if (s.q)                      // D is a multiple of 128 then
        launch_shrink_as<true, true>(s, tiles, stream);
    else if (s.D % 8 == 0 && is_aligned(s.in, 16) && is_aligned(s.w, 16))
        launch_shrink_as<false, true>(s, tiles, stream);
    else
        launch_shrink_as<false, false>(s, tiles, stream);
}

template <bool SCALED, bool WHOLE>
void launch_expand_as(const ExpandArgs& e, int64_t tiles, hipStream_t stream)
{
    const unsigned cols = e.out ? static_cast<unsigned>((e.D + EXPAND_COLS - 1) / EXPAND_COLS) : 1;
    const dim3 grid(cols, static_cast<unsigned>(tiles));     // neighbours write neighbouring columns
#define EXPAND(T_, RK_) hipLaunchKernelGGL((k_expand<T_, RK_, SCALED, WHOLE>), grid, dim3(EXPAND_THREADS), 0, stream, e)
    if (!e.b.plan) {
        if (e.r <= 32) EXPAND(SMALL_T, 1);
        else if (e.r <= 64) EXPAND(SMALL_T, 2);
        else EXPAND(SMALL_T, 4);
    } else {
        if (e.r <= 32) EXPAND(TILE_T, 1);
        else if (e.r <= 64) EXPAND(TILE_T, 2);
        else EXPAND(TILE_T, 4);
    }
#undef EXPAND
}

void launch_expand(const ExpandArgs& e, int64_t tiles, bool scaled, hipStream_t stream)
{
    if (scaled)                   // D is K, a multiple of 128
        launch_expand_as<true, true>(e, tiles, stream);
    else if (e.D % 8 == 0 && is_aligned(e.base, 16) && is_aligned(e.out, 16) && is_aligned(e.w, 16))
        launch_expand_as<false, true>(e, tiles, stream);
    else
        launch_expand_as<false, false>(e, tiles, stream);
}

// Whether a few rows' two products go in one launch: while every workgroup can
// read the first one's W for itself in about two microseconds.  One launch
// against two, kernels alone: K 4096, rank 16, one row 7.7 us against 8.5, 16
// adapters to 14336 columns 10.8 against 12.1; K 8192, rank 16, 10.9 against 8.5;
// K 2048, rank 64, 11.7 against 10.5.  The second launch costs the caller another
// 3 us.
bool one_launch(int64_t M, int64_t D1, int64_t r) { return M <= SMALL_M && r <= 64 && D1 * r <= 64 * 1024; }

void launch_small(const SmallArgs& a, int64_t tiles, hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(a.out ? (a.D2 + SMALL_COLS - 1) / SMALL_COLS : 1), static_cast<unsigned>(tiles));
    const bool whole1 = a.D1 % 8 == 0 && is_aligned(a.in, 16) && is_aligned(a.w1, 16);
    const bool whole2 = a.D2 % 8 == 0 && is_aligned(a.base, 16) && is_aligned(a.out, 16) && is_aligned(a.w2, 16);
#define SMALL_AS(RB_, W1_, W2_) hipLaunchKernelGGL((k_small<RB_, W1_, W2_>), grid, dim3(SMALL_THREADS), 0, stream, a)
#define SMALL_RB(W1_, W2_)                      \
    do {                                        \
        if (a.r <= 16) SMALL_AS(1, W1_, W2_);   \
        else if (a.r <= 32) SMALL_AS(2, W1_, W2_); \
        else SMALL_AS(4, W1_, W2_);             \
    } while (0)
    if (whole1 && whole2) SMALL_RB(true, true);
    else if (whole1) SMALL_RB(true, false);
    else if (whole2) SMALL_RB(false, true);
    else SMALL_RB(false, false);
#undef SMALL_RB
#undef SMALL_AS
}

template <bool WHOLE, bool WIDE>
void launch_wgrad_as(const WgradArgs& a, hipStream_t stream)
{
    const int rt = a.r <= 16 ? 1 : a.r <= 32 ? 2 : 4;
    const int64_t ys = a.chunked ? PlanLayout(a.b.M, a.b.L).CB : a.b.L;
    const unsigned cols = static_cast<unsigned>(a.job[0].cols + a.job[1].cols);
    const dim3 grid(WIDE ? (cols + WGRAD_WAVES - 1) / WGRAD_WAVES : cols, static_cast<unsigned>(ys),
                    static_cast<unsigned>((a.r + 16 * rt - 1) / (16 * rt)));
#define WGRAD(RT_, SMALL_) hipLaunchKernelGGL((k_wgrad<RT_, WHOLE, SMALL_, WIDE>), grid, dim3(WGRAD_THREADS), 0, stream, a)
    if (!a.b.plan) {
        if (rt == 1) WGRAD(1, true);
        else if (rt == 2) WGRAD(2, true);
        else WGRAD(4, true);
    } else {
        if (rt == 1) WGRAD(1, false);
        else if (rt == 2) WGRAD(2, false);
        else WGRAD(4, false);
    }
#undef WGRAD
    if (a.chunked)
        hipLaunchKernelGGL(k_wgrad_sum, dim3((cols * 32 + 255) / 256, static_cast<unsigned>(a.b.L), static_cast<unsigned>(a.r)),
                           dim3(256), 0, stream, a);
}

// Eight waves for one block of 128 columns, or one each: the latter leaves no wave
// idle with adapters of few rows and needs no sums in LDS, but an eighth of the
// workgroups, so from one a CU on.  Whole backward calls in us, shared against
// one each: 635 rows of 52 adapters, 9600 to 11704, rank 39, 212 against 113; 64 of 64,
// 4096 x 4096, rank 64, 88 and 54; 4096 of 64, rank 64, 196 and 132; 20000 of 8, rank
// 64, 330 and 315.  Below: 4096 of 8, rank 16, 60 and 80; 2048 of 4, rank 64, 58 and
// 81.  Low ranks with long runs of rows gain nothing: 8000 of 16, 4096 to 14336, rank
// 16, 170 and 181.  The rule counts adapters and knows nothing of how the rows are
// spread over them; 4096 rows, 4096 x 4096, in a graph: nine tenths with one of 64,
// rank 16, 77 and 73, rank 64, 188 and 162; but all with one of 64, 57 and 66, 102 and
// 124.
template <bool WHOLE>
void launch_wgrad(const WgradArgs& a, hipStream_t stream)
{
    const int64_t ys = a.chunked ? PlanLayout(a.b.M, a.b.L).CB : a.b.L, cols = a.job[0].cols + a.job[1].cols;
    const int64_t wide = (cols + WGRAD_WAVES - 1) / WGRAD_WAVES * ys * (a.r > 64 ? 2 : 1);
    if (wide >= 256 && (a.r > 16 || a.b.M <= 256 * static_cast<int64_t>(a.b.L)))
        launch_wgrad_as<WHOLE, true>(a, stream);
    else
        launch_wgrad_as<WHOLE, false>(a, stream);
}

}  // namespace

extern "C" {

size_t any4_lora_plan_bytes(int64_t M, int64_t L)
{
    if (M <= 0 || M > MAX_M || L < 1 || L > MAX_ADAPTERS)
        return 0;
    return plan_bytes(M, L);
}

any4_status any4_lora_plan(const int32_t* ids, void* plan, size_t bytes, int64_t M, int64_t L, hipStream_t stream)
{
    if (M < 0 || M > MAX_M || L < 1 || L > MAX_ADAPTERS)
        return ANY4_E_SHAPE;
    if (M == 0)
        return ANY4_OK;
    if (!ids || !plan)
        return ANY4_E_NULL;
    if (!is_aligned(ids, 4) || !is_aligned(plan, 16))
        return ANY4_E_ALIGN;
    if (bytes < plan_bytes(M, L))
        return ANY4_E_WORKSPACE;
    (void)hipGetLastError();
    launch_plan(ids, static_cast<int32_t*>(plan), M, L, stream);
    return launch_status();
}

size_t any4_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, int64_t L)
{
    if (M <= 0 || !sizes_ok(M, N, K, r, L) || one_launch(M, K, r))
        return 0;
    const bool ballots = by_ballots(M, L);
    return part_bytes(M, L, K, r, ballots) + (ballots ? 0 : plan_bytes(M, L));
}

any4_status any4_lora(const uint16_t* x, const uint16_t* A, const uint16_t* B, const float* scale, const int32_t* ids,
                      const void* plan, const uint16_t* y, uint16_t* out, float* h, int8_t* q, float* qs, int64_t M,
                      int64_t N, int64_t K, int64_t r, int64_t L, void* workspace, size_t workspace_bytes,
                      hipStream_t stream)
{
    if (!sizes_ok(M, N, K, r, L))
        return ANY4_E_SHAPE;
    if (M == 0)
        return ANY4_OK;
    const size_t need = any4_lora_workspace_size(M, N, K, r, L);
    if (!x || !A || !scale || !ids || (N > 0 && (!B || !y || !out)) || (!q != !qs) || (need && !workspace))
        return ANY4_E_NULL;
    if (!is_aligned(x, 16) || !is_aligned(A, 16) || !is_aligned(B, 2) || !is_aligned(y, 2) || !is_aligned(out, 2) ||
        !is_aligned(scale, 4) || !is_aligned(ids, 4) || !is_aligned(plan, 16) || !is_aligned(h, 4) ||
        !is_aligned(q, 16) || !is_aligned(qs, 4) || !is_aligned(workspace, 16))
        return ANY4_E_ALIGN;
    if (workspace_bytes < need)
        return ANY4_E_WORKSPACE;
    (void)hipGetLastError();
    float* part = static_cast<float*>(workspace);
    Batch b{ids, nullptr, static_cast<int>(M), static_cast<int>(L), plan != nullptr};
    const bool ballots = by_ballots(M, L);
    if (!ballots) {
        b.plan = static_cast<const int*>(plan);
        if (!plan) {
            int32_t* made = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + part_bytes(M, L, K, r, false));
            launch_plan(ids, made, M, L, stream);
            b.plan = made;
        }
    }
    const int r16 = round16(r), SK = split_of(M, L, K, r, ballots);
    const int64_t tiles = tile_bound(M, L, ballots);
    if (one_launch(M, K, r)) {
        launch_small(SmallArgs{b, x, A, B, scale, y, N > 0 ? out : nullptr, h, reinterpret_cast<uint8_t*>(q), qs,
                               static_cast<int>(K), static_cast<int>(N), static_cast<int>(r), false}, tiles, stream);
        return launch_status();
    }
    const ShrinkArgs s{b, x, A, part, reinterpret_cast<uint8_t*>(q), qs, static_cast<int>(K), static_cast<int>(r), r16, SK};
    launch_shrink(s, tiles, stream);
    const ExpandArgs e{b, part, B, scale, y, N > 0 ? out : nullptr, h, nullptr, nullptr, static_cast<int>(N), static_cast<int>(r), r16, SK};
    if (e.out || h)
        launch_expand(e, tiles, false, stream);
    return launch_status();
}

size_t any4_lora_backward_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, int64_t L)
{
    if (M <= 0 || N <= 0 || !sizes_ok(M, N, K, r, L))
        return 0;
    return part_bytes(M, L, N, r, M <= SMALL_M) + factor_bytes(M, L, r) + (M <= SMALL_M ? 0 : plan_bytes(M, L)) +
           wgrad_bytes(M, K, r) + wgrad_bytes(M, N, r);
}

any4_status any4_lora_backward(const uint16_t* dy, const uint16_t* x, const int8_t* q, const float* qs, const float* h,
                               const uint16_t* A, const uint16_t* B, const float* scale, const int32_t* ids,
                               const void* plan, const uint16_t* dx, uint16_t* dx_out, float* dA, float* dB, int64_t M,
                               int64_t N, int64_t K, int64_t r, int64_t L, void* workspace, size_t workspace_bytes,
                               hipStream_t stream)
{
    if (!sizes_ok(M, N, K, r, L) || N == 0)
        return ANY4_E_SHAPE;
    if (M == 0) {
        if (!is_aligned(dA, 4) || !is_aligned(dB, 4))
            return ANY4_E_ALIGN;
        (void)hipGetLastError();
        const size_t nA = dA ? static_cast<size_t>(L) * r * K : 0, nB = dB ? static_cast<size_t>(L) * r * N : 0;
        if (nA)
            hipLaunchKernelGGL(k_lora_zero, dim3(static_cast<unsigned>((nA + 255) / 256)), dim3(256), 0, stream, dA, nA);
        if (nB)
            hipLaunchKernelGGL(k_lora_zero, dim3(static_cast<unsigned>((nB + 255) / 256)), dim3(256), 0, stream, dB, nB);
        return nA || nB ? launch_status() : ANY4_OK;
    }
    if (!dy || !A || !B || !scale || !ids || !workspace || (dA && !x && (!q || !qs)) || (dB && !h))
        return ANY4_E_NULL;
    if (!is_aligned(dy, 2) || !is_aligned(x, 16) || !is_aligned(q, 16) || !is_aligned(qs, 4) || !is_aligned(h, 4) ||
        !is_aligned(A, 16) || !is_aligned(B, 2) || !is_aligned(scale, 4) || !is_aligned(ids, 4) ||
        !is_aligned(plan, 16) || !is_aligned(dx, 16) || !is_aligned(dx_out, 16) || !is_aligned(dA, 4) ||
        !is_aligned(dB, 4) || !is_aligned(workspace, 16))
        return ANY4_E_ALIGN;
    if (workspace_bytes < any4_lora_backward_workspace_size(M, N, K, r, L))
        return ANY4_E_WORKSPACE;
    (void)hipGetLastError();
    char* at = static_cast<char*>(workspace);
    float* part = reinterpret_cast<float*>(at);
    const bool small = M <= SMALL_M;
    at += part_bytes(M, L, N, r, small);
    float* factors = reinterpret_cast<float*>(at);
    at += factor_bytes(M, L, r);
    Batch b{ids, nullptr, static_cast<int>(M), static_cast<int>(L), plan != nullptr};
    if (!small) {
        b.plan = static_cast<const int*>(plan);
        if (!plan) {
            launch_plan(ids, reinterpret_cast<int32_t*>(at), M, L, stream);
            b.plan = reinterpret_cast<const int*>(at);
        }
        at += plan_bytes(M, L);
    }
    const int r16 = round16(r), SK = split_of(M, L, N, r, small);
    const int64_t tiles = tile_bound(M, L, small);
    const bool need_dh = dx_out || dA;
    if (need_dh && one_launch(M, N, r)) {
        launch_small(SmallArgs{b, dy, B, A, scale, dx, dx_out, factors, nullptr, nullptr, static_cast<int>(N),
                               static_cast<int>(K), static_cast<int>(r), true}, tiles, stream);
    } else if (need_dh) {
        const ShrinkArgs s{b, dy, B, part, nullptr, nullptr, static_cast<int>(N), static_cast<int>(r), r16, SK};
        launch_shrink(s, tiles, stream);
    }
    if ((need_dh && !one_launch(M, N, r)) || (dB && !small)) {      // without dh: only h is turned
        const ExpandArgs e{b, part, A, scale, dx, dx_out, small ? factors : nullptr, dB ? h : nullptr,
                           small || (!dA && !dB) ? nullptr : factors, static_cast<int>(K), static_cast<int>(r), r16, need_dh ? SK : 0};
        launch_expand(e, tiles, true, stream);
    }
    if (dA || dB) {
        const bool chunked = M > CHUNK;
        WgradArgs g{b, scale, {}, static_cast<int>(r), r16, chunked};
        g.job[0] = WgradJob{x, reinterpret_cast<const uint8_t*>(q), qs, factors, dA, reinterpret_cast<float*>(at),
                            static_cast<int>(K), dA ? static_cast<int>(K / 128) : 0, false};
        at += wgrad_bytes(M, K, r);
        g.job[1] = WgradJob{dy, nullptr, nullptr, small ? h : factors + 4 * factor_at(tiles, r16 / 16, 0), dB, reinterpret_cast<float*>(at), static_cast<int>(N),
                            dB ? static_cast<int>((N + 127) / 128) : 0, true};
        if (N % 8 == 0 && is_aligned(dy, 16) && is_aligned(dA, 16) && is_aligned(dB, 16))
            launch_wgrad<true>(g, stream);
        else
            launch_wgrad<false>(g, stream);
    }
    return launch_status();
}

any4_status any4_act8_save(const uint16_t* x, int8_t* q, float* qs, int64_t M, int64_t K, hipStream_t stream)
{
    if (M < 0 || M > ACT8_MAX_M || K < 0 || K % GROUP8 != 0 || K >= (static_cast<int64_t>(1) << 31) ||
        M * K * 2 >= (static_cast<int64_t>(1) << 31))
        return ANY4_E_SHAPE;
    if (M == 0 || K == 0)
        return ANY4_OK;
    if (!x || !q || !qs)
        return ANY4_E_NULL;
    if (!is_aligned(x, 16) || !is_aligned(q, 16) || !is_aligned(qs, 4))
        return ANY4_E_ALIGN;
    (void)hipGetLastError();
    const uint32_t slots = static_cast<uint32_t>(M * K / 8);
    hipLaunchKernelGGL(k_act8_save, dim3((slots + ACT8_THREADS - 1) / ACT8_THREADS), dim3(ACT8_THREADS), 0, stream, x,
                       reinterpret_cast<uint8_t*>(q), qs, slots);
    return launch_status();
}

any4_status any4_act8_load(const int8_t* q, const float* qs, uint16_t* x, int64_t M, int64_t K, hipStream_t stream)
{
    if (M < 0 || M > ACT8_MAX_M || K < 0 || K % GROUP8 != 0 || K >= (static_cast<int64_t>(1) << 31) ||
        M * K * 2 >= (static_cast<int64_t>(1) << 31))
        return ANY4_E_SHAPE;
    if (M == 0 || K == 0)
        return ANY4_OK;
    if (!q || !qs || !x)
        return ANY4_E_NULL;
    if (!is_aligned(q, 16) || !is_aligned(qs, 4) || !is_aligned(x, 16))
        return ANY4_E_ALIGN;
    (void)hipGetLastError();
    const uint32_t slots = static_cast<uint32_t>(M * K / 8);
    hipLaunchKernelGGL(k_act8_load, dim3((slots + ACT8_THREADS - 1) / ACT8_THREADS), dim3(ACT8_THREADS), 0, stream,
                       reinterpret_cast<const uint8_t*>(q), qs, x, slots);
    return launch_status();
}

}  // extern "C"
