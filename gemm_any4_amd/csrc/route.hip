// Routing to experts and the sum that the router weights, with their backward
// passes.  The C ABI and the formulas are in include/any4.h.
#include <type_traits>

#include "frag.h"

namespace {

constexpr int MAX_EXPERTS = 1024;
constexpr int MAX_K = 64;
constexpr int MAX_GROUPS = 64;
constexpr int64_t MAX_T = static_cast<int64_t>(1) << 20;

enum { SCORE_SOFTMAX, SCORE_SIGMOID };

constexpr int ROUTE_WAVES = 4;       // tokens of a workgroup, a wave each

// A logit: -inf where the expert is out (-inf, NaN), +inf as the largest finite value.
__device__ __forceinline__ float logit_at(const void* logits, int bf16, size_t i)
{
    const float l = bf16 ? bf16_to_f32(static_cast<const uint16_t*>(logits)[i]) : static_cast<const float*>(logits)[i];
    return l != l ? -INFINITY : fminf(l, 3.4028234663852886e38f);
}

// A value from another lane by DPP (0 where there is none): rows of 16 shifted, then
// the last lane of a row to the next row and of 32 lanes to the rest.
template <int CTRL, int ROW_MASK, typename T>
__device__ __forceinline__ T moved(T v, T otherwise)
{
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, otherwise), __builtin_bit_cast(int, v), CTRL, ROW_MASK, 0xf, false));
    } else {
        const u32x2_t a = __builtin_bit_cast(u32x2_t, v), o = __builtin_bit_cast(u32x2_t, otherwise);
        const u32x2_t r = {static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(o[0]), static_cast<int>(a[0]), CTRL, ROW_MASK, 0xf, false)),
                           static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(o[1]), static_cast<int>(a[1]), CTRL, ROW_MASK, 0xf, false))};
        return __builtin_bit_cast(T, r);
    }
}

template <typename T>
__device__ __forceinline__ T from_lane(T v, int lane)
{
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    } else {
        const u32x2_t a = __builtin_bit_cast(u32x2_t, v);
        const u32x2_t r = {static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(a[0]), lane)),
                           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(a[1]), lane))};
        return __builtin_bit_cast(T, r);
    }
}

// Over the wave's 64 lanes, the same for all: each lane joins with ever farther ones
// before it, and lane 63 has them all (a shuffle through LDS takes several times a
// DPP move's time, and routing is a chain of these).
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, T none, F join)
{
    v = join(v, moved<0x111, 0xf>(v, none));     // row_shr 1, 2, 4, 8
    v = join(v, moved<0x112, 0xf>(v, none));
    v = join(v, moved<0x114, 0xf>(v, none));
    v = join(v, moved<0x118, 0xf>(v, none));
    v = join(v, moved<0x142, 0xa>(v, none));     // row_bcast 15 to rows 1 and 3
    v = join(v, moved<0x143, 0xc>(v, none));     // row_bcast 31 to rows 2 and 3
    return from_lane(v, 63);
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v)
{
    return wave_reduce(v, static_cast<T>(0), [](T a, T b) { return a + b; });
}

template <typename T>
__device__ __forceinline__ T wave_max(T v)       // no NaN
{
    return wave_reduce(v, static_cast<T>(-INFINITY), [](T a, T b) { return a > b ? a : b; });
}

struct RouteArgs {
    const void* logits;
    const float* bias;
    float* w;
    int* ids;
    float scale;
    int T, E, k, groups, top_groups, score, renorm, bf16;
};

// exp(l - top) in 64 bits; 0 for an expert that is out
__device__ __forceinline__ double lift(float l, float top) { return l == -INFINITY ? 0.0 : exp(static_cast<double>(l) - top); }
__device__ __forceinline__ double sigmoid64(float l) { return l == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-static_cast<double>(l))); }

// A wave a token, lane l the experts l, l + 64, ...  Rank is what experts are chosen by:
// the logit, or (SCORED) the choice value in 64 bits, in which two experts' order does not
// hang on a rounding.  Bound by its chain of steps, k reductions over the wave among them:
// 8192 tokens, 8 of 256 experts in 4 of 8 groups, sigmoid and bias: 25 us (8.4 MB); 33
// tokens 3.5.
template <int V, bool SCORED>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void k_route(const RouteArgs p)
{
    typedef std::conditional_t<SCORED, double, float> Rank;
    __shared__ Rank shown[SCORED ? ROUTE_WAVES : 1][SCORED ? 64 * V : 1];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, t = blockIdx.x * ROUTE_WAVES + w;
    if (t >= p.T)
        return;
    const size_t row = static_cast<size_t>(t) * p.E;
    float l[V];
    Rank rank[V];
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + 64 * v;
        l[v] = e < p.E ? logit_at(p.logits, p.bf16, row + e) : -INFINITY;
        top = fmaxf(top, l[v]);
    }
    top = wave_max(top);
    double total = 0.0;              // of the softmax, where it is needed
    if (p.score == SCORE_SOFTMAX && (SCORED || !p.renorm)) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            total += lift(l[v], top);
        total = wave_sum(total);
    }
    if constexpr (SCORED) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane + 64 * v;
            const double s = p.score == SCORE_SOFTMAX ? lift(l[v], top) / total : sigmoid64(l[v]);
            const double c = p.bias && e < p.E ? s + p.bias[e] : s;
            rank[v] = l[v] == -INFINITY || c != c ? -INFINITY : c;
        }
        if (p.top_groups < p.groups) {
            const int size = p.E / p.groups;
#pragma unroll
            for (int v = 0; v < V; ++v)
                shown[w][lane + 64 * v] = rank[v];
            wave_sync();
            double score = -INFINITY;
            if (lane < p.groups) {
                double a = -INFINITY, b = -INFINITY;
                for (int i = 0; i < size; ++i) {
                    const double c = shown[w][lane * size + i];
                    b = c > a ? a : c > b ? c : b;
                    a = c > a ? c : a;
                }
                score = size > 1 ? a + b : a;
                score = score != score ? -INFINITY : score;      // +inf beside an expert that is out
            }
            int before = 0;
            for (int g = 0; g < p.groups; ++g) {
                const double o = from_lane(score, g);
                before += o > score || (o == score && g < lane);
            }
            const uint64_t kept = __ballot(lane < p.groups && before < p.top_groups);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = lane + 64 * v;
                if (e < p.E && !(kept >> (e / size) & 1))
                    rank[v] = -INFINITY;
            }
        }
        if (!p.bias)                 // the scores' order without their rounding
#pragma unroll
            for (int v = 0; v < V; ++v)
                rank[v] = rank[v] == -INFINITY ? -INFINITY : l[v];
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            rank[v] = l[v];
    }
    // the k of largest rank, one after another; lane j keeps the j-th.  Experts of one v
    // come before those of the next, lanes in order: the lowest index first.
    int mine = -1;
    float logit = -INFINITY;
    for (int j = 0; j < p.k; ++j) {
        Rank best = rank[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            best = rank[v] > best ? rank[v] : best;
        best = wave_max(best);
        if (best == -INFINITY)
            break;
        bool found = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint64_t hit = __ballot(rank[v] == best);
            if (!found && hit) {
                found = true;
                const int at = __builtin_ctzll(hit);
                const float its = from_lane(l[v], at);
                if (lane == j) {
                    mine = at + 64 * v;
                    logit = its;
                }
                if (lane == at)
                    rank[v] = -INFINITY;
            }
        }
    }
    double s;
    if (p.score == SCORE_SIGMOID)
        s = sigmoid64(logit);
    else if (p.renorm)
        s = lift(logit, wave_max(logit));     // the chosen ones' own largest: never all 0
    else
        s = total > 0.0 ? lift(logit, top) / total : 0.0;
    if (p.renorm) {
        const double sum = wave_sum(s);
        s = sum > 0.0 ? s / sum : 0.0;
    }
    if (lane < p.k) {
        p.w[static_cast<size_t>(t) * p.k + lane] = static_cast<float>(s * p.scale);
        p.ids[static_cast<size_t>(t) * p.k + lane] = mine;
    }
}

struct RouteBwdArgs {
    const float* dw;
    const void* logits;
    const int* ids;
    void* dlogits;
    float scale;
    int T, E, k, score, renorm, bf16;
};

// A wave a token.  Lane j has the j-th chosen expert and finds the derivative with
// respect to its logit; the softmax's own sum over all experts follows where
// the weights are not renormalised.  8192 tokens, 8 of 256: 13 us (16.8 MB).
template <int V>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void k_route_bwd(const RouteBwdArgs p)
{
    const int lane = threadIdx.x & 63, t = blockIdx.x * ROUTE_WAVES + (threadIdx.x >> 6);
    if (t >= p.T)
        return;
    const size_t row = static_cast<size_t>(t) * p.E;
    int id = -1;
    double dw = 0.0;
    float logit = -INFINITY;
    if (lane < p.k) {
        const int i = p.ids[static_cast<size_t>(t) * p.k + lane];
        if (static_cast<uint32_t>(i) < static_cast<uint32_t>(p.E)) {
            id = i;
            logit = logit_at(p.logits, p.bf16, row + i);
            dw = static_cast<double>(p.dw[static_cast<size_t>(t) * p.k + lane]) * p.scale;
        }
    }
    // d l_e = f_e (own_e - c): own_e what the chosen one's weight gives
    double own = 0.0, c = 0.0, total = 1.0;
    float top = 0.0f;
    const bool all = p.score == SCORE_SOFTMAX && !p.renorm;
    float l[V];
    if (all) {
        top = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane + 64 * v;
            l[v] = e < p.E ? logit_at(p.logits, p.bf16, row + e) : -INFINITY;
            top = fmaxf(top, l[v]);
        }
        top = wave_max(top);
        total = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            total += lift(l[v], top);
        total = wave_sum(total);
        const double s = total > 0.0 ? lift(logit, top) / total : 0.0;
        own = s * dw;
        c = wave_sum(own);
    } else if (p.score == SCORE_SOFTMAX) {
        const double e = lift(logit, wave_max(logit)), sum = wave_sum(e), s = sum > 0.0 ? e / sum : 0.0;
        const double mean = wave_sum(s * dw);
        own = s * (dw - mean);
    } else {
        const double s = sigmoid64(logit), rest = logit == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(static_cast<double>(logit)));
        if (p.renorm) {
            const double sum = wave_sum(s), inv = sum > 0.0 ? 1.0 / sum : 0.0;
            const double mean = wave_sum(s * inv * dw);
            own = s * inv * rest * (dw - mean);
        } else {
            own = s * rest * dw;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + 64 * v;
        double d = 0.0;
        for (int j = 0; j < p.k; ++j) {
            const int at = from_lane(id, j);
            const double o = from_lane(own, j);
            d += at == e ? o : 0.0;
        }
        if (all)
            d -= total > 0.0 ? lift(l[v], top) / total * c : 0.0;
        if (e < p.E) {
            const float f = static_cast<float>(d);
            if (p.bf16)
                static_cast<uint16_t*>(p.dlogits)[row + e] = static_cast<uint16_t>(f32_to_bf16(f));
            else
                static_cast<float*>(p.dlogits)[row + e] = f;
        }
    }
}

// ---------------------------------------------------------------------------
// the weighted sum
// ---------------------------------------------------------------------------
struct CombineArgs {
    const void* y;
    const float* w;
    const uint16_t* residual;
    uint16_t* out;
    int k, N, per;           // pieces of eight columns a row
    size_t pieces;
};

// Eight columns of a token a thread, the loads of up to JB pairs at a time; bound by
// its bytes.  What the loads depend on (Y32, rows of whole pieces, JB) is known to the
// compiler, and pairs past the last are read as the last again: a branch between the
// loads would make each wait for the one before.  8192 x 8 x 2048, 335 MB: 74 us, 4.5 TB/s.
template <bool Y32, bool WHOLE, int JB>
__global__ __launch_bounds__(256) void k_combine(const CombineArgs p)
{
    const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
    if (i >= p.pieces)
        return;
    const size_t t = i / p.per;
    const int col = static_cast<int>(i % p.per) * 8, valid = WHOLE ? 8 : p.N - col;
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s[e] = 0.0f;
    if (p.residual)
        get_values(p.residual, 0, t * p.N + col, valid, s);
    const size_t y = t * p.k * p.N + col;
    for (int j0 = 0; j0 < p.k; j0 += JB) {
        float v[JB][8], f[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int at = j0 + j < p.k ? j0 + j : p.k - 1;
            get_values(p.y, Y32, y + static_cast<size_t>(at) * p.N, valid, v[j]);
            f[j] = p.w ? p.w[t * p.k + at] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < JB; ++j)
            if (j0 + j < p.k)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] = fmaf(f[j], v[j][e], s[e]);
    }
    put_values(p.out, 0, t * p.N + col, valid, s);
}

struct CombineBwdArgs {
    const uint16_t* dout;
    const void* y;
    const float* w;
    uint16_t* dy;
    float* dw;
    int k, N;
};

// A workgroup a token, 2048 columns a round; the sums of up to JB pairs at a time, loads
// as above.  8192 x 8 x 2048, 570 MB: 89 us, 6.4 TB/s (y was read just before:
// some of it comes from the 256 MB cache).
template <bool Y32, bool WHOLE, int JB>
__global__ __launch_bounds__(256) void k_combine_bwd(const CombineBwdArgs p)
{
    __shared__ float red[4][JB];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t t = blockIdx.x;
    const uint16_t* dout = p.dout + t * p.N;
    for (int j0 = 0; j0 < p.k; j0 += JB) {
        float sum[JB], f[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            sum[j] = 0.0f;
            f[j] = p.w[t * p.k + (j0 + j < p.k ? j0 + j : p.k - 1)];
        }
        for (int col = threadIdx.x * 8; col < p.N; col += 2048) {
            const int valid = WHOLE ? 8 : p.N - col;
            float d[8];
            get_values(dout, 0, col, valid, d);
            if (p.dw) {
                float v[JB][8];
#pragma unroll
                for (int j = 0; j < JB; ++j)
                    get_values(p.y, Y32, (t * p.k + (j0 + j < p.k ? j0 + j : p.k - 1)) * p.N + col, valid, v[j]);
#pragma unroll
                for (int j = 0; j < JB; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum[j] = fmaf(d[e], v[j][e], sum[j]);
            }
            if (p.dy)
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    if (j0 + j >= p.k)
                        break;
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] = f[j] * d[e];
                    put_values(p.dy, 0, (t * p.k + j0 + j) * p.N + col, valid, o);
                }
        }
        if (!p.dw)
            continue;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const float s = wave_sum(sum[j]);
            if (lane == 0)
                red[wave][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < JB && j0 + static_cast<int>(threadIdx.x) < p.k)
            p.dw[t * p.k + j0 + threadIdx.x] = red[0][threadIdx.x] + red[1][threadIdx.x] + red[2][threadIdx.x] + red[3][threadIdx.x];
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int64_t GIB1 = static_cast<int64_t>(1) << 30;

bool route_ok(int64_t T, int64_t E, int64_t k, int score)
{
    return T >= 0 && T <= MAX_T && E >= 1 && E <= MAX_EXPERTS && k >= 1 && k <= MAX_K && k <= E && T * k <= MAX_T &&
           (score == SCORE_SOFTMAX || score == SCORE_SIGMOID);
}

bool combine_ok(int64_t T, int64_t k, int64_t N)
{
    return T >= 0 && T <= MAX_T && k >= 1 && k <= MAX_T && T * k <= MAX_T && N >= 0 && N < GIB1 && (T == 0 || N < GIB1 / (T * k));
}

// Calls f with the form of a weighted sum: fp32 or not, rows of whole pieces or not, how
// many pairs at a time.
template <typename F>
void by_form(bool y32, int64_t N, int64_t k, F&& f)
{
    auto pairs = [&](auto a, auto b) {
        if (k == 1) f(a, b, std::integral_constant<int, 1>{});
        else if (k == 2) f(a, b, std::integral_constant<int, 2>{});
        else if (k <= 4) f(a, b, std::integral_constant<int, 4>{});
        else f(a, b, std::integral_constant<int, 8>{});
    };
    auto rows = [&](auto a) {
        if (N % 8 == 0) pairs(a, std::true_type{});
        else pairs(a, std::false_type{});
    };
    if (y32) rows(std::true_type{});
    else rows(std::false_type{});
}

template <bool SCORED>
void launch_route(const RouteArgs& a, hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.T + ROUTE_WAVES - 1) / ROUTE_WAVES)), block(64 * ROUTE_WAVES);
#define ROUTE(V_) hipLaunchKernelGGL((k_route<V_, SCORED>), grid, block, 0, stream, a)
    if (a.E <= 64) ROUTE(1);
    else if (a.E <= 128) ROUTE(2);
    else if (a.E <= 256) ROUTE(4);
    else if (a.E <= 512) ROUTE(8);
    else ROUTE(16);
#undef ROUTE
}

}  // namespace

extern "C" {

any4_status any4_route(const void* logits, int logits_bf16, const float* bias, float* w, int32_t* ids, any4_score score, int renorm,
                       float scale, int64_t T, int64_t E, int64_t k, int64_t groups, int64_t top_groups, hipStream_t stream)
{
    if (!route_ok(T, E, k, score) || groups < 1 || groups > MAX_GROUPS || E % groups || top_groups < 1 || top_groups > groups ||
        k > top_groups * (E / groups))
        return ANY4_E_SHAPE;
    if (T == 0)
        return ANY4_OK;
    if (!logits || !w || !ids)
        return ANY4_E_NULL;
    if (!is_aligned(logits, logits_bf16 ? 2 : 4) || !is_aligned(bias, 4) || !is_aligned(w, 4) || !is_aligned(ids, 4))
        return ANY4_E_ALIGN;
    (void)hipGetLastError();
    const RouteArgs a{logits, bias, w, ids, scale, static_cast<int>(T), static_cast<int>(E), static_cast<int>(k), static_cast<int>(groups),
                      static_cast<int>(top_groups), static_cast<int>(score), renorm != 0, logits_bf16 != 0};
    if (bias || top_groups < groups)
        launch_route<true>(a, stream);
    else
        launch_route<false>(a, stream);
    return launch_status();
}

any4_status any4_route_backward(const float* dw, const void* logits, int logits_bf16, const int32_t* ids, void* dlogits, any4_score score,
                                int renorm, float scale, int64_t T, int64_t E, int64_t k, hipStream_t stream)
{
    if (!route_ok(T, E, k, score))
        return ANY4_E_SHAPE;
    if (T == 0)
        return ANY4_OK;
    if (!dw || !logits || !ids || !dlogits)
        return ANY4_E_NULL;
    const size_t size = logits_bf16 ? 2 : 4;
    if (!is_aligned(dw, 4) || !is_aligned(logits, size) || !is_aligned(ids, 4) || !is_aligned(dlogits, size))
        return ANY4_E_ALIGN;
    (void)hipGetLastError();
    const RouteBwdArgs a{dw, logits, ids, dlogits, scale, static_cast<int>(T), static_cast<int>(E), static_cast<int>(k),
                         static_cast<int>(score), renorm != 0, logits_bf16 != 0};
    const dim3 grid(static_cast<unsigned>((T + ROUTE_WAVES - 1) / ROUTE_WAVES)), block(64 * ROUTE_WAVES);
#define ROUTE(V_) hipLaunchKernelGGL((k_route_bwd<V_>), grid, block, 0, stream, a)
    if (E <= 64) ROUTE(1);
    else if (E <= 128) ROUTE(2);
    else if (E <= 256) ROUTE(4);
    else if (E <= 512) ROUTE(8);
    else ROUTE(16);
#undef ROUTE
    return launch_status();
}

any4_status any4_combine(const void* y, int y_f32, const float* w, const uint16_t* residual, uint16_t* out, int64_t T, int64_t k, int64_t N,
                         hipStream_t stream)
{
    if (!combine_ok(T, k, N))
        return ANY4_E_SHAPE;
    if (T == 0 || N == 0)
        return ANY4_OK;
    if (!y || !out)
        return ANY4_E_NULL;
    if (!is_aligned(y, y_f32 ? 4 : 2) || !is_aligned(w, 4) || !is_aligned(residual, 2) || !is_aligned(out, 2))
        return ANY4_E_ALIGN;
    (void)hipGetLastError();
    const int per = static_cast<int>((N + 7) / 8);
    const size_t pieces = static_cast<size_t>(T) * per;
    const CombineArgs a{y, w, residual, out, static_cast<int>(k), static_cast<int>(N), per, pieces};
    const dim3 grid(static_cast<unsigned>((pieces + 255) / 256));
    by_form(y_f32 != 0, N, k, [&](auto y32, auto whole, auto jb) {
        hipLaunchKernelGGL((k_combine<decltype(y32)::value, decltype(whole)::value, decltype(jb)::value>), grid, dim3(256), 0, stream, a);
    });
    return launch_status();
}

any4_status any4_combine_backward(const uint16_t* dout, const void* y, int y_f32, const float* w, uint16_t* dy, float* dw, int64_t T, int64_t k,
                                  int64_t N, hipStream_t stream)
{
    if (!combine_ok(T, k, N))
        return ANY4_E_SHAPE;
    if (T == 0 || (!dy && !dw) || (N == 0 && !dw))
        return ANY4_OK;
    if (!w || (N > 0 && (!dout || (dw && !y))))
        return ANY4_E_NULL;
    if (!is_aligned(dout, 2) || !is_aligned(y, y_f32 ? 4 : 2) || !is_aligned(w, 4) || !is_aligned(dy, 2) || !is_aligned(dw, 4))
        return ANY4_E_ALIGN;
    (void)hipGetLastError();
    const CombineBwdArgs a{dout, y, w, dy, dw, static_cast<int>(k), static_cast<int>(N)};
    by_form(y_f32 != 0, N, k, [&](auto y32, auto whole, auto jb) {
        hipLaunchKernelGGL((k_combine_bwd<decltype(y32)::value, decltype(whole)::value, decltype(jb)::value>), dim3(static_cast<unsigned>(T)),
                           dim3(256), 0, stream, a);
    });
    return launch_status();
}

}  // extern "C"
