// Expert routing: the K best of E scores for every token, their weights, and
// the weights' gradient.
//
// L lanes share a token; lane l of a group of `group_lanes` holds the group's
// experts 4 (l + group_lanes i) .. + 3.  The choice runs on 64-bit keys: the
// score (in 64 bits; the logit itself where its order is the score's) with the
// low ten bits of its significand replaced by the expert's index, reversed
// where that makes the lower index the larger key.  So keys never tie, equal
// scores go to the lower index, and scores further apart than 2^-42 of their
// size are told apart.  Each lane runs its experts through a sorted list of
// the KP largest keys, two instructions per level (max and min), and the
// lanes' lists are merged pairwise: the larger of a[i] and b[KP - 1 - i] are
// the KP largest of both, in bitonic order.
#include "rows_impl.h"

namespace rc {
namespace {

constexpr int kRouteThreads = 256;
constexpr double kNone = -__builtin_inf();
constexpr double kHuge = 1e300;

// v_max_f64 / v_min_f64 as they are: keys are never NaN, so the quieting that
// fmax would add has nothing to do.
__device__ __forceinline__ double max64(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double min64(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// Key of a score: kNone stays; the index takes the low ten bits.
__device__ __forceinline__ double key_of(double score, int expert) {
    const double v = score + 0.0;  // one zero
    if (v == kNone) return kNone;
    const uint64_t u = __builtin_bit_cast(uint64_t, v < kHuge ? v : kHuge);
    const uint64_t index = (u >> 63) ? (uint64_t)expert : (uint64_t)(RC_MAX_EXPERTS - 1 - expert);
    return __builtin_bit_cast(double, (u & ~uint64_t(RC_MAX_EXPERTS - 1)) | index);
}
__device__ __forceinline__ int expert_of(double key) {
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    const int low = (int)(u & (RC_MAX_EXPERTS - 1));
    return (u >> 63) ? low : RC_MAX_EXPERTS - 1 - low;
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

template <int L, class V>
__device__ __forceinline__ V sum_lanes(V v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor(v, o);
    return v;
}
template <int L, class V>
__device__ __forceinline__ V max_lanes(V v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        const V w = __shfl_xor(v, o);
        v = w > v ? w : v;
    }
    return v;
}

// The rank and row of this lane's token; false past the last.
template <int L>
__device__ __forceinline__ bool token_of(const RankSpans& tokens, int* rank, int32_t* row) {
    const int64_t t = group_index() * (kRouteThreads / L) + threadIdx.x / L;
    if (t >= tokens.total()) return false;
    *rank = rank_of(tokens, (int32_t)t, row);
    return true;
}

template <class T, int L, int V, int KP>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
    using E = typename T::E;
    int rank;
    int32_t row;
    // lanes past the last token repeat it, so that all take part in the exchanges
    const bool live = token_of<L>(a.tokens, &rank, &row);
    if (!live) {
        rank = 0;
        row = -1;
    }
    const int lane = threadIdx.x & (L - 1);
    const int group = lane / a.group_lanes, part = lane - group * a.group_lanes;
    const bool in_group = group < a.groups;
    const E* logits = static_cast<const E*>(a.logits[rank]) + (int64_t)row * a.num_experts;
    const int base = group * a.group_size;

    float x[V];
#pragma unroll
    for (int j = 0; j < V; j += 4) {
        const int at = (j / 4 * a.group_lanes + part) * 4;  // within the group
        if (live && in_group && a.vec && at < a.group_size) {
            if constexpr (sizeof(E) == 4) {
                F32::unpack(*reinterpret_cast<const u32x4*>(logits + base + at), x + j);
            } else {
                const uint64_t v = *reinterpret_cast<const uint64_t*>(logits + base + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j + i] = T::load(__builtin_bit_cast(E, (uint16_t)(v >> (16 * i))));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[j + i] = live && in_group && at + i < a.group_size ? T::load(logits[base + at + i]) : -__builtin_inff();
        }
    }

    // softmax: the largest logit, and whether the row has a NaN or +inf, which
    // leaves no score that is a number
    float top = -__builtin_inff();
    bool broken = false;
    if (!a.sigmoid) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            top = x[j] > top ? x[j] : top;
            broken |= !(x[j] < __builtin_inff());
        }
        top = max_lanes<L>(top);
        broken = max_lanes<L>((int)broken) != 0;
        if (top == -__builtin_inff()) top = 0.0f;
    }
    // scores are needed where their order is not the logits'
    const bool scored = a.bias || (a.groups > 1 && a.top2);
    double total = 0.0;
    if (!a.sigmoid && (scored || !a.renormalize)) {
#pragma unroll
        for (int j = 0; j < V; ++j) total += exp((double)x[j] - (double)top);
        total = sum_lanes<L>(total);
    }
    double c[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int at = (j / 4 * a.group_lanes + part) * 4 + j % 4;
        double v = (double)x[j];
        if (scored) {
            v = a.sigmoid ? sigmoid64(v) : exp(v - (double)top) / total;
            if (a.bias && in_group && at < a.group_size) v += (double)a.bias[base + at];
        }
        const bool choosable = x[j] > -__builtin_inff() && v > kNone && !broken;  // neither is NaN
        c[j] = choosable ? (v < kHuge ? v : kHuge) : kNone;
    }

    if (a.groups > 1) {
        double first = kNone, second = kNone;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            second = max64(second, min64(first, c[j]));
            first = max64(first, c[j]);
        }
        for (int o = 1; o < a.group_lanes; o <<= 1) {
            const double f = __shfl_xor(first, o), s = __shfl_xor(second, o);
            second = max64(min64(first, f), max64(second, s));
            first = max64(first, f);
        }
        const double score = a.top2 && a.group_size > 1 ? first + second : first;
        int better = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double other = __shfl(score, (threadIdx.x & (kWave - 1) & ~(L - 1)) + g * a.group_lanes);
            better += other > score || (other == score && g < group);
        }
        if (better >= a.top_groups) {
#pragma unroll
            for (int j = 0; j < V; ++j) c[j] = kNone;
        }
    }

    double list[KP];
#pragma unroll
    for (int k = 0; k < KP; ++k) list[k] = kNone;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        double v = key_of(c[j], base + (j / 4 * a.group_lanes + part) * 4 + j % 4);
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const double low = min64(list[k], v);
            list[k] = max64(list[k], v);
            v = low;
        }
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        double m[KP];
#pragma unroll
        for (int k = 0; k < KP; ++k) m[k] = __shfl_xor(list[KP - 1 - k], o);
#pragma unroll
        for (int k = 0; k < KP; ++k) list[k] = max64(list[k], m[k]);
#pragma unroll
        for (int h = KP / 2; h > 0; h >>= 1) {
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                if (k & h) continue;
                const double hi = max64(list[k], list[k + h]);
                list[k + h] = min64(list[k], list[k + h]);
                list[k] = hi;
            }
        }
    }

    // weights: lane l takes the choices l, l + L, ...
    constexpr int kEach = (KP + L - 1) / L;
    int expert[kEach];
    double score[kEach], best = kNone, sum = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        double key = kNone;
#pragma unroll
        for (int k = 0; k < KP; ++k)
            if (k == lane + i * L && k < a.top_k) key = list[k];
        expert[i] = key == kNone ? -1 : expert_of(key);
        score[i] = expert[i] < 0 ? kNone : (double)T::load(logits[expert[i]]);
        best = score[i] > best ? score[i] : best;
    }
    // the chosen softmax scores relative to the largest chosen, or to all
    const bool relative = !a.sigmoid && a.renormalize;
    if (relative) best = max_lanes<L>(best);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (expert[i] < 0) score[i] = 0.0;
        else if (a.sigmoid) score[i] = sigmoid64(score[i]);
        else score[i] = exp(score[i] - (relative ? best : (double)top));
        sum += score[i];
    }
    if (a.renormalize) sum = sum_lanes<L>(sum);
    else sum = a.sigmoid ? 1.0 : total;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int k = lane + i * L;
        if (!live || k >= a.top_k) continue;
        const int64_t at = (int64_t)row * a.top_k + k;
        a.experts[rank][at] = expert[i];
        a.weights[rank][at] = expert[i] >= 0 && sum > 0.0 ? (float)((double)a.scale * (score[i] / sum)) : 0.0f;
    }
}

// The weights' gradient.  Each token's row of E values is put together in LDS:
// cleared (or filled with the softmax's part that every expert has), then the
// chosen experts' parts are added by the lane that owns them, in order of k.
template <class T, int L>
__global__ __launch_bounds__(kRouteThreads) void route_grad_kernel(RouteArgs a) {
    using E = typename T::E;
    extern __shared__ float lds[];
    int rank;
    int32_t row;
    const bool live = token_of<L>(a.tokens, &rank, &row);
    if (!live) {
        rank = 0;
        row = -1;
    }
    const int lane = threadIdx.x & (L - 1);
    const int64_t at = (int64_t)row * a.num_experts;
    const E* logits = static_cast<const E*>(a.logits[rank]) + at;
    float* mine = lds + (threadIdx.x / L) * ((a.num_experts + 3) & ~3);

    constexpr int kEach = (RC_MAX_TOP_K + L - 1) / L;
    int expert[kEach];
    double x[kEach], g[kEach], p[kEach];
    double best = kNone, sum = 0.0, dot = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int k = lane + i * L;
        const int64_t j = (int64_t)row * a.top_k + k;
        expert[i] = live && k < a.top_k ? a.experts[rank][j] : -1;
        const bool has = expert[i] >= 0 && expert[i] < a.num_experts;
        if (!has) expert[i] = -1;
        x[i] = has ? (double)T::load(logits[expert[i]]) : kNone;
        g[i] = has ? (double)a.scale * (double)a.d_weights[rank][j] : 0.0;
        best = x[i] > best ? x[i] : best;
    }
    const bool any = max_lanes<L>((int)(expert[0] >= 0 || expert[kEach - 1] >= 0)) != 0;
    const bool full = !a.sigmoid && !a.renormalize;  // the softmax over all experts
    float top = -__builtin_inff(), total = 0.0f;
    if (full && any && live) {
        for (int e = lane; e < a.num_experts; e += L) {
            const float v = T::load(logits[e]);
            top = v > top ? v : top;
        }
    }
    if (full) {
        top = max_lanes<L>(top);
        if (any && live)
            for (int e = lane; e < a.num_experts; e += L) total += expf(T::load(logits[e]) - top);
        total = sum_lanes<L>(total);
    }
    if (!a.sigmoid && a.renormalize) best = max_lanes<L>(best);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        p[i] = 0.0;
        if (expert[i] < 0) continue;
        p[i] = a.sigmoid ? sigmoid64(x[i]) : full ? exp(x[i] - (double)top) / (double)total : exp(x[i] - best);
        sum += p[i];
    }
    if (a.renormalize) {
        sum = sum_lanes<L>(sum);
        if (!(sum > 0.0)) sum = __builtin_inf();
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) dot += g[i] * (a.renormalize ? p[i] / sum : p[i]);
    dot = sum_lanes<L>(dot);
    double d[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (a.renormalize) d[i] = p[i] / sum * (g[i] - dot);
        else d[i] = g[i] * p[i];
        if (a.sigmoid && expert[i] >= 0) d[i] *= sigmoid64(-x[i]);
    }
    // the row
    for (int e = lane; e < a.num_experts; e += L) {
        float v = 0.0f;
        if (full && any && live) v = -(float)dot * (expf(T::load(logits[e]) - top) / total);
        mine[e] = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < RC_MAX_TOP_K; ++k) {
        if (k < a.top_k) {
            const int from = (threadIdx.x & (kWave - 1) & ~(L - 1)) + k % L;
            const int e = __shfl(expert[k / L], from);
            const float v = (float)__shfl(d[k / L], from);
            if (e >= 0 && e % L == lane) mine[e] += v;
        }
    }
    __syncthreads();
    if (!live) return;
    E* out = static_cast<E*>(a.d_logits[rank]) + at;
    if (a.vec) {
        for (int e = lane * 4; e < a.num_experts; e += L * 4) {
            if constexpr (sizeof(E) == 4) {
                *reinterpret_cast<u32x4*>(out + e) = F32::pack(mine + e);
            } else {
                uint64_t v = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v |= (uint64_t)__builtin_bit_cast(uint16_t, T::store(mine[e + i])) << (16 * i);
                *reinterpret_cast<uint64_t*>(out + e) = v;
            }
        }
    } else {
        for (int e = lane; e < a.num_experts; e += L) out[e] = T::store(mine[e]);
    }
}

int pow2_up(int v) {
    int p = 1;
    while (p < v) p *= 2;
    return p;
}

// Experts per lane, to the next multiple of four, where L lanes share a token.
int per_lane(const RouteArgs& a, int L) {
    const int lanes = L / pow2_up(a.groups);
    return lanes ? (a.group_size + 4 * lanes - 1) / (4 * lanes) * 4 : 1 << 30;
}

template <class T, int L, int V>
int run_route(RouteArgs a, hipStream_t s) {
    a.group_lanes = L / pow2_up(a.groups);
    constexpr int per = kRouteThreads / L;
    const dim3 grid = grid_of(((int64_t)a.tokens.total() + per - 1) / per);
    auto fn = a.top_k <= 4 ? route_kernel<T, L, V, 4> : a.top_k <= 8 ? route_kernel<T, L, V, 8> : route_kernel<T, L, V, 16>;
    hipLaunchKernelGGL(fn, grid, dim3(kRouteThreads), 0, s, a);
    return hipGetLastError();
}

template <class T>
int pick_route(const RouteArgs& a, hipStream_t s) {
    const int few = per_lane(a, 8), many = per_lane(a, 64);
    if (few <= 8) return run_route<T, 8, 8>(a, s);
    if (few <= 32) return run_route<T, 8, 32>(a, s);
    if (many <= 8) return run_route<T, 64, 8>(a, s);
    return run_route<T, 64, 32>(a, s);
}

template <class T>
int pick_route_grad(const RouteArgs& a, hipStream_t s) {
    const int row = ((a.num_experts + 3) & ~3) * 4;
    if (a.num_experts <= 256) {
        constexpr int per = kRouteThreads / 8;
        hipLaunchKernelGGL((route_grad_kernel<T, 8>), grid_of(((int64_t)a.tokens.total() + per - 1) / per),
                           dim3(kRouteThreads), per * row, s, a);
    } else {
        constexpr int per = kRouteThreads / 64;
        hipLaunchKernelGGL((route_grad_kernel<T, 64>), grid_of(((int64_t)a.tokens.total() + per - 1) / per),
                           dim3(kRouteThreads), per * row, s, a);
    }
    return hipGetLastError();
}

}  // namespace

int launch_route(const RouteArgs& a, int dtype, void* stream) {
    return RC_BY_TYPE(pick_route, a, static_cast<hipStream_t>(stream));
}
int launch_route_grad(const RouteArgs& a, int dtype, void* stream) {
    return RC_BY_TYPE(pick_route_grad, a, static_cast<hipStream_t>(stream));
}

}  // namespace rc
