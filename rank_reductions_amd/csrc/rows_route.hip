// Expert routing: the K best of E scores for every token, their weights, and
// the weights' gradient.
//
// L lanes share a token; lane l of a group of `group_lanes` holds the group's
// experts 4 (l + group_lanes i) .. + 3.  The choice runs on 64-bit keys: the
// score with the low ten bits of its significand replaced by the expert's
// index, reversed where that makes the lower index the larger key.  So keys
// never tie and equal scores go to the lower index.  Each lane sorts its
// experts' keys KP at a time, a comparator being two instructions (max and
// min), and merges them: the larger of a[i] and b[KP - 1 - i] are the KP
// largest of both, in bitonic order.  The lanes' lists are merged likewise.
// Sorting takes 9 instructions per expert for KP = 8; running each expert
// through a sorted list takes 16.
//
// The choice has to be that of the values in 64 bits.  Without a bias the
// logits' order is the scores', and the keys are made from the logits, exactly.
// But logits that share a score in 64 bits (kind_of below) are told apart by
// their index: once some are seen among the chosen, the scores are compared.
// With a bias the scores are computed in float32, with a bound on their error;
// where two that decide something are closer than that, the scores that could
// matter - a handful - are computed again in 64 bits and decide, to their last
// bit.  A double exp and division for every expert cost more than all the rest:
// 131072 tokens of 256 experts in 8 groups with a bias, eight chosen, took 151 us
// that way and take 67 (without bias or groups 35).
//
// Bound by instruction issue where there are many tokens: that case issues
// 1760 vector instructions a wave of eight tokens, 48 us of the 67 if none ever
// waited; its 143 MB are 21 us at the 6.7 TB/s of this library's copies.
#include "rows_impl.h"

namespace rc {
namespace {

constexpr int kRouteThreads = 256;
constexpr double kNone = -__builtin_inf();
constexpr float kNone32 = -__builtin_inff();
constexpr double kNoKey = -1e300;  // keys of what cannot be chosen lie below
constexpr float kU = 0x1p-24f;
constexpr float kHuge = 3.4028234663852886e38f;

// v_max / v_min as they are: no operand is ever NaN, so the quieting that fmax
// and fmin would add has nothing to do.
__device__ __forceinline__ double max_of(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double min_of(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float max_of(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float min_of(float a, float b) {
    float r;
    asm("v_min_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// Key of a score that is not NaN or +inf, for `reversed` = RC_MAX_EXPERTS - 1
// - expert.
__device__ __forceinline__ double key_of(double score, uint32_t reversed) {
    const uint64_t u = __builtin_bit_cast(uint64_t, score);
    const uint32_t hi = score == kNone ? 0xffe00000u : (uint32_t)(u >> 32);
    const uint32_t index = reversed ^ ((uint32_t)((int32_t)hi >> 31) & (RC_MAX_EXPERTS - 1));
    const uint32_t lo = ((uint32_t)u & ~(uint32_t)(RC_MAX_EXPERTS - 1)) | index;
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double key_of(float score, uint32_t reversed) {
    // a float's double has 29 zeros at its end
    const uint64_t u = __builtin_bit_cast(uint64_t, max_of((double)score, __builtin_bit_cast(double, 0xffe0000000000000ull)));
    const uint32_t hi = (uint32_t)(u >> 32);
    const uint32_t lo = ((reversed ^ (uint32_t)((int32_t)hi >> 31)) & (RC_MAX_EXPERTS - 1)) | (uint32_t)u;
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int expert_of(double key) {
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    const int low = (int)(u & (RC_MAX_EXPERTS - 1));
    return (u >> 63) ? low : RC_MAX_EXPERTS - 1 - low;
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// exp(t) for t <= 0 within 2^-36 of itself, 0 where a double's would be near
// its end: 2^n times the series of r = t - n ln 2, |r| < 0.347, up to r^9 (the
// next term is 2^-37, the roundings 2^-50).
__device__ __forceinline__ double exp_of(double t) {
    t = max_of(t, -1000.0);
    const double n = __builtin_rint(t * 1.4426950408889634), r = __builtin_fma(n, -0.69314718055994531, t);
    double s = 1.0 / 362880;
    s = __builtin_fma(s, r, 1.0 / 40320);
    s = __builtin_fma(s, r, 1.0 / 5040);
    s = __builtin_fma(s, r, 1.0 / 720);
    s = __builtin_fma(s, r, 1.0 / 120);
    s = __builtin_fma(s, r, 1.0 / 24);
    s = __builtin_fma(s, r, 1.0 / 6);
    s = __builtin_fma(s, r, 0.5);
    s = __builtin_fma(s, r, 1.0);
    s = __builtin_fma(s, r, 1.0);
    return __builtin_amdgcn_ldexp(s, (int)n);
}

// exp(x) for x <= 0 within (1.25 |x| + 2) kU of itself, and the sigmoid within
// 5 kU: the exponent's rounding and the constant's, one step of v_exp and of
// v_rcp, and one sum.
constexpr float kLog2e = 1.44269504088896341f;
constexpr double kOffLog2e = (1.44269504088896341 - (double)kLog2e) * 0.69314718055994531;
__device__ __forceinline__ float exp32(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float sigmoid32(float x) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e)); }

// The value that lane (l ^ O) holds, in a step of a butterfly: from O = 4 on,
// all lanes of the O below hold the same, so that any lane of the other half
// will do.
template <int O>
__device__ __forceinline__ uint32_t across(uint32_t v) {
    if constexpr (O == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true);       // quad_perm 1 0 3 2
    else if constexpr (O == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true);  // quad_perm 2 3 0 1
    else if constexpr (O == 4) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true); // row_half_mirror
    else if constexpr (O == 8) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true); // row_mirror
    else return (uint32_t)__shfl_xor((int)v, O);
}
template <int O>
__device__ __forceinline__ float across(float v) {
    return __builtin_bit_cast(float, across<O>(__builtin_bit_cast(uint32_t, v)));
}
template <int O>
__device__ __forceinline__ double across(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = across<O>((uint32_t)u), hi = across<O>((uint32_t)(u >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int O>
__device__ __forceinline__ int across(int v) {
    return (int)across<O>((uint32_t)v);
}

// f(mine, other's) over the L lanes of a token, a step of the butterfly at a time.
template <int L, int O = 1, class V, class F>
__device__ __forceinline__ V all_lanes(V v, F f) {
    if constexpr (O < L) return all_lanes<L, O * 2>(f(v, across<O>(v)), f);
    else return v;
}
template <int L, class V>
__device__ __forceinline__ V sum_lanes(V v) {
    return all_lanes<L>(v, [](V a, V b) { return a + b; });
}
template <int L, class V>
__device__ __forceinline__ V max_lanes(V v) {
    return all_lanes<L>(v, [](V a, V b) { return a > b ? a : b; });
}

// The rank and row of this lane's token; false past the last.
template <int L>
__device__ __forceinline__ bool token_of(const RankSpans& tokens, int* rank, int32_t* row) {
    const int64_t t = group_index() * (kRouteThreads / L) + threadIdx.x / L;
    if (t >= tokens.total()) return false;
    *rank = rank_of(tokens, (int32_t)t, row);
    return true;
}

// Where a lane's V experts lie: expert base + at(j) for j < V, at(j) < size.
struct Part {
    int group, base, size, lanes, part;
    bool in_group;
    __device__ __forceinline__ int at(int j) const { return (j / 4 * lanes + part) * 4 + j % 4; }
};

__device__ __forceinline__ void order(double& hi, double& lo) {
    const double m = max_of(hi, lo);
    lo = min_of(hi, lo);
    hi = m;
}

// Sorts N values (a power of two), the largest first: Batcher's odd-even merge
// sort, 5, 19 and 63 comparators for 4, 8 and 16.
template <int N>
__device__ __forceinline__ void sort_values(double* v) {
#pragma unroll
    for (int p = 1; p < N; p *= 2) {
#pragma unroll
        for (int k = p; k >= 1; k /= 2) {
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k) {
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(v[i + j], v[i + j + k]);
            }
        }
    }
}

// list (sorted) becomes the KP largest of it and v; returns the one left out.
template <int KP>
__device__ __forceinline__ double insert(double* list, double v) {
#pragma unroll
    for (int k = 0; k < KP; ++k) order(list[k], v);
    return v;
}

// list (sorted) becomes the KP largest of it and of m (sorted), sorted.
template <int KP>
__device__ __forceinline__ void merge_into(double* list, const double* m) {
#pragma unroll
    for (int k = 0; k < KP; ++k) list[k] = max_of(list[k], m[KP - 1 - k]);
#pragma unroll
    for (int h = KP / 2; h > 0; h >>= 1) {
#pragma unroll
        for (int k = 0; k < KP; ++k)
            if (!(k & h)) order(list[k], list[k + h]);
    }
}

// Merges the lanes' sorted lists: all L lanes end with the KP largest.
template <int L, int KP, int O = 1>
__device__ __forceinline__ void merge_lists(double* list) {
    if constexpr (O < L) {
        double m[KP];
#pragma unroll
        for (int k = 0; k < KP; ++k) m[k] = across<O>(list[k]);
        merge_into<KP>(list, m);
        merge_lists<L, KP, O * 2>(list);
    }
}

// Scores in full, each with its expert, for the few that are computed in 64 bits.
__device__ __forceinline__ void order(double& hi, int& hi_expert, double& lo, int& lo_expert) {
    const bool swap = lo > hi || (lo == hi && lo_expert < hi_expert);
    const double s = swap ? lo : hi, t = swap ? hi : lo;
    const int e = swap ? lo_expert : hi_expert, f = swap ? hi_expert : lo_expert;
    hi = s;
    lo = t;
    hi_expert = e;
    lo_expert = f;
}
template <int L, int KP, int O = 1>
__device__ __forceinline__ void merge_scored(double* score, int* expert) {
    if constexpr (O < L) {
        double m[KP];
        int e[KP];
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            m[k] = across<O>(score[k]);
            e[k] = across<O>(expert[k]);
        }
#pragma unroll
        for (int k = 0; k < KP; ++k) order(score[k], expert[k], m[KP - 1 - k], e[KP - 1 - k]);
#pragma unroll
        for (int h = KP / 2; h > 0; h >>= 1) {
#pragma unroll
            for (int k = 0; k < KP; ++k)
                if (!(k & h)) order(score[k], expert[k], score[k + h], expert[k + h]);
        }
        merge_scored<L, KP, O * 2>(score, expert);
    }
}

// The largest two of what has been seen, with c.
__device__ __forceinline__ void best_two(float& first, float& second, float c) {
    second = __builtin_amdgcn_fmed3f(first, second, c);
    first = max_of(first, c);
}
__device__ __forceinline__ void best_two(double& first, double& second, double c) {
    second = max_of(second, min_of(first, c));
    first = max_of(first, c);
}

// The value of the lane mirrored within four.
__device__ __forceinline__ float quad_mirror(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x1b, 0xf, 0xf, true));
}
__device__ __forceinline__ double quad_mirror(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, 0x1b, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), 0x1b, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Whether the lane's group is among the top_groups best, by the two best
// scores of each lane's experts (joined over the lanes of a group here); sets
// *doubt where another group's score is within margin.
template <int L, class C>
__device__ __forceinline__ bool group_kept(const RouteArgs& a, const Part& p, C& first, C& second, C margin, bool* doubt) {
    for (int o = 1; o < p.lanes; o <<= 1) {
        const C f = __shfl_xor(first, o), s = __shfl_xor(second, o);
        second = max_of(min_of(first, f), max_of(second, s));
        first = max_of(first, f);
    }
    C of_group = first;
    if (a.top2 && a.group_size > 1) {
        of_group = first + second;
        // float32's largest where the sum lies beyond it: not an infinity, which is
        // apart from no other and, below, is a group with nothing to add
        if constexpr (sizeof(C) == 4) of_group = second > kNone32 ? __builtin_amdgcn_fmed3f(of_group, -kHuge, kHuge) : kNone32;
    }
    int better = 0;
    auto against = [&](C other, bool lower) {
        better += other > of_group || (other == of_group && lower);
        const C apart = other > of_group ? other - of_group : of_group - other;  // NaN: both kNone
        *doubt |= apart <= margin;
    };
    const int lane = threadIdx.x & (L - 1);
    if constexpr (L == 8) {
        // the token's seven other lanes, of those the ones that stand for a group in this lane's place
        const C other[8] = {of_group, across<1>(of_group), across<2>(of_group), quad_mirror(of_group),
                            quad_mirror(across<4>(of_group)), across<2>(across<4>(of_group)),
                            across<1>(across<4>(of_group)), across<4>(of_group)};
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            const int from = lane ^ k;
            if ((from & (p.lanes - 1)) == p.part && from < a.groups * p.lanes && p.in_group) against(other[k], from < lane);
        }
    } else {
        for (int g = 0; g < a.groups; ++g) {
            const C other = __shfl(of_group, (threadIdx.x & (kWave - 1) & ~(L - 1)) + g * p.lanes);
            if (g != p.group && p.in_group) against(other, g < p.group);
        }
    }
    return better < a.top_groups;
}

// Four consecutive logits.
template <class T>
__device__ __forceinline__ void load4(const typename T::E* p, float* x) {
    using E = typename T::E;
    if constexpr (sizeof(E) == 4) {
        F32::unpack(*reinterpret_cast<const u32x4*>(p), x);
    } else {
        const uint64_t v = *reinterpret_cast<const uint64_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = T::load(__builtin_bit_cast(E, (uint16_t)(v >> (16 * i))));
    }
}

// Where piece q (four logits) of the wave's token t lies in the wave's LDS:
// turned within eight pieces by the piece and the token, so that lanes that
// read pieces eight apart, of eight tokens, meet all banks.
__device__ __forceinline__ int staged_at(int t, int q, int pieces) { return t * pieces + (q ^ (((q >> 3) + t) & 7)); }

// With more than eight choices, 168 registers, a few of them spilled, for three
// waves per SIMD: without the bound most variants take 172 to 175, for two
// (131072 tokens, ten chosen of 512 experts: 301 us with it, 386 without; of 32:
// 29 and 37).
template <class T, int L, int V, int KP>
__global__ __launch_bounds__(kRouteThreads, KP == 16 ? 3 : 1) void route_kernel(RouteArgs a) {
    using E = typename T::E;
    extern __shared__ __align__(16) unsigned char route_lds[];
    int rank;
    int32_t row;
    // lanes past the last token have no experts, but take part in the exchanges
    const bool live = token_of<L>(a.tokens, &rank, &row);
    if (!live) {
        rank = 0;
        row = -1;
    }
    const int lane = threadIdx.x & (L - 1);
    Part p;
    p.lanes = a.group_lanes;
    p.group = lane / a.group_lanes;
    p.part = lane - p.group * a.group_lanes;
    p.size = a.group_size;
    p.base = p.group * a.group_size;
    p.in_group = live && p.group < a.groups;
    const E* logits = static_cast<const E*>(a.logits[rank]) + (int64_t)row * a.num_experts;

    float x[V];
    if (L == 8 && a.staged) {
        // A lane that holds a group of its own reads a line of its own in each
        // load, 64 lines a wave, which the L1 cannot keep until their next
        // quarter is read: whole rows by whole waves, then, through LDS.
        constexpr int kTokens = kWave / L;
        const int w = lane_id(), pieces = (a.num_experts / 4 + 7) & ~7;
        E* stage = reinterpret_cast<E*>(route_lds) + (threadIdx.x / kWave) * kTokens * pieces * 4;
        const uint64_t mine = live ? reinterpret_cast<uint64_t>(logits) : 0;
        float v[kTokens][4];
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)mine, t * L);
            const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(mine >> 32), t * L);
            const E* from = reinterpret_cast<const E*>((uint64_t)hi << 32 | lo);
            if (from && w < a.num_experts / 4) load4<T>(from + 4 * w, v[t]);
        }
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            if (w >= a.num_experts / 4) continue;
            E e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = T::store(v[t][i]);  // exact: it was loaded from one
            __builtin_memcpy(__builtin_assume_aligned(stage + 4 * staged_at(t, w, pieces), 4 * sizeof(E)), e, sizeof e);
        }
        wave_sync();
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const int at = p.at(j);
            if (p.in_group && at < p.size) {
                load4<T>(stage + 4 * staged_at(w / L, (p.base + at) / 4, pieces), x + j);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j + i] = kNone32;
            }
        }
    } else if (a.vec) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = kNone32;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const int at = p.at(j);
            if (p.in_group && at < p.size) load4<T>(logits + p.base + at, x + j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = p.at(j);
            x[j] = p.in_group && at < p.size ? T::load(logits[p.base + at]) : kNone32;
        }
    }

    // softmax: the largest logit, and whether the row has a NaN or +inf, which
    // leaves no score that is a number
    float top = kNone32;
    bool broken = false;
    if (!a.sigmoid) {
        // the bits of +inf and of NaNs are the largest, as signed numbers where the
        // sign is clear and as unsigned ones where it is set
        int32_t high = 0;
        uint32_t negative = 0;
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const int32_t u = __builtin_bit_cast(int32_t, x[j]), v = __builtin_bit_cast(int32_t, x[j + 1]);
            asm("v_max3_f32 %0, %0, %1, %2" : "+v"(top) : "v"(x[j]), "v"(x[j + 1]));
            high = max(high, max(u, v));
            negative = max(negative, max((uint32_t)u, (uint32_t)v));
        }
        top = max_lanes<L>(top);
        broken = max_lanes<L>((int)(high >= 0x7f800000 || negative > 0xff800000u)) != 0;
        if (top == kNone32) top = 0.0f;
    }
    // scores are needed where their order is not the logits'
    const bool scored = a.bias || (a.groups > 1 && a.top2);
    // The softmax's sum over all experts, and its reciprocal for comparing.  Where
    // the weights are divided by it (no renormalisation) it is a sum in 64 bits,
    // with what exp32 is off by its constant, a part kOffLog2e t of each; below,
    // the chosen experts' terms, the largest as a rule, become those in 64 bits.
    // Weights are off by 1.4 roundings at worst then, 0.43 rms (0.42 if rounded
    // once); with a float32 sum 10, and 1.1 to 1.6 rms.  131072 tokens of 256
    // experts: 39.9 us for 36.7; with every exponential in 64 bits 49.7.
    double total = 0.0;
    float share = 0.0f;
    auto below_top = [&](float v) { return max_of(v - top, -200.0f); };
    if (!a.sigmoid && !a.renormalize) {
        float off = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float t = below_top(x[j]), e = exp32(t);
            off = __builtin_fmaf(e, t, off);
            total += (double)e;
        }
        total = sum_lanes<L>(__builtin_fma(kOffLog2e, (double)off, total));
        share = 1.0f / (float)total;
    } else if (!a.sigmoid && scored) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum += exp32(x[j] - top);
        share = 1.0f / sum_lanes<L>(sum);
    }
    auto score32 = [&](float v) { return a.sigmoid ? sigmoid32(v) : exp32(v - top) * share; };
    // the scores of all, kNone32 for logits that are that or NaN (the kind is
    // asked once, not for each)
    auto score_all = [&](float* to) {
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < V; ++j) to[j] = x[j] > kNone32 ? sigmoid32(x[j]) : kNone32;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) to[j] = x[j] > kNone32 ? exp32(x[j] - top) * share : kNone32;
        }
    };
    // x becomes what the choice goes by: nothing above the largest float, and
    // kNone32 for a NaN (v_max takes the other operand)
    auto tidy = [&](float v) { return min_of(max_of(v, kNone32), kHuge); };
    if (a.bias) {
        float b[V];
#pragma unroll
        for (int j = 0; j < V; ++j) b[j] = 0.0f;
        if (a.bias_vec) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const int at = p.at(j);
                if (p.in_group && at < p.size) F32::unpack(*reinterpret_cast<const u32x4*>(a.bias + p.base + at), b + j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int at = p.at(j);
                if (p.in_group && at < p.size) b[j] = a.bias[p.base + at];
            }
        }
        score_all(x);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = tidy(x[j] + b[j]);
    } else if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = tidy(x[j] + 0.0f);  // one zero
    } else {
        // a NaN or +inf leaves nothing to choose from
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] += 0.0f;
    }
    // How close two values that decide something may come, of size up to
    // `size`.  The error of a score, in kU.  Sigmoid: 5.  Softmax: s <= share is
    // off by (2.25 t + 3) s for its own exponential, t = top - v and s t <= 0.4,
    // and by (V + 25) s for the sum's: its rounding, and that of exponentials
    // whose mean t is at most about log E.  Adding the bias rounds by the
    // result, a group's sum of two by as much again: the difference of two such
    // sums is off by this at most.
    const float error = a.sigmoid ? 6.0f : 2.0f + share * (float)(V + 32);
    auto near_of = [&](float size) { return 4.0f * kU * (error + 2.0f * (size < kHuge ? max_of(size, 1.0f) : 1.0f)); };

    // scores in 64 bits, from the logits and the bias
    double sum64 = 0.0;
    auto logit = [&](int j) -> double {
        const int at = p.at(j);
        return p.in_group && at < p.size ? (double)T::load(logits[p.base + at]) : kNone;
    };
    auto sum_exact = [&]() {
        if (a.sigmoid || sum64 != 0.0) return;
#pragma unroll 4
        for (int j = 0; j < V; ++j) sum64 += exp(logit(j) - (double)top);
        sum64 = sum_lanes<L>(sum64);
    };
    auto exact = [&](int j) -> double {
        const double v = logit(j);
        double c = a.sigmoid ? sigmoid64(v) : exp(v - (double)top) / sum64;
        const int at = p.at(j);
        if (a.bias && p.in_group && at < p.size) c += (double)a.bias[p.base + at];
        return c < 1e290 ? c : 1e290;
    };

    // Distinct logits u > v may share a score in 64 bits only if both are of one
    // kind.  Sigmoid: 1, from 20 on (the score's steps of 2^-53 outgrow the
    // logit's from 23 on); 2, up to 2^-16 in size; 3, from -700 down (below -709
    // scores are 0).  Softmax: 3, from 690 below the largest (scores are below
    // the normal range, or 0); 2, up to 2^-16 in size.  For others u - v is
    // 2^-40 or more (a step of a float32 beyond 2^-16), while the rounding of
    // v - top, 2^-44 below 690, and of the exponential and the quotient move
    // what is compared by less than 2^-42.
    const float high = a.sigmoid ? 20.0f : __builtin_inff(), low = a.sigmoid ? -700.0f : top - 690.0f, tiny = 0x1p-16f;
    auto kind_of = [&](float v) { return v <= low ? 3 : v >= high ? 1 : __builtin_fabsf(v) <= tiny ? 2 : 0; };
    // the least logit that may share v's score
    auto least_of = [&](float v) { return v <= low ? -kHuge : v >= high ? high : __builtin_fabsf(v) <= tiny ? -tiny : v; };

    bool kept = true;
    if (a.groups > 1) {
        float first = kNone32, second = kNone32;
        bool doubt = false;
        const bool by_score = scored && !a.bias;
        if (by_score) {
            float c[V];
            score_all(c);
#pragma unroll
            for (int j = 0; j < V; ++j) best_two(first, second, c[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) best_two(first, second, x[j]);
        }
        // the sizes of what is compared: a lane's two best, of all lanes
        float near = -1.0f;
        if (scored) {
            const float f = __builtin_fabsf(first), g = __builtin_fabsf(second);
            near = near_of(max_lanes<L>(max_of(f < kHuge ? f : 0.0f, g < kHuge ? g : 0.0f)));
        }
        kept = group_kept<L>(a, p, first, second, near, &doubt);
        if (!scored) {
            // whether the best of two groups are of one kind and differ
            const int kind = first > kNone32 ? kind_of(first) : 0;
            if (__builtin_expect(__any(kind), 0)) {
#pragma unroll 1
                for (int q = 1; q <= 3; ++q) {
                    const float most = max_lanes<L>(kind == q ? first : kNone32);
                    const float least = -max_lanes<L>(kind == q ? -first : kNone32);
                    doubt |= kind == q && most > least;
                }
            }
        }
        if (__any(doubt)) {
            // what may be among its group's two best
            const float from = scored ? (a.top2 ? second : first) - near : least_of(first);
            uint32_t close = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float c = by_score ? score32(x[j]) : x[j];
                close = close + close + (uint32_t)(x[j] > kNone32 && c >= from);
            }
            sum_exact();
            double first64 = kNone, second64 = kNone;
            while (__any(close)) {
                if (close) {
                    best_two(first64, second64, exact(V - 1 - __builtin_ctz(close)));
                    close &= close - 1;
                }
            }
            bool never = false;
            kept = group_kept<L>(a, p, first64, second64, -1.0, &never);
        }
    }
    kept &= !broken;

    auto reversed = [&](int j) { return (uint32_t)(RC_MAX_EXPERTS - 1 - (p.base + p.at(j))); };
    double list[KP], lowest;
    if constexpr (V < KP) {
#pragma unroll
        for (int k = 0; k < KP; ++k) list[k] = kNone;
#pragma unroll
        for (int j = 0; j < V; ++j) insert<KP>(list, key_of(x[j], reversed(j)));
        lowest = list[V - 1];
    } else {
#pragma unroll
        for (int j = 0; j < KP; ++j) list[j] = key_of(x[j], reversed(j));
        sort_values<KP>(list);
        lowest = list[KP - 1];
#pragma unroll
        for (int j0 = KP; j0 < V; j0 += KP) {
            double m[KP];
#pragma unroll
            for (int j = 0; j < KP; ++j) m[j] = key_of(x[j0 + j], reversed(j0 + j));
            sort_values<KP>(m);
            lowest = min_of(lowest, m[KP - 1]);
            merge_into<KP>(list, m);
        }
    }
#pragma unroll
    for (int k = 0; k < KP; ++k) list[k] = kept ? list[k] : kNone;
    float own[KP];  // the lane's best scores
#pragma unroll
    for (int k = 0; k < KP; ++k) own[k] = (float)list[k];
    merge_lists<L, KP>(list);

    if (a.bias) {
        // neighbours among the chosen, and whatever else comes close to the last of them
        const float best = __builtin_fabsf((float)list[0]);
        float last = 0.0f, least = -1.0f;  // least: the smallest distance
        bool all = true;                   // top_k could be chosen
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            if (k < a.top_k) {
                const float c = (float)list[k];
                const bool has = list[k] > kNoKey;
                if (k > 0 && has) least = k == 1 ? last - c : min_of(least, last - c);
                all &= has;
                last = has ? c : last;
            }
        }
        const float near = near_of(max_of(best, __builtin_fabsf(last)));
        bool doubt = least >= 0.0f && least <= near;
        const float from = all ? max_of(last - near, -kHuge) : -kHuge;  // -inf is never chosen
        // A lane's KP best show whether more than top_k come as close, but for the
        // lane whose KP best are all among those.
        int count = 0;
#pragma unroll
        for (int k = 0; k < KP; ++k) count += own[k] >= from;
        if (V > KP && __any(own[KP - 1] >= from)) {
            count = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) count += kept && x[j] >= from;
        }
        doubt |= all && sum_lanes<L>(count) > a.top_k;
        doubt = max_lanes<L>((int)doubt) != 0;
        if (__any(doubt)) {
            uint32_t close = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) close = close + close + (uint32_t)(x[j] >= from);
            if (!kept) close = 0;
            sum_exact();
            if (!doubt) close = 0;
            double list64[KP];
#pragma unroll
            for (int k = 0; k < KP; ++k) list64[k] = kNone;
            double past = kNone;  // the best that the lane's list has no place for
            for (uint32_t left = close; __any(left);) {
                double key = kNone;
                if (left) {
                    const int j = V - 1 - __builtin_ctz(left);
                    key = key_of(exact(j), reversed(j));
                    left &= left - 1;
                }
                past = max_of(past, insert<KP>(list64, key));
            }
            uint32_t held[KP];  // of the lane's best keys, what is the score's
#pragma unroll
            for (int k = 0; k < KP; ++k) held[k] = (uint32_t)(__builtin_bit_cast(uint64_t, list64[k]) >> 10);
            merge_lists<L, KP>(list64);
            // Keys whose scores agree to 2^-42: the bits cut off decide.  They are
            // few enough to be chosen anew, scores and experts apart; with no keys
            // before, 256 experts with a bias and no groups took 67 us for 63; a
            // bias of zeros on bf16 logits, with equal scores in every row, 73 for 114
            // (110 since).
            bool same = false;
            uint64_t before = 0;
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                if (k < a.top_k && list64[k] > kNoKey) {
                    const uint64_t u = __builtin_bit_cast(uint64_t, list64[k]) >> 10;
                    same |= u == before;
                    before = u;
                }
            }
            int as_last = (uint32_t)(__builtin_bit_cast(uint64_t, past) >> 10) == (uint32_t)before;
#pragma unroll
            for (int k = 0; k < KP; ++k) as_last += held[k] == (uint32_t)before;
            same |= sum_lanes<L>(as_last) > 1;
            same &= doubt;
#pragma unroll
            for (int k = 0; k < KP; ++k) list[k] = doubt ? list64[k] : list[k];
            if (__any(same)) {
                if (!same) close = 0;
                double score[KP];
                int of[KP];
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    score[k] = kNone;
                    of[k] = RC_MAX_EXPERTS;
                }
                while (__any(close)) {
                    double v = kNone;
                    int e = RC_MAX_EXPERTS;
                    if (close) {
                        const int j = V - 1 - __builtin_ctz(close);
                        v = exact(j);
                        e = p.base + p.at(j);
                        close &= close - 1;
                    }
#pragma unroll
                    for (int k = 0; k < KP; ++k) order(score[k], of[k], v, e);
                }
                merge_scored<L, KP>(score, of);
                // from here on only a key's index counts
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    const double key = score[k] > kNone ? __builtin_bit_cast(double, (uint64_t)(RC_MAX_EXPERTS - 1 - of[k])) : kNone;
                    list[k] = same ? key : list[k];
                }
            }
        }
    }

    // weights, in 64 bits: lane l takes the choices l, l + L, ...
    constexpr int kEach = (KP + L - 1) / L;
    int expert[kEach];
    double chosen[kEach], best = kNone, sum = 0.0;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        double key = kNone;
#pragma unroll
        for (int k = 0; k < KP; ++k)
            if (k == lane + i * L && k < a.top_k) key = list[k];
        expert[i] = key > kNoKey ? expert_of(key) : -1;
        chosen[i] = expert[i] < 0 ? kNone : (double)T::load(logits[expert[i]]);
        odd |= expert[i] >= 0 && kind_of((float)key);
    }
    if (!a.bias && __builtin_expect(__any(odd), 0)) {
        // neighbours among the chosen that may share a score, and whatever lies
        // below the last of them and may share its
        float last = 0.0f;
        bool all = true, same = false;  // all: top_k could be chosen
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            if (k >= a.top_k) continue;
            const float c = (float)list[k];
            const bool has = list[k] > kNoKey;
            same |= has && k > 0 && c < last && c >= least_of(last);
            all &= has;
            last = c;
        }
        const float from = all ? least_of(last) : -kHuge;
        bool below = all && kept && from < last && (float)lowest < last;
        if (__any(same || max_lanes<L>((int)below))) {
            // what may be chosen; from memory, since with x held for it the kernel
            // would take a tenth more registers
            uint32_t close = 0;
            below = false;
#pragma unroll 4
            for (int j = 0; j < V; ++j) {
                const int at = p.at(j);
                const float v = kept && p.in_group && at < p.size ? tidy(T::load(logits[p.base + at]) + 0.0f) : kNone32;
                below |= v >= from && v < last;
                close = close + close + (uint32_t)(v >= from);
            }
            same |= all && max_lanes<L>((int)below);
            if (!same) close = 0;
            sum_exact();
            // the next best each time, by score and then by index
            double score = __builtin_inf();
            int of = -1;
#pragma unroll 1
            for (int k = 0; k < a.top_k; ++k) {
                double next = kNone;
                int e = RC_MAX_EXPERTS;
                for (uint32_t left = close; left; left &= left - 1) {
                    const int j = V - 1 - __builtin_ctz(left), at = p.base + p.at(j);
                    const double s = exact(j);
                    const bool after = s < score || (s == score && at > of);
                    if (after && (s > next || (s == next && at < e))) {
                        next = s;
                        e = at;
                    }
                }
                score = max_lanes<L>(next);
                of = RC_MAX_EXPERTS - max_lanes<L>(next == score ? RC_MAX_EXPERTS - e : 0);
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    if (!same || k != lane + i * L) continue;
                    expert[i] = of < RC_MAX_EXPERTS ? of : -1;
                    chosen[i] = expert[i] < 0 ? kNone : (double)T::load(logits[expert[i]]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) best = chosen[i] > best ? chosen[i] : best;
    // the chosen softmax scores relative to the largest chosen, or to all
    const bool relative = !a.sigmoid && a.renormalize;
    double more = 0.0;
    if (relative) best = max_lanes<L>(best);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (expert[i] < 0) chosen[i] = 0.0;
        else if (a.sigmoid) chosen[i] = sigmoid64(chosen[i]);
        else {
            const float t = below_top((float)chosen[i]);
            chosen[i] = exp(chosen[i] - (relative ? best : (double)top));
            const double e = (double)exp32(t);  // as in the sum
            if (!relative) more += chosen[i] - __builtin_fma(kOffLog2e * e, (double)t, e);
        }
        sum += chosen[i];
    }
    if (a.renormalize) sum = sum_lanes<L>(sum);
    else if (a.sigmoid) sum = 1.0;
    else sum = total + sum_lanes<L>(more);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int k = lane + i * L;
        if (!live || k >= a.top_k) continue;
        const int64_t at = (int64_t)row * a.top_k + k;
        a.experts[rank][at] = expert[i];
        a.weights[rank][at] = expert[i] >= 0 && sum > 0.0 ? (float)((double)a.scale * (chosen[i] / sum)) : 0.0f;
    }
}

// The weights' gradient.  Each token's row of E values is put together in LDS:
// cleared (or filled with the softmax's part that every expert has), then each
// lane writes its choices' parts; where a token names an expert twice, its parts
// are added in order of k.  Bound by the writes and the 64-bit scores of the
// chosen: 131072 tokens of 256 experts, eight chosen by sigmoid, 37 us (22 at
// the 6.7 TB/s of this library's copies); two exponentials and divisions a score
// instead of one, and all adds in order of k, took 42.  The softmax over all
// experts reads the rows three times and takes two exponentials an expert: 100.
template <class T, int L, int KP>
__global__ __launch_bounds__(kRouteThreads) void route_grad_kernel(RouteArgs a) {
    using E = typename T::E;
    extern __shared__ __align__(16) float lds[];
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

    constexpr int kEach = (KP + L - 1) / L;
    int expert[kEach];
    double x[kEach], g[kEach], p[kEach], rest[kEach];
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
    // whether a token names an expert twice: each choice writes its number at its
    // expert's place, and one of two finds the other's
    bool alone = true;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (expert[i] >= 0) mine[expert[i]] = (float)(lane + i * L);
    wave_sync();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (expert[i] >= 0) alone &= mine[expert[i]] == (float)(lane + i * L);
    wave_sync();
    const bool doubled = __any(!alone);
    const int first_lane = threadIdx.x & (kWave - 1) & ~(L - 1);

    const bool full = !a.sigmoid && !a.renormalize;  // the softmax over all experts
    bool any = max_lanes<L>((int)(expert[0] >= 0 || expert[kEach - 1] >= 0)) != 0;
    float part[kEach], top = kNone32, all = 0.0f;  // all: what every expert has of the softmax's part, but for its exponential
    // f(expert, logit) for the lane's experts, and -inf behind the last
    auto each = [&](auto f) {
        if (!any || !live) return;
        for (int e = lane * 4; e < a.num_experts; e += L * 4) {
            float v[4];
            if (a.vec) load4<T>(logits + e, v);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = e + i < a.num_experts ? T::load(logits[e + i]) : kNone32;
#pragma unroll
            for (int i = 0; i < 4; ++i) f(e + i, v[i]);
        }
    };
    if (full) {
        // the largest logit's expert, the lowest of several
        int m = a.num_experts;
        bool broken = false;
        each([&](int e, float v) {
            broken |= v != v;
            m = v > top ? e : m;
            top = v > top ? v : top;
        });
        const float own = top;
        top = max_lanes<L>(top);
        m = a.num_experts - max_lanes<L>(own == top ? a.num_experts - m : 0);
        // no score is a number, and none has a part
        any &= !max_lanes<L>((int)broken) && __builtin_fabsf(top) < __builtin_inff();
        double others = 0.0;  // exponentials but the largest's, which is one
        each([&](int e, float v) { others += e == m ? 0.0 : exp_of((double)v - (double)top); });
        others = sum_lanes<L>(others);
        const double share = 1.0 / (1.0 + others);
        // With D_e the sum of the g of e's choices, d_e = s_e (D_e - sum_j s_j D_j).
        // What stands in brackets is (D_e - D_m) - sum_j s_j (D_j - D_m): near one
        // expert that outweighs the others, the sum's terms are as small as the
        // result, and nothing cancels.
        double of_m = 0.0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            p[i] = any && expert[i] >= 0 ? exp(x[i] - (double)top) * share : 0.0;
            if (expert[i] == m) of_m += g[i];
            else dot += g[i] * p[i];
        }
        of_m = sum_lanes<L>(of_m);
        dot = sum_lanes<L>(dot);
        const double apart = dot - of_m * (others * share);
        all = any ? (float)(-(dot + of_m * share) * share) : 0.0f;
        double d[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) d[i] = g[i];
        if (doubled) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) d[i] = 0.0;
#pragma unroll 1
            for (int k = 0; k < a.top_k; ++k) {
                const int from = first_lane + k % L;
                const int e = __shfl(k < L ? expert[0] : expert[kEach - 1], from);
                const double v = __shfl(k < L ? g[0] : g[kEach - 1], from);
#pragma unroll
                for (int i = 0; i < kEach; ++i) d[i] += e == expert[i] ? v : 0.0;
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) part[i] = (float)(p[i] * ((expert[i] == m ? 0.0 : d[i] - of_m) - apart));
    } else {
        int m = 0;
        if (a.renormalize) {
            // the largest logit's choice, the first of several
            best = max_lanes<L>(best);
#pragma unroll
            for (int i = 0; i < kEach; ++i) m = max(m, x[i] == best ? KP - (lane + i * L) : 0);
            m = KP - max_lanes<L>(m);
            if (best == kNone) best = 0.0;
        }
        double of_m = 0.0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (lane + i * L == m) of_m = g[i];
            p[i] = 0.0;
            if (expert[i] < 0) continue;
            if (a.sigmoid) {
                // s and 1 - s, from one exponential and one division
                const double e = exp(-__builtin_fabs(x[i])), one = 1.0 / (1.0 + e);
                p[i] = x[i] < 0.0 ? e * one : one;
                rest[i] = x[i] < 0.0 ? one : e * one;
            } else p[i] = exp(x[i] - best);
            sum += p[i];
        }
        if (a.renormalize) {
            sum = sum_lanes<L>(sum);
            if (!(sum > 0.0)) sum = __builtin_inf();
            of_m = sum_lanes<L>(of_m);
            // g - sum_j q_j g_j as (g - g_m) - sum_j q_j (g_j - g_m): as above
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                p[i] /= sum;
                g[i] -= of_m;
                dot += g[i] * p[i];
            }
            dot = sum_lanes<L>(dot);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            double d = p[i] * (g[i] - dot);
            if (a.sigmoid && expert[i] >= 0) d *= rest[i];
            part[i] = (float)d;
        }
    }
    // the row; lane l makes the experts 4 l .. 4 l + 3 and every 4 L on
    for (int e = lane * 4; e < a.num_experts; e += L * 4) {
        float v[4] = {};
        if (full && any && live) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e + i < a.num_experts) v[i] = all * expf(T::load(logits[e + i]) - top);
        }
        *reinterpret_cast<u32x4*>(mine + e) = F32::pack(v);
    }
    wave_sync();
    if (full || !doubled) {  // of the full softmax, the chosen experts' parts are whole
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (expert[i] >= 0) mine[expert[i]] = part[i];
    } else {
        // in order of k, each expert's by the lane that holds it
#pragma unroll 1
        for (int k = 0; k < a.top_k; ++k) {
            const int from = first_lane + k % L;
            const int e = __shfl(k < L ? expert[0] : expert[kEach - 1], from);
            const float v = __shfl(k < L ? part[0] : part[kEach - 1], from);
            if (e >= 0 && e / 4 % L == lane) mine[e] += v;
        }
    }
    wave_sync();
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
        for (int e0 = lane * 4; e0 < a.num_experts; e0 += L * 4)
            for (int e = e0; e < min(e0 + 4, a.num_experts); ++e) out[e] = T::store(mine[e]);
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
    a.staged = L == 8 && a.vec && a.group_lanes < L;
    const int lds = a.staged ? per * ((a.num_experts / 4 + 7) & ~7) * 4 * (int)sizeof(typename T::E) : 0;
    hipLaunchKernelGGL(fn, grid, dim3(kRouteThreads), lds, s, a);
    return hipGetLastError();
}

// Lanes per token: 8, so that a wave's instructions serve eight tokens; 64
// where there are so few tokens that latency counts (64 tokens of 256 experts:
// 7.3 us against 18.5), or more experts than eight lanes hold (more than 256, or
// 32 in a group).  Those cost four times as much on many tokens: 131072 of 512
// experts, eight chosen, take 167 us, of 256 experts 35; nothing lies between.
constexpr int64_t kFewTokens = 2048;
template <class T>
int pick_route(const RouteArgs& a, hipStream_t s) {
    const int few = per_lane(a, 8), many = per_lane(a, 64);
    if (few <= 4) return run_route<T, 8, 4>(a, s);
    if (many <= 4 && a.tokens.total() <= kFewTokens) return run_route<T, 64, 4>(a, s);
    if (few <= 8) return run_route<T, 8, 8>(a, s);
    if (few <= 16) return run_route<T, 8, 16>(a, s);
    if (few <= 32) return run_route<T, 8, 32>(a, s);
    if (many <= 8) return run_route<T, 64, 8>(a, s);
    if (many <= 16) return run_route<T, 64, 16>(a, s);
    return run_route<T, 64, 32>(a, s);
}

template <class T>
int pick_route_grad(const RouteArgs& a, hipStream_t s) {
    const int row = ((a.num_experts + 3) & ~3) * 4;
    if (a.num_experts <= 256) {
        constexpr int per = kRouteThreads / 8;
        auto fn = a.top_k <= 8 ? route_grad_kernel<T, 8, 8> : route_grad_kernel<T, 8, RC_MAX_TOP_K>;
        hipLaunchKernelGGL(fn, grid_of(((int64_t)a.tokens.total() + per - 1) / per),
                           dim3(kRouteThreads), per * row, s, a);
    } else {
        constexpr int per = kRouteThreads / 64;
        hipLaunchKernelGGL((route_grad_kernel<T, 64, RC_MAX_TOP_K>), grid_of(((int64_t)a.tokens.total() + per - 1) / per),
                           dim3(kRouteThreads), per * row, s, a);
    }
    return hipGetLastError();
}

}  // namespace

// This file is compiled once per element type of the logits (RC_ROW_TYPE), so
// that the instantiations compile in parallel.
#define RC_JOIN2(a, b) a##b
#define RC_JOIN(a, b) RC_JOIN2(a, b)

int RC_JOIN(launch_route_, RC_ROW_TYPE)(const RouteArgs& a, void* stream) {
    return pick_route<RC_ROW_TYPE>(a, static_cast<hipStream_t>(stream));
}
int RC_JOIN(launch_route_grad_, RC_ROW_TYPE)(const RouteArgs& a, void* stream) {
    return pick_route_grad<RC_ROW_TYPE>(a, static_cast<hipStream_t>(stream));
}

}  // namespace rc
