// Dispatch and combine: the plan (a counting sort of all ranks' choices by
// expert) and the row moves between tokens and experts' ranks.
//
// A row move gives one wave a piece of one token's row: a dispatched row is read
// once and written to its K places, a combined one is the sum of K places, held
// in float32 and rounded once.  All wait for memory: 16384 tokens of 4096
// bf16, eight places each, take 221 us to dispatch (1.2 GB at 5.5 TB/s), 258 to
// combine (4.7 TB/s) and 433 for the combination's gradient (2.3 GB at 5.3),
// where this library's copies, which limit what is under way, move 6.7.  With
// 10 and 16 places the rates are alike (4.9 to 5.3 in a row of calls).
// The plan is bound by latency: 131072 entries 15.8 us in two launches, 512 in
// one, 5.3 us.
#include "rows_sort.h"

namespace rc {
namespace {

// ---------------------------------------------------------------- the plan

// Writes one rank's offsets and counts: first[e] is the first row of expert e
// in its rank's buffer, total[e] the entries that chose it.
__device__ __forceinline__ void write_offsets(const PlanArgs& a, const int32_t* start, int e, int32_t count) {
    const int rank = e / a.per_rank, j = e - rank * a.per_rank;
    const int64_t first = start[e] - start[rank * a.per_rank];
    a.counts[rank][j] = count;
    a.offsets[rank][j] = (int32_t)min(first, a.capacity[rank]);
    if (j == a.per_rank - 1) a.offsets[rank][j + 1] = (int32_t)min(first + count, a.capacity[rank]);
}

__device__ __forceinline__ void write_slot(const PlanArgs& a, int rank, int32_t i, bool has, int expert, int32_t slot) {
    const bool fits = has && slot < a.capacity[has ? expert / a.per_rank : 0];
    a.slots[rank][i] = fits ? slot : -1;
}

// Places of the entries of one block.
__global__ __launch_bounds__(kSortThreads) void plan_place_kernel(PlanArgs a) {
    __shared__ int32_t count[kSortWaves * kSortBins];
    __shared__ int32_t start[kSortBins];
    __shared__ int32_t total[kSortBins];
    __shared__ int32_t base[kSortBins];
    __shared__ int32_t carry[kSortWaves];
    const SortPass& s = a.sort;
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    int32_t block;
    const int rank = rank_of(s.blocks, blockIdx.x, &block);
    const int at = wave * kStrips * kWave + lane;
    int32_t key[kStrips];
#pragma unroll
    for (int k = 0; k < kStrips; ++k) {
        int32_t val;
        if (!sort_entry<true>(s, rank, block, at + k * kWave, &key[k], &val)) key[k] = -1;
    }
    BlockSums sums;
    sums.load(s);
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) {
        base[d] = total[d] = 0;
        for (int w = 0; w < kSortWaves; ++w) count[w * kSortBins + d] = 0;
    }
    __syncthreads();
    sums.add(s, base, total);
    __syncthreads();
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) start[d] = total[d];
    __syncthreads();
    exclusive_sum<kSortThreads>(start, s.bins, carry);
    for (int e = threadIdx.x; e < s.bins; e += kSortThreads) {
        base[e] += start[e] - start[e / a.per_rank * a.per_rank];
        if (blockIdx.x == 0) write_offsets(a, start, e, total[e]);
    }
#pragma unroll
    for (int k = 0; k < kStrips; ++k)
        if (key[k] >= 0 && key[k] < a.num_experts) atomicAdd(&count[wave * kSortBins + key[k]], 1);
    wave_starts<kSortWaves>(count, base, s.bins);
#pragma unroll
    for (int k = 0; k < kStrips; ++k) {
        const bool has = key[k] >= 0 && key[k] < a.num_experts;
        const int32_t slot = strip_rank(key[k], s.bits, has, &count[wave * kSortBins]);
        if (key[k] >= 0) write_slot(a, rank, block * kSortBlock + at + k * kWave, has, key[k], slot);
    }
}

// The whole plan in one workgroup, for few entries: one launch instead of two.
constexpr int kSmallWaves = 8;
constexpr int kSmallStrips = 8;
constexpr int kSmallEntries = kSmallWaves * kSmallStrips * kWave;
__global__ __launch_bounds__(kSmallWaves* kWave) void plan_small_kernel(PlanArgs a) {
    __shared__ int32_t count[kSmallWaves * kSortBins];
    __shared__ int32_t start[kSortBins];
    __shared__ int32_t total[kSortBins];
    __shared__ int32_t carry[kSmallWaves];
    constexpr int kThreads = kSmallWaves * kWave;
    const SortPass& s = a.sort;
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int32_t n = s.spans.total();
    const int strips = (n + kThreads - 1) / kThreads;  // of each wave
    const int32_t at = wave * strips * kWave + lane;
    int32_t key[kSmallStrips], index[kSmallStrips], rank[kSmallStrips];
#pragma unroll
    for (int k = 0; k < kSmallStrips; ++k) {
        key[k] = -1;
        index[k] = rank[k] = 0;
        if (k < strips && at + k * kWave < n) {
            rank[k] = rank_of(s.spans, at + k * kWave, &index[k]);
            key[k] = first_key(s, rank[k], index[k]);
        }
    }
    for (int d = threadIdx.x; d < s.bins; d += kThreads)
        for (int w = 0; w < kSmallWaves; ++w) count[w * kSortBins + d] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSmallStrips; ++k)
        if (key[k] >= 0 && key[k] < a.num_experts) atomicAdd(&count[wave * kSortBins + key[k]], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < s.bins; d += kThreads) {
        int32_t sum = 0;
        for (int w = 0; w < kSmallWaves; ++w) sum += count[w * kSortBins + d];
        start[d] = total[d] = sum;
    }
    __syncthreads();
    exclusive_sum<kThreads>(start, s.bins, carry);
    for (int e = threadIdx.x; e < s.bins; e += kThreads) {
        write_offsets(a, start, e, total[e]);
        // the start of each expert within its rank, then of each wave's part
        int32_t run = start[e] - start[e / a.per_rank * a.per_rank];
        for (int w = 0; w < kSmallWaves; ++w) {
            const int32_t c = count[w * kSortBins + e];
            count[w * kSortBins + e] = run;
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSmallStrips; ++k) {
        if (k < strips) {  // alike in all lanes
            const bool has = key[k] >= 0 && key[k] < a.num_experts;
            const int32_t slot = strip_rank(key[k], s.bits, has, &count[wave * kSortBins]);
            if (key[k] >= 0) write_slot(a, rank[k], index[k], has, key[k], slot);
        }
    }
}

// ---------------------------------------------------------------- row moves

constexpr int kRowThreads = 256;

// The ranks' tables of a launch, one entry per lane (lane l holds rank
// l mod kMaxRanks): the argument block is read in one round of independent
// loads, and entries picked with lane moves, where indexing it by a rank that
// was itself just loaded takes a dependent trip to memory each time.
struct Tables {
    const int32_t* experts;
    const int32_t* slots;
    const void* near;   // the ranks' buffers by token
    const void* far;    // the ranks' row buffers
    int64_t capacity;
    int32_t first;      // the rank's first token
};

__device__ __forceinline__ Tables tables_of(const ExchangeArgs& a, const void* const* near, const void* const* far) {
    const int r = lane_id() & (kMaxRanks - 1);
    return {a.experts[r], a.slots[r], near[r], far[r], a.capacity[r], a.tokens.first[r]};
}

template <class P>
__device__ __forceinline__ P* lane_ptr(P* p, int lane) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane), hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
    return reinterpret_cast<P*>((uint64_t)hi << 32 | lo);
}

// The rank of token n of all (alike in all lanes), and the token within it.
__device__ __forceinline__ int rank_by_lane(const Tables& t, int nranks, int32_t n, int32_t* token) {
    const int rank = __popcll(__ballot(lane_id() < nranks && t.first <= n)) - 1;
    *token = n - __builtin_amdgcn_readlane(t.first, rank);
    return rank;
}

// One wave's piece of one token's row.
struct Piece {
    int rank;
    int32_t token;   // within the rank
    int64_t col;     // first element of the lane's first vector
};

template <class T, int U>
__device__ __forceinline__ bool piece_of(const ExchangeArgs& a, const Tables& t, Piece* p) {
    const int64_t item = group_index() * (kRowThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (item >= (int64_t)a.tokens.total() * a.chunks) return false;
    const int32_t n = (int32_t)(item / a.chunks);
    p->rank = rank_by_lane(t, a.tokens.nranks, n, &p->token);
    p->col = (item - (int64_t)n * a.chunks) * (kWave * T::n * U) + lane_id() * T::n;
    return true;
}

// Lane k's choice k of the token: the rank of its expert, or -1, and its row there.
struct Choice {
    int rank;
    int32_t slot;
};
__device__ __forceinline__ Choice choice_of(const ExchangeArgs& a, const Tables& t, int rank, int32_t token) {
    Choice c{-1, 0};
    int32_t expert = -1;
    const int lane = lane_id();
    const int32_t* slots = lane_ptr(t.slots, rank);
    const int32_t* experts = lane_ptr(t.experts, rank);
    if (lane < a.top_k) {
        c.slot = slots[(int64_t)token * a.top_k + lane];
        expert = experts[(int64_t)token * a.top_k + lane];
    }
    const bool has = expert >= 0 && expert < a.num_experts && c.slot >= 0;
    const int d = has ? (int)((uint32_t)expert / (uint32_t)a.per_rank) : 0;
    const int64_t capacity = __shfl(t.capacity, d);
    if (has && c.slot < capacity) c.rank = d;
    return c;
}
// The address of the row in the buffers that the lanes hold, or NULL.
template <class E>
__device__ __forceinline__ E* row_at(const Choice& c, const void* buffers, int64_t width) {
    const int d = c.rank < 0 ? 0 : c.rank;
    const uint64_t base = __shfl(reinterpret_cast<unsigned long long>(buffers), d);
    return c.rank < 0 ? nullptr : reinterpret_cast<E*>(base) + c.slot * width;
}

template <class T, int U>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(ExchangeArgs a) {
    using E = typename T::E;
    const Tables t = tables_of(a, a.in, a.out);
    Piece p;
    if (!piece_of<T, U>(a, t, &p)) return;
    const E* src = static_cast<const E*>(lane_ptr(t.near, p.rank)) + (int64_t)p.token * a.width;
    u32x4 v[U];
    bool full[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t col = p.col + u * (kWave * T::n);
        full[u] = col + T::n <= a.width;
        if (full[u]) v[u] = load16<T>(src + col);
    }
    E* mine = row_at<E>(choice_of(a, t, p.rank, p.token), t.far, a.width);
    for (int k = 0; k < a.top_k; ++k) {
        E* dst = lane_ptr(mine, k);
        if (!dst) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t col = p.col + u * (kWave * T::n);
            if (full[u]) store16<T>(dst + col, v[u]);
            else
                for (int64_t c = col; c < a.width; ++c) dst[c] = src[c];
        }
    }
}

template <class T, int KP, int U>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(ExchangeArgs a) {
    using E = typename T::E;
    const Tables t = tables_of(a, a.out, a.in);
    const float* weights = a.weights[lane_id() & (kMaxRanks - 1)];
    Piece p;
    if (!piece_of<T, U>(a, t, &p)) return;
    const int lane = lane_id();
    float weight = 1.0f;
    if (a.weighted) {
        const float* of_rank = lane_ptr(weights, p.rank);
        if (lane < a.top_k) weight = of_rank[(int64_t)p.token * a.top_k + lane];
    }
    E* mine = row_at<E>(choice_of(a, t, p.rank, p.token), t.far, a.width);
    const E* src[KP];
    float w[KP];
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        src[k] = lane_ptr(mine, k);
        w[k] = lane_value(weight, k);
    }
    E* dst = static_cast<E*>(const_cast<void*>(lane_ptr(t.near, p.rank))) + (int64_t)p.token * a.width;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t col = p.col + u * (kWave * T::n);
        if (col + T::n <= a.width) {
            u32x4 v[KP];
#pragma unroll
            for (int k = 0; k < KP; ++k)
                if (src[k]) v[k] = load16<T>(src[k] + col);
            float acc[T::n] = {};
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                if (!src[k]) continue;
                float f[T::n];
                T::unpack(v[k], f);
#pragma unroll
                for (int i = 0; i < T::n; ++i) acc[i] = __builtin_fmaf(w[k], f[i], acc[i]);
            }
            store16<T>(dst + col, T::pack(acc));
        } else {
            for (int64_t c = col; c < a.width; ++c) {
                float acc = 0.0f;
#pragma unroll
                for (int k = 0; k < KP; ++k)
                    if (src[k]) acc = __builtin_fmaf(w[k], T::load(src[k][c]), acc);
                dst[c] = T::store(acc);
            }
        }
    }
}

// One workgroup per token: its waves take the row's pieces in turn, each lane
// summing its own products, then all lanes' sums are joined in a fixed tree.
// Rows and their products are read once for both gradients.
constexpr int kGradThreads = 256;
template <class T, int KP>
__global__ __launch_bounds__(kGradThreads) void combine_grad_kernel(ExchangeArgs a) {
    using E = typename T::E;
    __shared__ float part[kGradThreads / kWave][KP];
    const Tables t = tables_of(a, a.d_out, a.in);
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const float* weights = a.weights[lane & (kMaxRanks - 1)];
    const void* d_rows = a.out[lane & (kMaxRanks - 1)];
    if (group_index() >= a.tokens.total()) return;
    int32_t token;
    const int rank = rank_by_lane(t, a.tokens.nranks, (int32_t)group_index(), &token);
    const float* of_rank = lane_ptr(weights, rank);
    const float weight = lane < a.top_k ? of_rank[(int64_t)token * a.top_k + lane] : 0.0f;
    const Choice c = choice_of(a, t, rank, token);
    E* row = row_at<E>(c, t.far, a.width);
    E* d_row = row_at<E>(c, d_rows, a.width);
    const E* src = static_cast<const E*>(lane_ptr(t.near, rank)) + (int64_t)token * a.width;
    const E* at[KP];
    E* to[KP];
    float w[KP], dot[KP] = {};
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        at[k] = lane_ptr(row, k);
        to[k] = lane_ptr(d_row, k);
        w[k] = lane_value(weight, k);
    }
    for (int64_t col = (int64_t)threadIdx.x * T::n; col < a.width; col += kGradThreads * T::n) {
        if (col + T::n <= a.width) {
            const u32x4 dv = load16<T>(src + col);
            u32x4 v[KP];
#pragma unroll
            for (int k = 0; k < KP; ++k)
                if (at[k]) v[k] = load16<T>(at[k] + col);
            float dy[T::n];
            T::unpack(dv, dy);
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                if (!at[k]) continue;
                float f[T::n], g[T::n];
                T::unpack(v[k], f);
#pragma unroll
                for (int i = 0; i < T::n; ++i) {
                    dot[k] = __builtin_fmaf(dy[i], f[i], dot[k]);
                    g[i] = w[k] * dy[i];
                }
                store16<T>(to[k] + col, T::pack(g));
            }
        } else {
            for (int64_t i = col; i < a.width; ++i) {
                const float dy = T::load(src[i]);
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    if (!at[k]) continue;
                    dot[k] = __builtin_fmaf(dy, T::load(at[k][i]), dot[k]);
                    to[k][i] = T::store(w[k] * dy);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < KP; ++k) {
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) dot[k] += __shfl_xor(dot[k], o);
        if (lane == 0) part[wave][k] = dot[k];
    }
    __syncthreads();
    if (threadIdx.x < (unsigned)a.top_k) {
        float sum = 0.0f;
        for (int w2 = 0; w2 < kGradThreads / kWave; ++w2) sum += part[w2][threadIdx.x];
        a.d_weights[rank][(int64_t)token * a.top_k + threadIdx.x] = row ? sum : 0.0f;
    }
}

hipError_t last() { return hipGetLastError(); }

int bits_of(int64_t values) {
    int b = 0;
    while ((int64_t(1) << b) < values) ++b;
    return b;
}

// 16-byte vectors per lane and piece: two, or one where that gives too few
// waves to fill the GPU.
constexpr int64_t kFillWaves = 4096;
template <class T>
int vectors_of(const ExchangeArgs& a) {
    const int64_t two = kWave * T::n * 2;
    return (a.width + two - 1) / two * a.tokens.total() >= kFillWaves ? 2 : 1;
}
template <class T>
dim3 pieces_of(ExchangeArgs* a, int vectors) {
    const int64_t piece = kWave * T::n * vectors, per = kRowThreads / kWave;
    a->chunks = (int32_t)((a->width + piece - 1) / piece);
    return grid_of(((int64_t)a->tokens.total() * a->chunks + per - 1) / per);
}

template <class T>
int run_dispatch(ExchangeArgs a, hipStream_t s) {
    const int u = vectors_of<T>(a);
    const dim3 grid = pieces_of<T>(&a, u);
    hipLaunchKernelGGL((u == 2 ? dispatch_kernel<T, 2> : dispatch_kernel<T, 1>), grid, dim3(kRowThreads), 0, s, a);
    return last();
}

template <class T, int U>
int run_combine_u(ExchangeArgs a, hipStream_t s) {
    const dim3 grid = pieces_of<T>(&a, U);
    auto fn = a.top_k <= 2 ? combine_kernel<T, 2, U> : a.top_k <= 4 ? combine_kernel<T, 4, U>
            : a.top_k <= 8 ? combine_kernel<T, 8, U> : combine_kernel<T, 16, U>;
    hipLaunchKernelGGL(fn, grid, dim3(kRowThreads), 0, s, a);
    return last();
}
template <class T>
int run_combine(const ExchangeArgs& a, hipStream_t s) {
    return vectors_of<T>(a) == 2 ? run_combine_u<T, 2>(a, s) : run_combine_u<T, 1>(a, s);
}

template <class T>
int run_combine_grad(const ExchangeArgs& a, hipStream_t s) {
    auto fn = a.top_k <= 2 ? combine_grad_kernel<T, 2> : a.top_k <= 4 ? combine_grad_kernel<T, 4>
            : a.top_k <= 8 ? combine_grad_kernel<T, 8> : combine_grad_kernel<T, 16>;
    hipLaunchKernelGGL(fn, grid_of(a.tokens.total()), dim3(kGradThreads), 0, s, a);
    return last();
}

}  // namespace

int64_t plan_workspace_bytes(const RankSpans& entries, int num_experts) {
    if (entries.total() <= kSmallEntries) return 0;
    return ((int64_t)sort_blocks(entries).total() + 1) * num_experts * 4;
}

int launch_plan(PlanArgs a, void* workspace, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    SortPass& p = a.sort;
    p.id64 = 0;
    p.drop = 1;
    p.shift = 0;
    p.bits = bits_of(a.num_experts);
    p.bins = a.num_experts;
    p.hist = static_cast<int32_t*>(workspace);
    if (p.spans.total() <= kSmallEntries) {
        hipLaunchKernelGGL(plan_small_kernel, dim3(1), dim3(kSmallWaves * kWave), 0, s, a);
        return last();
    }
    p.blocks = sort_blocks(p.spans);
    launch_counts<true>(p, s);
    hipLaunchKernelGGL(plan_place_kernel, dim3(p.blocks.total()), dim3(kSortThreads), 0, s, a);
    return last();
}

int launch_dispatch(const ExchangeArgs& a, int dtype, void* stream) {
    return RC_BY_TYPE(run_dispatch, a, static_cast<hipStream_t>(stream));
}
int launch_combine(const ExchangeArgs& a, int dtype, void* stream) {
    return RC_BY_TYPE(run_combine, a, static_cast<hipStream_t>(stream));
}
int launch_combine_grad(const ExchangeArgs& a, int dtype, void* stream) {
    return RC_BY_TYPE(run_combine_grad, a, static_cast<hipStream_t>(stream));
}

}  // namespace rc
