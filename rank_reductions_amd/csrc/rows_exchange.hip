// Dispatch and combine: the plan (a counting sort of all ranks' choices by
// expert) and the row moves between tokens and experts' ranks.
//
// All are bound by memory.  A row move gives one wave a piece of one token's
// row: a dispatched row is read once and written to its K places, a combined
// one is the sum of K places, held in float32 and rounded once.
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

// Places of the entries of one block, with the blocks' starts in hist.
__global__ __launch_bounds__(kSortThreads) void plan_place_kernel(PlanArgs a) {
    __shared__ int32_t count[kSortWaves * kSortBins];
    __shared__ int32_t start[kSortBins];
    __shared__ int32_t base[kSortBins];
    __shared__ int32_t carry[kSortWaves];
    const SortPass& s = a.sort;
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int32_t* total = s.hist + (int64_t)s.blocks.total() * s.bins;
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) {
        start[d] = total[d];
        for (int w = 0; w < kSortWaves; ++w) count[w * kSortBins + d] = 0;
    }
    __syncthreads();
    exclusive_sum<kSortThreads>(start, s.bins, carry);
    for (int e = threadIdx.x; e < s.bins; e += kSortThreads) {
        base[e] = start[e] - start[e / a.per_rank * a.per_rank] + s.hist[(int64_t)blockIdx.x * s.bins + e];
        if (blockIdx.x == 0) write_offsets(a, start, e, total[e]);
    }
    int32_t block;
    const int rank = rank_of(s.blocks, blockIdx.x, &block);
    const int at = wave * kStrips * kWave + lane;
    int32_t key[kStrips];
#pragma unroll
    for (int k = 0; k < kStrips; ++k) {
        int32_t val;
        const bool in = sort_entry<true>(s, rank, block, at + k * kWave, &key[k], &val);
        if (!in) key[k] = -1;
        else if (key[k] < a.num_experts) atomicAdd(&count[wave * kSortBins + key[k]], 1);
    }
    wave_starts<kSortWaves>(count, base, s.bins);
#pragma unroll
    for (int k = 0; k < kStrips; ++k) {
        const bool has = key[k] >= 0 && key[k] < a.num_experts;
        const int32_t slot = strip_rank(key[k], s.bits, has, &count[wave * kSortBins]);
        if (key[k] >= 0) write_slot(a, rank, block * kSortBlock + at + k * kWave, has, key[k], slot);
    }
}

// The whole plan in one workgroup, for few entries.
constexpr int kSmallWaves = 8;
constexpr int kSmallEntries = 8192;
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
    for (int d = threadIdx.x; d < s.bins; d += kThreads)
        for (int w = 0; w < kSmallWaves; ++w) count[w * kSortBins + d] = 0;
    __syncthreads();
    const int32_t at = wave * strips * kWave + lane;
    for (int k = 0; k < strips; ++k) {
        int32_t i;
        const bool in = at + k * kWave < n;
        const int rank = rank_of(s.spans, in ? at + k * kWave : 0, &i);
        const int32_t key = in ? first_key(s, rank, i) : a.num_experts;
        if (key < a.num_experts) atomicAdd(&count[wave * kSortBins + key], 1);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < s.bins; d += kThreads) {
        int32_t sum = 0;
        for (int w = 0; w < kSmallWaves; ++w) sum += count[w * kSortBins + d];
        start[d] = total[d] = sum;
    }
    __syncthreads();
    exclusive_sum<kThreads>(start, s.bins, carry);
    for (int e = threadIdx.x; e < s.bins; e += kThreads) write_offsets(a, start, e, total[e]);
    // total becomes the start of each expert within its rank
    __syncthreads();
    for (int e = threadIdx.x; e < s.bins; e += kThreads) total[e] = start[e] - start[e / a.per_rank * a.per_rank];
    wave_starts<kSmallWaves>(count, total, s.bins);
    for (int k = 0; k < strips; ++k) {
        int32_t i;
        const bool in = at + k * kWave < n;
        const int rank = rank_of(s.spans, in ? at + k * kWave : 0, &i);
        const int32_t key = in ? first_key(s, rank, i) : a.num_experts;
        const bool has = key < a.num_experts;
        const int32_t slot = strip_rank(key, s.bits, has, &count[wave * kSortBins]);
        if (in) write_slot(a, rank, i, has, key, slot);
    }
}

// ---------------------------------------------------------------- row moves

constexpr int kRowThreads = 256;
constexpr int kRowVecs = 2;  // 16-byte vectors per lane and piece

// One wave's piece of one token's row.
struct Piece {
    int rank;
    int32_t token;   // within the rank
    int64_t col;     // first element of the lane's first vector
};

template <class T>
__device__ __forceinline__ bool piece_of(const RankSpans& tokens, int32_t chunks, Piece* p) {
    const int64_t item = group_index() * (kRowThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (item >= (int64_t)tokens.total() * chunks) return false;
    const int32_t token = (int32_t)(item / chunks);
    p->rank = rank_of(tokens, token, &p->token);
    p->col = (item - (int64_t)token * chunks) * (kWave * T::n * kRowVecs) + lane_id() * T::n;
    return true;
}

// Lane k's choice k of the token: the address of its row, or NULL.  `base` is
// the table of the experts' ranks' row buffers.
template <class E>
__device__ __forceinline__ E* place_of(const ExchangeArgs& a, const void* const* base, int rank, int32_t token, int k) {
    const int32_t slot = a.slots[rank][(int64_t)token * a.top_k + k];
    const int32_t expert = a.experts[rank][(int64_t)token * a.top_k + k];
    if (expert < 0 || expert >= a.num_experts || slot < 0) return nullptr;
    const int d = expert / a.per_rank;
    if (slot >= a.capacity[d]) return nullptr;
    return static_cast<E*>(const_cast<void*>(base[d])) + slot * a.width;
}

template <class E>
__device__ __forceinline__ E* from_lane(E* p, int lane) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane), hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
    return reinterpret_cast<E*>((uint64_t)hi << 32 | lo);
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(ExchangeArgs a) {
    using E = typename T::E;
    Piece p;
    if (!piece_of<T>(a.tokens, a.chunks, &p)) return;
    const int lane = lane_id();
    E* mine = lane < a.top_k ? place_of<E>(a, a.out, p.rank, p.token, lane) : nullptr;
    const E* src = static_cast<const E*>(a.in[p.rank]) + (int64_t)p.token * a.width;
    u32x4 v[kRowVecs];
    bool full[kRowVecs];
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) {
        const int64_t col = p.col + u * (kWave * T::n);
        full[u] = col + T::n <= a.width;
        if (full[u]) v[u] = load16<T>(src + col);
    }
    for (int k = 0; k < a.top_k; ++k) {
        E* dst = from_lane(mine, k);
        if (!dst) continue;
#pragma unroll
        for (int u = 0; u < kRowVecs; ++u) {
            const int64_t col = p.col + u * (kWave * T::n);
            if (full[u]) store16<T>(dst + col, v[u]);
            else
                for (int64_t c = col; c < a.width; ++c) dst[c] = src[c];
        }
    }
}

template <class T, int KP>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(ExchangeArgs a) {
    using E = typename T::E;
    Piece p;
    if (!piece_of<T>(a.tokens, a.chunks, &p)) return;
    const int lane = lane_id();
    E* mine = lane < a.top_k ? place_of<E>(a, a.in, p.rank, p.token, lane) : nullptr;
    float weight = 1.0f;
    if (a.weighted && lane < a.top_k) weight = a.weights[p.rank][(int64_t)p.token * a.top_k + lane];
    const E* src[KP];
    float w[KP];
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        src[k] = from_lane(mine, k);
        w[k] = lane_value(weight, k);
    }
    E* dst = static_cast<E*>(a.out[p.rank]) + (int64_t)p.token * a.width;
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) {
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
constexpr int kGradThreads = 256;
template <class T, int KP>
__global__ __launch_bounds__(kGradThreads) void combine_grad_kernel(ExchangeArgs a) {
    using E = typename T::E;
    __shared__ float part[kGradThreads / kWave][KP];
    if (group_index() >= a.tokens.total()) return;
    int32_t token;
    const int rank = rank_of(a.tokens, (int32_t)group_index(), &token);
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    E* row = lane < a.top_k ? place_of<E>(a, a.in, rank, token, lane) : nullptr;
    E* d_row = lane < a.top_k ? place_of<E>(a, a.out, rank, token, lane) : nullptr;
    const float weight = lane < a.top_k ? a.weights[rank][(int64_t)token * a.top_k + lane] : 0.0f;
    const E* src = static_cast<const E*>(a.d_out[rank]) + (int64_t)token * a.width;
    const E* at[KP];
    E* to[KP];
    float w[KP], dot[KP] = {};
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        at[k] = from_lane(row, k);
        to[k] = from_lane(d_row, k);
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
            for (int64_t c = col; c < a.width; ++c) {
                const float dy = T::load(src[c]);
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    if (!at[k]) continue;
                    dot[k] = __builtin_fmaf(dy, T::load(at[k][c]), dot[k]);
                    to[k][c] = T::store(w[k] * dy);
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
        for (int w = 0; w < kGradThreads / kWave; ++w) sum += part[w][threadIdx.x];
        a.d_weights[rank][(int64_t)token * a.top_k + threadIdx.x] = row ? sum : 0.0f;
    }
}

hipError_t last() { return hipGetLastError(); }

int bits_of(int64_t values) {
    int b = 0;
    while ((int64_t(1) << b) < values) ++b;
    return b;
}

template <class T>
int32_t chunks_of(int64_t width) {
    const int64_t piece = kWave * T::n * kRowVecs;
    return (int32_t)((width + piece - 1) / piece);
}

template <class T>
int run_dispatch(ExchangeArgs a, hipStream_t s) {
    a.chunks = chunks_of<T>(a.width);
    const int64_t items = (int64_t)a.tokens.total() * a.chunks, per = kRowThreads / kWave;
    hipLaunchKernelGGL(dispatch_kernel<T>, grid_of((items + per - 1) / per), dim3(kRowThreads), 0, s, a);
    return last();
}

template <class T>
int run_combine(ExchangeArgs a, hipStream_t s) {
    a.chunks = chunks_of<T>(a.width);
    const int64_t items = (int64_t)a.tokens.total() * a.chunks, per = kRowThreads / kWave;
    const dim3 grid = grid_of((items + per - 1) / per);
    auto fn = a.top_k <= 2 ? combine_kernel<T, 2> : a.top_k <= 4 ? combine_kernel<T, 4>
            : a.top_k <= 8 ? combine_kernel<T, 8> : combine_kernel<T, 16>;
    hipLaunchKernelGGL(fn, grid, dim3(kRowThreads), 0, s, a);
    return last();
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
    const int32_t blocks = p.blocks.total();
    hipLaunchKernelGGL(sort_count_kernel<true>, dim3(blocks), dim3(kSortThreads), 0, s, p);
    hipLaunchKernelGGL(sort_scan_kernel, dim3((p.bins + kWave - 1) / kWave), dim3(kScanWaves * kWave), 0, s, p.hist, blocks, p.bins);
    hipLaunchKernelGGL(plan_place_kernel, dim3(blocks), dim3(kSortThreads), 0, s, a);
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
