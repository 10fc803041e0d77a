// The sharded embedding: lookup of rows by token id, and the table's gradient
// by sorted ids.
//
// Lookup: one wave per piece of a token's row; bound by memory: 65536 tokens of
// 4096 bf16 take 149 us (0.54 GB written and 0.34 read, 5.9 TB/s; the 13600 rows
// that they name are 0.11).
//
// Gradient: dW[v] = scale * sum of dy over the tokens whose id is v.  The ids
// of all ranks are sorted (stably, with their positions), so that the rows of
// one id lie side by side in the list.  The list is cut into windows of up to
// kPiece entries, one workgroup each (and per piece of the columns): it sums
// the ids that begin in its window, running on past the window's end, so no
// workgroup takes more than a window and a piece.  An id with more than
// kPiece entries is cut into pieces of kPiece from its first entry on; the
// workgroup in whose window a piece begins leaves its sum in the workspace
// and a second kernel joins them.  What an id's sum adds, and in what order,
// thus depends on its own tokens only.  Other workgroups of the same launch
// clear the table's rows that no id names.  Bound by memory: dy is read once
// and the table written once, 65536 tokens of 4096 bf16 into 32000 rows of
// float32 in 221 us (1.06 GB at 4.8 TB/s); the sort before it takes 33 and the
// joins 15.
#include "rows_sort.h"

#include <algorithm>

namespace rc {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowVecs = 2;  // 16-byte vectors per lane and piece

__device__ __forceinline__ int64_t id_of(const void* ids, int32_t id64, int32_t i) {
    return id64 ? static_cast<const int64_t*>(ids)[i] : (int64_t) static_cast<const int32_t*>(ids)[i];
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void embedding_kernel(EmbeddingArgs a) {
    using E = typename T::E;
    const int64_t item = group_index() * (kRowThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (item >= (int64_t)a.tokens.total() * a.chunks) return;
    const int32_t n = (int32_t)(item / a.chunks);
    int32_t token;
    const int rank = rank_of(a.tokens, n, &token);
    const int64_t first = (item - (int64_t)n * a.chunks) * (kWave * T::n * kRowVecs) + lane_id() * T::n;
    const int64_t id = id_of(a.ids[rank], a.id64, token);
    const bool named = id >= 0 && id < a.vocab;
    const int32_t shard = named ? (int32_t)id / (int32_t)a.shard : 0;
    const E* src = static_cast<const E*>(a.table[shard]) + (named ? id - shard * a.shard : 0) * a.width;
    E* dst = static_cast<E*>(a.out[rank]) + (int64_t)token * a.width;
    const bool copy = a.scale == 1.0f;
    u32x4 v[kRowVecs];
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) {
        const int64_t col = first + u * (kWave * T::n);
        v[u] = u32x4{0, 0, 0, 0};
        if (named && col + T::n <= a.width) v[u] = load16<T>(src + col);
    }
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) {
        const int64_t col = first + u * (kWave * T::n);
        if (col + T::n <= a.width) {
            if (!copy && named) {
                float f[T::n];
                T::unpack(v[u], f);
#pragma unroll
                for (int i = 0; i < T::n; ++i) f[i] *= a.scale;
                v[u] = T::pack(f);
            }
            store16<T>(dst + col, v[u]);
        } else {
            for (int64_t c = col; c < a.width; ++c) {
                if (!named) dst[c] = T::store(0.0f);
                else dst[c] = copy ? src[c] : T::store(T::load(src[c]) * a.scale);
            }
        }
    }
}

// ---------------------------------------------------------------- sorting the ids

// One pass's places over one block.
template <bool FIRST, bool LAST>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortPass s) {
    __shared__ int32_t count[kSortWaves * kSortBins];
    __shared__ int32_t start[kSortBins];
    __shared__ int32_t before[kSortBins];
    __shared__ int32_t carry[kSortWaves];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    int32_t block;
    const int rank = rank_of(s.blocks, blockIdx.x, &block);
    const int at = wave * kStrips * kWave + lane;
    const int32_t ones = (1 << s.bits) - 1;
    int32_t key[kStrips], val[kStrips];
#pragma unroll
    for (int k = 0; k < kStrips; ++k)
        if (!sort_entry<FIRST>(s, rank, block, at + k * kWave, &key[k], &val[k])) key[k] = -1;
    BlockSums sums;
    sums.load(s);
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) {
        before[d] = start[d] = 0;
        for (int w = 0; w < kSortWaves; ++w) count[w * kSortBins + d] = 0;
    }
    __syncthreads();
    sums.add(s, before, start);
    __syncthreads();
    exclusive_sum<kSortThreads>(start, s.bins, carry);
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) start[d] += before[d];
#pragma unroll
    for (int k = 0; k < kStrips; ++k)
        if (key[k] >= 0) atomicAdd(&count[wave * kSortBins + ((key[k] >> s.shift) & ones)], 1);
    wave_starts<kSortWaves>(count, start, s.bins);
#pragma unroll
    for (int k = 0; k < kStrips; ++k) {
        const bool has = key[k] >= 0;
        const int32_t place = strip_rank((key[k] >> s.shift) & ones, s.bits, has, &count[wave * kSortBins]);
        if (has) {
            s.out_keys[place] = key[k];
            s.out_vals[place] = val[k];
            if (LAST && s.named && key[k] < s.key_limit) s.named[key[k]] = 1;  // whoever else writes it writes the same
        }
    }
}

// Few ids, in one launch: an id's place is the number of ids below it, and of
// equal ones before it, counted by comparing it with all (kept in LDS).  A
// workgroup places 64 ids, one per lane; its waves share out what they are
// compared with.  Each workgroup also makes its part of the table's named bytes.
// 1700 ids take 7.7 us; two counting passes in one workgroup took 10.8, and the
// launches for more ids take 27 and up.
constexpr int kRankThreads = 1024;
constexpr int kRankWaves = kRankThreads / kWave;
constexpr int kRankIds = 8192;
constexpr int kRankEach = kRankIds / kRankThreads;
constexpr int kNamedChunk = 4096;  // table rows at a time
constexpr int64_t kRankGroups = 256;
__global__ __launch_bounds__(kRankThreads) void sort_rank_kernel(SortPass s) {
    __shared__ __align__(16) int32_t keys[kRankIds];
    __shared__ int32_t part[kRankWaves][kWave];
    __shared__ __align__(16) uint8_t named[kNamedChunk];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int32_t n = s.spans.total(), blocks = (n + kWave - 1) / kWave;
    int32_t own[kRankEach];
#pragma unroll
    for (int k = 0; k < kRankEach; ++k) {
        const int32_t j = k * kRankThreads + threadIdx.x;
        own[k] = 0x7fffffff;  // behind all ids
        if (j < n) {
            int32_t i;
            const int rank = rank_of(s.spans, j, &i);
            own[k] = first_key(s, rank, i);
        }
    }
#pragma unroll
    for (int k = 0; k < kRankEach; ++k)
        if (k * kRankThreads < n) keys[k * kRankThreads + threadIdx.x] = own[k];
    __syncthreads();
    const int32_t mine = blockIdx.x;
    if (mine < blocks) {
        const int32_t i = mine * kWave + lane, key = keys[i];
        const int32_t from = (int32_t)((int64_t)wave * blocks / kRankWaves), to = (int32_t)((int64_t)(wave + 1) * blocks / kRankWaves);
        int32_t below = 0;
        // f(j): what an id j places into the block has to lie below
        auto compare = [&](int32_t b, auto f) {
#pragma unroll
            for (int j = 0; j < kWave; j += 4) {
                const u32x4 v = *reinterpret_cast<const u32x4*>(keys + b * kWave + j);
#pragma unroll
                for (int c = 0; c < 4; ++c) below += v[c] < f(j + c);
            }
        };
        for (int32_t b = from; b < to; ++b) {
            const uint32_t limit = (uint32_t)key + (b < mine);
            if (b != mine) compare(b, [&](int) { return limit; });
            else compare(b, [&](int j) { return (uint32_t)key + (j < lane); });
        }
        part[wave][lane] = below;
        __syncthreads();
        if (wave == 0 && i < n) {
            int32_t place = 0;
#pragma unroll
            for (int w = 0; w < kRankWaves; ++w) place += part[w][lane];
            s.out_keys[place] = key;
            s.out_vals[place] = i;
        }
    }
    if (!s.named) return;
    for (int64_t base = (int64_t)blockIdx.x * kNamedChunk; base < s.key_limit; base += (int64_t)gridDim.x * kNamedChunk) {
        __syncthreads();
        reinterpret_cast<uint32_t*>(named)[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kRankEach; ++k) {
            const int64_t at = own[k] - base;
            if (at >= 0 && at < kNamedChunk) named[at] = 1;
        }
        __syncthreads();
        const int at = threadIdx.x * 16;
        if (at < kNamedChunk && base + at < s.key_limit)  // the bytes are padded to 16
            *reinterpret_cast<u32x4*>(s.named + base + at) = *reinterpret_cast<const u32x4*>(named + at);
    }
}
static_assert(kNamedChunk == 4 * kRankThreads, "a word each to clear");

// ---------------------------------------------------------------- summing

constexpr int kSumThreads = 256;
// Rows of dy in flight per lane.  1700 ids, 1000 columns, 64 and more of them one
// id's, us a call: 39 with two, 31 with four, 29 with eight or sixteen.
constexpr int kAhead = 8;
// Workgroups that keep the GPU busy.
constexpr int64_t kSumGroups = 8192;
constexpr int64_t kFillGroups = 4000;

// First of the sorted keys in [lo, hi) that is not below `key`, for arguments
// that all lanes share: 64 probes at a time, so that
// 65536 keys take three dependent loads rather than 16 (the keys come from
// another launch, mostly from beyond this XCD's L2).
__device__ __forceinline__ int32_t wave_lower_bound(const int32_t* keys, int32_t lo, int32_t hi, int64_t key) {
    while (lo < hi) {
        const int32_t step = (hi - lo + (kWave - 1)) / kWave;
        const int64_t p = lo + (int64_t)lane_id() * step;
        const int less = __popcll(__ballot(p < hi && keys[p < hi ? p : lo] < key));
        if (less == 0) break;
        hi = (int32_t)min((int64_t)hi, lo + (int64_t)less * step);
        lo += (less - 1) * step + 1;
    }
    return lo;
}

// The gradient's row v in its shard.
template <class G>
__device__ __forceinline__ typename G::E* table_row(const EmbeddingGradArgs& a, int64_t v) {
    const int32_t shard = (int32_t)v / (int32_t)a.shard;
    return static_cast<typename G::E*>(a.table[shard]) + (v - shard * a.shard) * a.width;
}

// A lane's columns: as many as one of its stores takes, in kParts pieces a
// wave's width apart, so that every store of a wave is of consecutive bytes and
// no line waits in L2 for its other half (65536 tokens into a float32 table:
// the same time as two 16-byte stores to a lane's own 32 bytes).
template <class T, class G>
struct Cols {
    static constexpr int kPart = T::n < G::n ? T::n : G::n;
    static constexpr int kParts = T::n / kPart;
    static constexpr int kWords = kPart * (int)sizeof(typename T::E) / 4;
};
typedef uint32_t u32x2m __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A part's elements; with FULL false only the first `rem`, the others zero.
// (One register per element there: packing them would wait for each load.)
template <class T, int PART, int WORDS, bool FULL>
__device__ __forceinline__ void load_part(const typename T::E* src, int rem, uint32_t* w) {
    if constexpr (!FULL) {
#pragma unroll
        for (int i = 0; i < PART; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < PART; ++i) {
            if (i >= rem) continue;
            if constexpr (sizeof(typename T::E) == 4) w[i] = __builtin_bit_cast(uint32_t, src[i]);
            else w[i] = __builtin_bit_cast(uint16_t, src[i]);
        }
    } else if constexpr (WORDS == 4) {
        const u32x4 v = load16<T>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = v[i];
    } else {
        const u32x2 v = *reinterpret_cast<const u32x2m*>(src);
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = v[i];
    }
}
template <class T, bool FULL>
__device__ __forceinline__ float element_of(const uint32_t* w, int i) {
    if constexpr (sizeof(typename T::E) == 4) {
        const uint32_t u = w[i];
        return __builtin_bit_cast(float, u);
    } else if constexpr (!FULL) {
        const uint16_t u = (uint16_t)w[i];
        return T::load(__builtin_bit_cast(typename T::E, u));
    } else {
        const uint16_t u = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
        return T::load(__builtin_bit_cast(typename T::E, u));
    }
}

// Writes N elements (G::n of them) of a table row, or `rem`.
template <class G, int N>
__device__ __forceinline__ void finish_row(const EmbeddingGradArgs& a, typename G::E* row, int rem, const float* sum) {
    static_assert(N == G::n);
    if (rem == N) {
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = sum[i] * a.scale;
        if (a.accumulate) {
            float old[N];
            G::unpack(load16<G>(row), old);
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] += old[i];
        }
        store16_past<G>(row, G::pack(f));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < rem) row[i] = G::store((a.accumulate ? G::load(row[i]) : 0.0f) + sum[i] * a.scale);
    }
}

// What a workgroup sums: the positions [begin, end) of its window's list.
struct SumRange {
    int begin, end;
    int carried;              // positions below it belong to a piece of an id that began earlier
    int hot;                  // positions from it on, to an id of several pieces
    uint64_t stops[2];        // positions that end an id or a piece
    float *carried_out, *hot_out;
};

// The sums of a lane's columns: col and rem are its parts' first columns and
// elements, with FULL all of them.  AHEAD rows are in flight; the addresses and
// the ends are alike in all lanes, so the loop has no branch before a load (with
// one, and with the zeros of a row's ragged end written between the loads, each
// row waited for the one before: 41 us for the 29 above, and 281 for the 268 of
// 65536 tokens of 4096 columns).
template <class T, class G, int AHEAD, bool FULL>
__device__ __forceinline__ void sum_rows(const EmbeddingGradArgs& a, const SumRange& r, const typename T::E* const* rows,
                                         const int32_t* key, const int64_t* col, const int* rem) {
    using C = Cols<T, G>;
    using E = typename T::E;
    constexpr int kWords = FULL ? C::kWords : C::kPart;
    float acc[C::kParts][C::kPart] = {};
    for (int j0 = r.begin; j0 < r.end; j0 += AHEAD) {
        uint32_t w[AHEAD][C::kParts][kWords];
        const E* src[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const uint64_t p = reinterpret_cast<uint64_t>(rows[min(j0 + u, r.end - 1)]);
            const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p), hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
            src[u] = reinterpret_cast<const E*>((uint64_t)hi << 32 | lo);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int h = 0; h < C::kParts; ++h) load_part<T, C::kPart, C::kWords, FULL>(src[u] + col[h], rem[h], w[u][h]);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int j = j0 + u;
            if (j >= r.end) break;
#pragma unroll
            for (int h = 0; h < C::kParts; ++h)
#pragma unroll
                for (int i = 0; i < C::kPart; ++i) acc[h][i] += element_of<T, FULL>(w[u][h], i);
            if (!((j < kWave ? r.stops[0] >> j : r.stops[1] >> (j - kWave)) & 1)) continue;
            const bool piece = j < r.carried || j >= r.hot;
            float* out = j < r.carried ? r.carried_out : r.hot_out;
            typename G::E* row = piece ? nullptr : table_row<G>(a, key[j]);
#pragma unroll
            for (int h = 0; h < C::kParts; ++h) {
                if (!piece) {
                    finish_row<G, C::kPart>(a, row + col[h], FULL ? C::kPart : rem[h], acc[h]);
                } else if (FULL) {
#pragma unroll
                    for (int i = 0; i < C::kPart; i += 4) store16<F32>(out + col[h] + i, F32::pack(acc[h] + i));
                } else {
#pragma unroll
                    for (int i = 0; i < C::kPart; ++i)
                        if (i < rem[h]) out[col[h] + i] = acc[h][i];
                }
#pragma unroll
                for (int i = 0; i < C::kPart; ++i) acc[h][i] = 0.0f;
            }
        }
    }
}

// T: type of dy; G: type of the table's gradient.
template <class T, class G>
__global__ __launch_bounds__(kSumThreads) void embedding_grad_kernel(EmbeddingGradArgs a) {
    using E = typename T::E;
    __shared__ int32_t keys[2 * kPiece + 2];  // of the positions p0 - 1 .. p0 + window + kPiece
    __shared__ const E* rows[2 * kPiece];
    const int lane = lane_id();
    const int32_t n = a.tokens.total();
    int64_t group = group_index();
    bool clears;
    if (a.spacing) {
        const int32_t turn = (int32_t)group / a.spacing;
        clears = (int32_t)group % a.spacing == 0 && turn < a.fill_groups;
        group = clears ? turn : group - min(a.fill_groups, turn + 1);
    } else {
        clears = group >= a.windows;
        if (clears) group -= a.windows;
    }
    if (group >= (clears ? a.fill_groups : a.windows)) return;
    if (clears) {
        // clear the rows of these ids that no token names
        const int64_t first = group * a.fill_rows;
        const int64_t v = first + lane;
        const bool mine = lane < a.fill_rows && v < a.vocab;
        uint64_t clear = __ballot(mine && !(n && a.named[v]));
        const int64_t lo = (int64_t)blockIdx.z * (kSumThreads * T::n), hi = min(lo + kSumThreads * T::n, a.width);
        while (clear) {
            const int j = __builtin_ctzll(clear);
            clear &= clear - 1;
            typename G::E* row = table_row<G>(a, first + j);
            for (int64_t c = lo + threadIdx.x * G::n; c < hi; c += kSumThreads * G::n) {
                if (c + G::n <= hi) store16_past<G>(row + c, u32x4{0, 0, 0, 0});
                else
                    for (int64_t i = c; i < hi; ++i) row[i] = G::store(0.0f);
            }
        }
        return;
    }
    const int W = a.window;
    const int32_t p0 = (int32_t)(group * W);
    for (int t = threadIdx.x; t < W + kPiece + 2; t += kSumThreads) {
        const int64_t p = (int64_t)p0 - 1 + t;
        keys[t] = p >= 0 && p < n ? a.keys[p] : -1;
        if (t >= 1 && t <= W + kPiece) {
            const E* src = nullptr;
            if (p < n) {
                int32_t token;
                const int rank = rank_of(a.tokens, a.vals[p], &token);
                src = static_cast<const E*>(a.d_out[rank]) + (int64_t)token * a.width;
            }
            rows[t - 1] = src;
        }
    }
    __syncthreads();
    // positions from here on count from p0; key[i] is position i's
    const int32_t* key = keys + 1;
    const int32_t none = (int32_t)a.vocab;  // ids that name no row sort last
    const int32_t mine = lane < W ? key[lane] : -1, after = key[W + lane];
    const bool real = mine >= 0 && mine < none;
    const bool first = real && mine != key[lane - 1];
    const uint64_t begins = __ballot(first);
    const uint64_t longs = __ballot(first && mine == key[lane + kPiece]);
    const int valid = __popcll(__ballot(real)) + __popcll(__ballot(after >= 0 && after < none));
    // first position past the window that is not of the window's last id
    const uint64_t other = __ballot(after != key[W - 1]);
    const int last_end = min(valid, W + (other ? (int)__builtin_ctzll(other) : kPiece));
    int begin = begins ? (int)__builtin_ctzll(begins) : 2 * kPiece;
    int carried = 0;  // positions below it belong to a piece of an id that began earlier
    if (key[0] >= 0 && key[0] < none && key[0] == key[-1]) {
        const int32_t s = wave_lower_bound(a.keys, 0, p0, key[0]);
        if (s + (int64_t)kPiece < n && a.keys[s + kPiece] == key[0]) {
            const int ps = (int)(((int64_t)p0 - s + kPiece - 1) / kPiece * kPiece + s - p0);
            const int end = begins ? begin : last_end;  // of the id, or past the piece
            if (ps < W && ps < end) {
                carried = min(ps + kPiece, end);
                begin = ps;
            }
        }
    }
    int end;
    const int hot = longs ? (int)__builtin_ctzll(longs) : 2 * kPiece;
    if (longs) end = hot + kPiece;
    else if (begins) end = last_end;
    else end = carried;
    if (begin >= end) return;
    SumRange r;
    r.begin = __builtin_amdgcn_readfirstlane(begin);
    r.end = __builtin_amdgcn_readfirstlane(end);
    r.carried = __builtin_amdgcn_readfirstlane(carried);
    r.hot = hot;
    for (int i = 0; i < 2; ++i) {
        const int j = i * kWave + lane;
        r.stops[i] = __ballot(j < r.end && (j + 1 == r.end || j + 1 == r.carried || key[j + 1] != key[j]));
    }
    // where the sums of the carried piece and of the long id's first go
    r.carried_out = a.partial + 2 * (int64_t)((p0 + r.begin) / kPiece) * a.width;
    r.hot_out = a.partial + (2 * (int64_t)((p0 + hot) / kPiece) + 1) * a.width;

    using C = Cols<T, G>;
    int64_t col[C::kParts];
    int rem[C::kParts];
    bool full = true, some = false;
#pragma unroll
    for (int h = 0; h < C::kParts; ++h) {
        col[h] = ((int64_t)blockIdx.z * kSumThreads + threadIdx.x / kWave * kWave) * T::n + (h * kWave + lane) * C::kPart;
        rem[h] = (int)max((int64_t)0, min((int64_t)C::kPart, a.width - col[h]));
        full &= rem[h] == C::kPart;
        some |= rem[h] > 0;
    }
    if (full) sum_rows<T, G, kAhead, true>(a, r, rows, key, col, rem);
    else if (some) sum_rows<T, G, 2, false>(a, r, rows, key, col, rem);
}

// Joins the pieces of the long id that begins in the block of kPiece entries,
// if there is one: runs of kRun pieces, each summed by a wave of its own with
// all its loads in flight, added in order.  Piece i is there if the entry
// kPiece i past the id's first is still the id's; it lies i blocks on.  65536
// tokens, a hundred long ids: 14.6 us; with eight blocks to a workgroup 18, with
// 1024 columns to a workgroup 21.
constexpr int kRun = 16;
constexpr int kJoinRuns = 4;          // at a time
constexpr int kJoinCols = kWave * 4;
template <class G>
__global__ __launch_bounds__(kJoinRuns* kWave) void embedding_join_kernel(EmbeddingGradArgs a) {
    __shared__ __align__(16) float sums[kJoinRuns][kJoinCols];
    const int lane = lane_id(), run = threadIdx.x / kWave, here = lane * 4;
    const int32_t n = a.tokens.total();
    const int64_t block = group_index(), p = block * kPiece + lane;
    const int32_t key = p < n ? a.keys[p] : -1;
    const int32_t before = p > 0 && p < n ? a.keys[p - 1] : -1;
    const int32_t past = p + kPiece < n ? a.keys[p + kPiece] : -1;
    const uint64_t longs = __ballot(key >= 0 && key < a.vocab && before != key && past == key);
    if (!longs) return;  // alike in all waves
    const int at = (int)__builtin_ctzll(longs);
    const int32_t id = __shfl(key, at);
    const int64_t s = block * kPiece + at;
    const int64_t col = (int64_t)blockIdx.z * kJoinCols + here;
    const int rem = (int)max((int64_t)0, min((int64_t)4, a.width - col));
    float total[4] = {};
    for (int64_t base = 0;; base += kJoinRuns * kRun) {
        const int64_t q = s + (base + lane) * kPiece;
        const int pieces = __popcll(__ballot(q < n && a.keys[q < n ? q : s] == id));  // of these runs
        const int mine = max(0, min(kRun, pieces - run * kRun));
        // the first piece of all is the second kind of its block
        const float* src = a.partial + 2 * (block + base + run * kRun) * a.width + col;
        float f[kRun][4];
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            if (u < mine) {
                const float* row = src + (2 * (int64_t)u + (base + run * kRun + u == 0)) * a.width;
                if (rem == 4) F32::unpack(load16<F32>(row), f[u]);
                else
#pragma unroll
                    for (int c = 0; c < 4; ++c) f[u][c] = c < rem ? row[c] : 0.0f;
            }
        }
        float sum[4] = {};
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            if (u < mine) {
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[c] += f[u][c];
            }
        }
        *reinterpret_cast<u32x4*>(&sums[run][here]) = F32::pack(sum);
        __syncthreads();
        for (int w = 0; w < kJoinRuns && w * kRun < pieces; ++w) {
#pragma unroll
            for (int c = 0; c < 4; ++c) total[c] += sums[w][here + c];
        }
        __syncthreads();
        if (pieces < kJoinRuns * kRun) break;
    }
    if (run != 0) return;
    typename G::E* row = table_row<G>(a, id) + col;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c < rem) row[c] = G::store((a.accumulate ? G::load(row[c]) : 0.0f) + total[c] * a.scale);
}
static_assert(kJoinRuns * kRun == kWave, "one lane looks for each piece");

int bits_of(int64_t values) {
    int b = 0;
    while ((int64_t(1) << b) < values) ++b;
    return b;
}

// The sort's passes over keys in [0, vocab]: as few as the digits' width
// allows, of equal width.
void passes_of(int64_t vocab, int* passes, int* bits) {
    const int all = bits_of(vocab + 1), most = bits_of(kSortBins);
    *passes = (all + most - 1) / most;
    *bits = (all + *passes - 1) / *passes;
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// Where the gradient's workspace keeps what.
struct Layout {
    int64_t keys[2], vals[2], hist, named, partial, bytes;
};
Layout layout_of(const RankSpans& tokens, int64_t vocab, int64_t width) {
    Layout l{};
    const int64_t n = tokens.total(), list = align256(n * 4);
    if (n == 0) return l;
    l.keys[0] = 0;
    l.keys[1] = list;
    l.vals[0] = 2 * list;
    l.vals[1] = 3 * list;
    l.hist = 4 * list;
    int passes, bits;
    passes_of(vocab, &passes, &bits);
    // the first pass cuts each rank's ids into blocks of their own
    const int64_t hist = n <= kRankIds ? 0 : ((int64_t)sort_blocks(tokens).total() + 1) * (int64_t(1) << bits) * 4;
    l.named = l.hist + align256(hist);
    l.partial = l.named + align256(vocab);
    l.bytes = l.partial + (n + kPiece - 1) / kPiece * 2 * width * 4;
    return l;
}

template <class T>
int run_embedding(EmbeddingArgs a, hipStream_t s) {
    const int64_t piece = kWave * T::n * kRowVecs;
    a.chunks = (int32_t)((a.width + piece - 1) / piece);
    const int64_t items = (int64_t)a.tokens.total() * a.chunks, per = kRowThreads / kWave;
    hipLaunchKernelGGL(embedding_kernel<T>, grid_of((items + per - 1) / per), dim3(kRowThreads), 0, s, a);
    return hipGetLastError();
}

template <class T, class G>
int run_sum(EmbeddingGradArgs a, hipStream_t s) {
    const int64_t cols = kSumThreads * T::n, chunks = (a.width + cols - 1) / cols, n = a.tokens.total();
    // Shorter windows, and fewer rows to clear at once, where the longest would
    // leave the GPU idle.  Where there are twice as many summing workgroups, the
    // clearing ones come between them, so that reads and writes are under way
    // together; at odd distances, since at every second or fourth place each
    // kind would get half of the shader engines.  65536 tokens of 4096 columns
    // and 32000 rows, us a call: 281 at a distance of three, 372 at two, 294
    // with the clearing last (268 at three since rows are loaded eight ahead).
    a.window = kPiece;
    while (a.window > 4 && n / a.window * chunks < kSumGroups) a.window /= 2;
    a.windows = (int32_t)((n + a.window - 1) / a.window);
    a.fill_rows = kWave;
    while (a.fill_rows > 4 && a.vocab / a.fill_rows * chunks < kFillGroups) a.fill_rows /= 2;
    a.fill_groups = a.accumulate ? 0 : (int32_t)((a.vocab + a.fill_rows - 1) / a.fill_rows);
    const int64_t groups = (int64_t)a.windows + a.fill_groups;
    a.spacing = a.fill_groups && a.windows >= 2 * (int64_t)a.fill_groups ? (int32_t)((groups / a.fill_groups - 1) | 1) : 0;
    if (groups)
        hipLaunchKernelGGL((embedding_grad_kernel<T, G>), grid_of(groups, chunks), dim3(kSumThreads), 0, s, a);
    if (n > kPiece)
        hipLaunchKernelGGL(embedding_join_kernel<G>,
                           grid_of((n + kPiece - 1) / kPiece, (a.width + kJoinCols - 1) / kJoinCols),
                           dim3(kJoinRuns * kWave), 0, s, a);
    return hipGetLastError();
}

}  // namespace

int launch_embedding(const EmbeddingArgs& a, int dtype, void* stream) {
    return RC_BY_TYPE(run_embedding, a, static_cast<hipStream_t>(stream));
}

int64_t embedding_grad_workspace_bytes(const RankSpans& tokens, int64_t vocab, int64_t width) {
    return layout_of(tokens, vocab, width).bytes;
}

int launch_embedding_grad(EmbeddingGradArgs a, SortPass sort, int dtype, int grad_dtype, void* workspace, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int32_t n = a.tokens.total();
    const Layout l = layout_of(a.tokens, a.vocab, a.width);
    char* ws = static_cast<char*>(workspace);
    int32_t *keys[2], *vals[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = reinterpret_cast<int32_t*>(ws + l.keys[i]);
        vals[i] = reinterpret_cast<int32_t*>(ws + l.vals[i]);
    }
    int passes, bits;
    passes_of(a.vocab, &passes, &bits);
    sort.drop = 0;
    sort.named = a.accumulate || !n ? nullptr : reinterpret_cast<uint8_t*>(ws + l.named);
    a.named = sort.named;
    if (n > 0 && n <= kRankIds) {
        sort.out_keys = keys[0];
        sort.out_vals = vals[0];
        const int64_t chunks = sort.named ? (a.vocab + kNamedChunk - 1) / kNamedChunk : 0;
        const int64_t groups = std::max<int64_t>((n + kWave - 1) / kWave, std::min<int64_t>(chunks, kRankGroups));
        hipLaunchKernelGGL(sort_rank_kernel, dim3((unsigned)groups), dim3(kRankThreads), 0, s, sort);
    } else if (n > 0) {
        sort.bits = bits;
        sort.bins = 1 << bits;
        sort.hist = reinterpret_cast<int32_t*>(ws + l.hist);
        for (int p = 0; p < passes; ++p) {
            const int to = (passes - 1 - p) & 1;
            sort.shift = p * bits;
            sort.out_keys = keys[to];
            sort.out_vals = vals[to];
            if (p == 1) {  // one list from here on
                for (int r = 1; r <= kMaxRanks; ++r) sort.spans.first[r] = n;
                sort.spans.nranks = 1;
            }
            if (p >= 1) {
                sort.keys = keys[to ^ 1];
                sort.vals = vals[to ^ 1];
            }
            sort.blocks = sort_blocks(sort.spans);
            const int32_t blocks = sort.blocks.total();
            if (p == 0) launch_counts<true>(sort, s);
            else launch_counts<false>(sort, s);
            const bool last = p + 1 == passes;
            auto place = p == 0 ? (last ? sort_place_kernel<true, true> : sort_place_kernel<true, false>)
                                : (last ? sort_place_kernel<false, true> : sort_place_kernel<false, false>);
            hipLaunchKernelGGL(place, dim3(blocks), dim3(kSortThreads), 0, s, sort);
        }
    }
    a.keys = keys[0];
    a.vals = vals[0];
    a.partial = reinterpret_cast<float*>(ws + l.partial);
    if (dtype == RC_F32) return run_sum<F32, F32>(a, s);
    if (dtype == RC_F16) return grad_dtype == RC_F32 ? run_sum<F16, F32>(a, s) : run_sum<F16, F16>(a, s);
    return grad_dtype == RC_F32 ? run_sum<BF16, F32>(a, s) : run_sum<BF16, BF16>(a, s);
}

}  // namespace rc
