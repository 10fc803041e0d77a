// A stable counting sort by one digit of up to kSortBins values, the shared
// base of the dispatch plan (one pass over the experts) and of the embedding
// gradient (one pass per digit of the token ids).
//
// Three launches: digit counts of each block of kSortBlock entries, an
// exclusive sum over the blocks for each digit, and the places - an entry's
// place is the start of its digit, plus the entries of that digit in earlier
// blocks, earlier waves of the block, earlier strips of the wave and lower
// lanes.  The lanes of a strip that hold the same digit find each other with
// one ballot per digit bit.  Counts are integers, so atomics on them do not
// touch the order, which is the entries' own.
#pragma once

#include "rows_impl.h"

namespace rc {
namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kStrips = kSortBlock / kSortThreads;  // strips of 64 entries per wave

// Key of entry i of rank r in the first pass: ids outside [0, limit) sort last.
__device__ __forceinline__ int32_t first_key(const SortPass& s, int r, int32_t i) {
    const int64_t id = s.id64 ? static_cast<const int64_t*>(s.ids[r])[i] : (int64_t) static_cast<const int32_t*>(s.ids[r])[i];
    return id >= 0 && id < s.key_limit ? (int32_t)id : (int32_t)s.key_limit;
}

// Entry `at` of block `block`: its key, and its value (position in the
// sequence of all ranks' entries).  False past the block's entries.
template <bool FIRST>
__device__ __forceinline__ bool sort_entry(const SortPass& s, int rank, int32_t block, int at, int32_t* key, int32_t* val) {
    const int32_t i = block * kSortBlock + at;  // within the rank's entries
    if (i < 0 || i >= s.spans.first[rank + 1] - s.spans.first[rank]) return false;
    if (FIRST) {
        *key = first_key(s, rank, i);
        *val = s.spans.first[rank] + i;
    } else {
        *key = s.keys[i];
        *val = s.vals[i];
    }
    return true;
}

// Lanes of the wave whose digit is this lane's (0 for a lane without one).
__device__ __forceinline__ uint64_t same_digit(int digit, int bits, bool has) {
    uint64_t mask = __ballot(has);
    for (int b = 0; b < bits; ++b) {
        const bool one = (digit >> b) & 1;
        const uint64_t m = __ballot(one);
        mask &= one ? m : ~m;
    }
    return has ? mask : 0;
}

__device__ __forceinline__ void wave_sync() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); __builtin_amdgcn_wave_barrier(); }

// Position of this lane's entry among those of its digit that the wave has
// met, counting from count[digit], which moves on by the strip's.
__device__ __forceinline__ int32_t strip_rank(int digit, int bits, bool has, volatile int32_t* count) {
    const uint64_t mask = same_digit(digit, bits, has);
    const int below = __popcll(mask & ((1ull << lane_id()) - 1));
    const int32_t base = has ? count[digit] : 0;
    wave_sync();
    if (has && below == 0) count[digit] = base + __popcll(mask);
    wave_sync();
    return base + below;
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortPass s) {
    __shared__ int32_t count[kSortBins];
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) count[d] = 0;
    __syncthreads();
    int32_t block;
    const int rank = rank_of(s.blocks, blockIdx.x, &block);
    for (int k = 0; k < kStrips; ++k) {
        int32_t key, val;
        if (sort_entry<FIRST>(s, rank, block, k * kSortThreads + threadIdx.x, &key, &val) &&
            !(s.drop && key == s.key_limit))
            atomicAdd(&count[(key >> s.shift) & ((1 << s.bits) - 1)], 1);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) s.hist[(int64_t)blockIdx.x * s.bins + d] = count[d];
}

// Exclusive sums over the blocks, for 64 digits per workgroup; the totals
// follow the last block's row.
constexpr int kScanWaves = 16;
__global__ __launch_bounds__(kScanWaves* kWave) void sort_scan_kernel(int32_t* hist, int32_t blocks, int32_t bins) {
    __shared__ int32_t part[kScanWaves][kWave];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int d = blockIdx.x * kWave + lane;
    const int per = (blocks + kScanWaves - 1) / kScanWaves;
    const int lo = min(wave * per, blocks), hi = min(lo + per, blocks);
    int32_t sum = 0;
    if (d < bins)
        for (int b = lo; b < hi; ++b) sum += hist[(int64_t)b * bins + d];
    part[wave][lane] = sum;
    __syncthreads();
    if (d >= bins) return;
    int32_t run = 0;
    for (int w = 0; w < wave; ++w) run += part[w][lane];
    for (int b = lo; b < hi; ++b) {
        const int32_t c = hist[(int64_t)b * bins + d];
        hist[(int64_t)b * bins + d] = run;
        run += c;
    }
    if (wave == kScanWaves - 1) hist[(int64_t)blocks * bins + d] = run;
}

// In-place exclusive sum of v[0..bins) by a workgroup of THREADS; `carry`
// holds one word per wave.
template <int THREADS>
__device__ __forceinline__ void exclusive_sum(int32_t* v, int bins, int32_t* carry) {
    constexpr int kPer = (kSortBins + THREADS - 1) / THREADS;
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    int32_t own[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int d = threadIdx.x * kPer + i;
        own[i] = d < bins ? v[d] : 0;
        sum += own[i];
    }
    int32_t incl = sum;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int32_t up = __shfl_up(incl, o);
        incl += lane >= o ? up : 0;
    }
    if (lane == kWave - 1) carry[wave] = incl;
    __syncthreads();
    int32_t before = incl - sum;
    for (int w = 0; w < wave; ++w) before += carry[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int d = threadIdx.x * kPer + i;
        if (d < bins) v[d] = before;
        before += own[i];
    }
    __syncthreads();
}

// Counts of each wave's digits: count[w][d] over the wave's own contiguous
// strips, then turned into the block-wide exclusive start of (w, d) on top of
// base[d].
template <int WAVES>
__device__ __forceinline__ void wave_starts(int32_t* count, const int32_t* base, int bins) {
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += WAVES * kWave) {
        int32_t run = base[d];
        for (int w = 0; w < WAVES; ++w) {
            const int32_t c = count[w * kSortBins + d];
            count[w * kSortBins + d] = run;
            run += c;
        }
    }
    __syncthreads();
}

}  // namespace
}  // namespace rc
