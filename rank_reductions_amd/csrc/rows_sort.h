// A stable counting sort by one digit of up to kSortBins values, the shared
// base of the dispatch plan (one pass over the experts) and of the embedding
// gradient (one pass per digit of the token ids).
//
// Launches: digit counts of each block of kSortBlock entries, and the places -
// an entry's place is the start of its digit, plus the entries of that digit
// in earlier blocks, earlier waves of the block, earlier strips of the wave
// and lower lanes.  The lanes of a strip that hold the same digit find each
// other with one ballot per digit bit.  While blocks * digits stay under
// kFusedCounts every block adds the blocks before it up by itself; a launch
// between the two does so beyond.  Counts are integers, so atomics on them do
// not touch the order, which is the entries' own.
//
// Bound by latency, not by bytes: a launch and two or three dependent loads
// each.  Blocks of 1024 entries rather than 4096, all loads of a lane issued
// together and no scan launch between took the plan of 131072 entries over 64
// experts from 35.5 us to 16.6 us, the two passes over 65536 ids from 62 us to
// 34 us.
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

// This workgroup's share of clearing s.named (16-byte aligned, and padded to 16).
__device__ __forceinline__ void clear_named(const SortPass& s, int64_t group, int64_t groups, int threads) {
    u32x4* at = reinterpret_cast<u32x4*>(s.named);
    for (int64_t i = group * threads + threadIdx.x; i < (s.key_limit + 15) / 16; i += groups * threads) at[i] = u32x4{0, 0, 0, 0};
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortPass s) {
    __shared__ int32_t count[kSortBins];
    int32_t block;
    const int rank = rank_of(s.blocks, blockIdx.x, &block);
    int32_t key[kStrips];
#pragma unroll
    for (int k = 0; k < kStrips; ++k) {
        int32_t val;
        if (!sort_entry<FIRST>(s, rank, block, k * kSortThreads + threadIdx.x, &key[k], &val)) key[k] = -1;
    }
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) count[d] = 0;
    if (FIRST && s.named) clear_named(s, blockIdx.x, gridDim.x, kSortThreads);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStrips; ++k)
        if (key[k] >= 0 && !(s.drop && key[k] == s.key_limit)) atomicAdd(&count[(key[k] >> s.shift) & ((1 << s.bits) - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < s.bins; d += kSortThreads) s.hist[(int64_t)blockIdx.x * s.bins + d] = count[d];
}

// Up to this many counts, each block adds them up itself: at 16384 a lane
// reads 64 of them, 32 at a time; the launch between took 4.7 us.
constexpr int64_t kFusedCounts = 16384;
constexpr int kBatch = 32;

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
    if (d < bins) {
#pragma unroll 8
        for (int b = lo; b < hi; ++b) sum += hist[(int64_t)b * bins + d];
    }
    part[wave][lane] = sum;
    __syncthreads();
    if (d >= bins) return;
    int32_t run = 0;
    for (int w = 0; w < wave; ++w) run += part[w][lane];
    for (int b0 = lo; b0 < hi; b0 += kBatch) {
        int32_t c[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) c[u] = b0 + u < hi ? hist[(int64_t)(b0 + u) * bins + d] : 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (b0 + u < hi) hist[(int64_t)(b0 + u) * bins + d] = run;
            run += c[u];
        }
    }
    if (wave == kScanWaves - 1) hist[(int64_t)blocks * bins + d] = run;
}

// Entries of a digit in the blocks before this one, and in all, for the digits
// that a thread looks after: held in registers until add() puts them into LDS,
// so that their loads are under way together with the block's keys (a barrier
// waits for every load before it).
struct BlockSums {
    static constexpr int kDigits = kSortBins / kSortThreads;
    int32_t lower[kDigits], all[kDigits];
    int width;  // threads per set of digits; the sets share out the blocks

    __device__ __forceinline__ void load(const SortPass& s) {
        const int32_t blocks = s.blocks.first[kMaxRanks], me = blockIdx.x;
        width = 1;
        while (width < s.bins && width < kSortThreads) width *= 2;
        const int parts = kSortThreads / width, part = threadIdx.x / width;
#pragma unroll
        for (int i = 0; i < kDigits; ++i) {
            lower[i] = all[i] = 0;
            const int d = (threadIdx.x & (width - 1)) + i * width;
            if (d >= s.bins) continue;
            if (s.scanned) {
                if (part == 0) {
                    lower[i] = s.hist[(int64_t)me * s.bins + d];
                    all[i] = s.hist[(int64_t)blocks * s.bins + d];
                }
                continue;
            }
            for (int b0 = part; b0 < blocks; b0 += parts * kBatch) {
                int32_t c[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int b = b0 + u * parts;
                    c[u] = b < blocks ? s.hist[(int64_t)b * s.bins + d] : 0;
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    all[i] += c[u];
                    lower[i] += b0 + u * parts < me ? c[u] : 0;
                }
            }
        }
    }
    // before[d] and total[d], cleared; a barrier is due on both sides.
    __device__ __forceinline__ void add(const SortPass& s, int32_t* before, int32_t* total) const {
#pragma unroll
        for (int i = 0; i < kDigits; ++i) {
            const int d = (threadIdx.x & (width - 1)) + i * width;
            if (d >= s.bins) continue;
            atomicAdd(&before[d], lower[i]);
            atomicAdd(&total[d], all[i]);
        }
    }
};

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

// Runs the counting half of a pass (and the sums between, where they are a
// launch of their own).  s.blocks, bins, bits and shift are set.
template <bool FIRST>
void launch_counts(SortPass& s, hipStream_t stream) {
    const int32_t blocks = s.blocks.total();
    hipLaunchKernelGGL(sort_count_kernel<FIRST>, dim3(blocks), dim3(kSortThreads), 0, stream, s);
    s.scanned = (int64_t)blocks * s.bins > kFusedCounts;
    if (s.scanned)
        hipLaunchKernelGGL(sort_scan_kernel, dim3((s.bins + kWave - 1) / kWave), dim3(kScanWaves * kWave), 0, stream,
                           s.hist, blocks, s.bins);
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
