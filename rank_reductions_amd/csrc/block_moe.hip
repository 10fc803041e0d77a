// A mixture-of-experts layer for a few tokens in two kernels.
//
// The first computes silu(G x) * (U x) for every (token, expert) entry, the
// second D times that and the weighted sum over a token's experts.  With few
// tokens the time is that of reading the chosen experts' weights, so each weight
// is read once, by one wave, straight into the registers that the matrix
// instructions take: 16 rows of weights by 16 entries, sums over 16 bytes a lane
// and row at a time.  Entries of an expert share its weights' pass; a lane's
// column of the product is one entry, so an entry's result does not hang on which
// others stand beside it.
#include "blocks_impl.h"

namespace rc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4a1 __attribute__((ext_vector_type(4), aligned(1)));

struct E4M3 {
    using E = uint8_t;
    static constexpr int n = 16;
};

// 16 bytes of a row from element k on; with Full all are there, else zeros
// from element `count` on.
template <class T, bool Full>
__device__ __forceinline__ u32x4 load_row(const typename T::E* row, int k, int count) {
    constexpr int n = 16 / sizeof(typename T::E), per = n / 4;
    if (Full || k + n <= count) return *reinterpret_cast<const u32x4a1*>(row + k);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < n; ++i) {
        if (k + i >= count) continue;
        const typename T::E e = row[k + i];
        uint32_t u;
        if constexpr (sizeof(e) == 4) u = __builtin_bit_cast(uint32_t, e);
        else if constexpr (sizeof(e) == 2) u = __builtin_bit_cast(uint16_t, e);
        else u = e;
        v[i / per] |= u << (8 * sizeof(e) * (i % per));
    }
    return v;
}

__device__ __forceinline__ f32x4 mma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma_f16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma_f32(u32x4 a, u32x4 b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = a[i], q = b[i];
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, p), __builtin_bit_cast(float, q), c, 0, 0, 0);
    }
    return c;
}
// Half of 16 e4m3 values by half of 16 others.
__device__ __forceinline__ f32x4 mma_e4m3(u32x4 a, u32x4 b, int half, f32x4 c) {
    const uint64_t p = (uint64_t)a[2 * half + 1] << 32 | a[2 * half], q = (uint64_t)b[2 * half + 1] << 32 | b[2 * half];
    return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8((long)p, (long)q, c, 0, 0, 0);
}
// Half of 16 e4m3 values as eight 16-bit ones, which hold them exactly.
__device__ __forceinline__ u32x4 as_bf16(u32x4 v, int half) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[2 * half + i / 2];
        const bf16x2 p = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
        o[i] = __builtin_bit_cast(uint32_t, p);
    }
    return o;
}
__device__ __forceinline__ u32x4 as_f16(u32x4 v, int half) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[2 * half + i / 2];
        const f16x2 p = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
        o[i] = __builtin_bit_cast(uint32_t, p);
    }
    return o;
}

// The two bfloat16 numbers whose sum is nearest to v (within 2^-16 of it); the
// second is zero where the first is not finite.
__device__ __forceinline__ void two_bf16(float v, uint16_t* hi, uint16_t* lo) {
    const __bf16 h = (__bf16)v;
    const float f = (float)h;
    *hi = __builtin_bit_cast(uint16_t, h);
    *lo = __builtin_bit_cast(uint16_t, (__bf16)(__builtin_isfinite(f) ? v - f : 0.0f));
}

// The first product's step: kK elements of a row's sum, of which each of the
// four lanes that share a row takes a quarter.
template <class X, class W>
struct Up {
    static constexpr int kK = 64 / (int)sizeof(typename W::E);
    static constexpr int kX = kK / 4 * (int)sizeof(typename X::E) / 16;  // 16-byte vectors of x
    __device__ __forceinline__ static f32x4 mma(u32x4 w, const u32x4* x, f32x4 c) {
        if constexpr (sizeof(typename W::E) == 4) {
            return mma_f32(w, x[0], c);
        } else if constexpr (sizeof(typename X::E) == 1) {
            return mma_e4m3(w, x[0], 1, mma_e4m3(w, x[0], 0, c));
        } else if constexpr (sizeof(typename W::E) == 1) {
            if constexpr (__is_same(X, F16)) return mma_f16(as_f16(w, 1), x[1], mma_f16(as_f16(w, 0), x[0], c));
            else return mma_bf16(as_bf16(w, 1), x[1], mma_bf16(as_bf16(w, 0), x[0], c));
        } else if constexpr (__is_same(X, F16)) {
            return mma_f16(w, x[0], c);
        } else {
            return mma_bf16(w, x[0], c);
        }
    }
};

// The second product's: the hidden values are float32, or two bfloat16 each,
// and the weights taken as bfloat16 (float16 ones, of 11 bits, as the sum of two).
template <class W>
struct Down {
    static constexpr int kK = 64 / (int)sizeof(typename W::E);
    static constexpr bool kWide = sizeof(typename W::E) == 4;
    static constexpr int kH = kWide ? 1 : kK / 32;  // 16-byte vectors of one kind of hidden value
    __device__ __forceinline__ static f32x4 mma(u32x4 w, const u32x4* hi, const u32x4* lo, f32x4 c) {
        if constexpr (kWide) {
            return mma_f32(w, hi[0], c);
        } else if constexpr (sizeof(typename W::E) == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 v = as_bf16(w, h);
                c = mma_bf16(v, lo[h], mma_bf16(v, hi[h], c));
            }
            return c;
        } else if constexpr (__is_same(W, F16)) {
            float f[8], l[8];
            F16::unpack(w, f);
            const u32x4 first = BF16::pack(f);
            float g[8];
            BF16::unpack(first, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = __builtin_isfinite(g[i]) ? f[i] - g[i] : 0.0f;
            return mma_bf16(first, lo[0], mma_bf16(BF16::pack(l), hi[0], mma_bf16(first, hi[0], c)));
        } else {
            return mma_bf16(w, lo[0], mma_bf16(w, hi[0], c));
        }
    }
};

constexpr int kTile = 16;   // rows of weights, and entries, of a product
constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;
constexpr int kMaxWords = RC_MAX_EXPERTS / 32;

// The expert of entry i, -1 for none.
__device__ __forceinline__ int expert_of(const MoeArgs& a, int32_t i) {
    int32_t local;
    const int rank = rank_of(a.entries, i, &local);
    const int e = a.experts[rank][local];
    return e >= 0 && e < a.num_experts ? e : -1;
}

// The `which`-th expert that some entry names, -1 if there are no more: `words`
// has a bit for each expert.  The whole wave calls.
__device__ __forceinline__ int nth_expert(const uint32_t* words, int num_words, int which) {
    const int lane = lane_id();
    uint32_t w = lane < num_words ? words[lane] : 0;
    const int own = __popc(w);
    int upto = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    const uint64_t here = __ballot(which < upto && which >= upto - own);
    if (!here) return -1;
    const int at = __ffsll((unsigned long long)here) - 1;
    int left = which - (upto - own);
    for (; left > 0; --left) w &= w - 1;
    return __builtin_amdgcn_readlane(lane * 32 + __ffs((int)w) - 1, __builtin_amdgcn_readfirstlane(at));
}

// G x and U x for kTile rows of each and N tiles of entries, the sum cut over the
// workgroup's waves; then the waves' parts added and the hidden values written.
template <class X, class W, int N>
__device__ __forceinline__ void up_tiles(const MoeArgs& a, int expert, const uint16_t* list, int first, int count, float* parts) {
    using M = Up<X, W>;
    constexpr int kAhead = N == 4 ? 2 : 4;
    const int lane = lane_id(), wave = threadIdx.x / kWave, sub = lane / kTile;
    const int rank = expert / a.per_rank, local = expert - rank * a.per_rank;
    const int tile = blockIdx.x * kTile, row = min(tile + lane % kTile, a.inner - 1);
    const int64_t K = a.width;
    const typename W::E* gate = (const typename W::E*)a.gate_up[rank] + ((int64_t)local * 2 * a.inner + row) * K;
    const typename W::E* up = gate + a.inner * K;
    const typename X::E* x[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = first + n * kTile + lane % kTile;
        int32_t at;  // columns behind the last entry repeat the first, and are dropped
        const int r = rank_of(a.entries, list[i < count ? i : 0], &at);
        x[n] = (const typename X::E*)a.x[r] + (int64_t)(at / a.top_k) * K;
    }
    f32x4 g[N] = {}, u[N] = {};
    const int steps = ((int)K + M::kK - 1) / M::kK, whole = (int)K / M::kK, each = (steps + kUpWaves - 1) / kUpWaves;
    const int s0 = wave * each, s1 = min(s0 + each, steps), full = min(s1, whole);
    const int mine = sub * (M::kK / 4);
    int s = s0;
    for (; s + kAhead <= full; s += kAhead) {
        u32x4 wg[kAhead], wu[kAhead], xv[kAhead][N][M::kX];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = (s + j) * M::kK + mine;
            wg[j] = load_row<W, true>(gate, k, 0);
            wu[j] = load_row<W, true>(up, k, 0);
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int v = 0; v < M::kX; ++v) xv[j][n][v] = load_row<X, true>(x[n], k + v * 16 / (int)sizeof(typename X::E), 0);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                g[n] = M::mma(wg[j], xv[j][n], g[n]);
                u[n] = M::mma(wu[j], xv[j][n], u[n]);
            }
    }
    for (; s < s1; ++s) {
        const int k = s * M::kK + mine;
        const u32x4 wg = load_row<W, false>(gate, k, (int)K), wu = load_row<W, false>(up, k, (int)K);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            u32x4 xv[M::kX];
#pragma unroll
            for (int v = 0; v < M::kX; ++v) xv[v] = load_row<X, false>(x[n], k + v * 16 / (int)sizeof(typename X::E), (int)K);
            g[n] = M::mma(wg, xv, g[n]);
            u[n] = M::mma(wu, xv, u[n]);
        }
    }
    // [wave][gate, up][entry][row]
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int at = (n * kTile + lane % kTile) * kTile + sub * 4;
        *reinterpret_cast<f32x4*>(parts + (2 * wave) * N * kTile * kTile + at) = g[n];
        *reinterpret_cast<f32x4*>(parts + (2 * wave + 1) * N * kTile * kTile + at) = u[n];
    }
    __syncthreads();
    for (int at = threadIdx.x; at < N * kTile * kTile; at += kUpWaves * kWave) {
        const int i = first + at / kTile, r = tile + at % kTile;
        if (i >= count) continue;
        float gs = 0.0f, us = 0.0f;
#pragma unroll
        for (int w = 0; w < kUpWaves; ++w) {
            gs += parts[(2 * w) * N * kTile * kTile + at];
            us += parts[(2 * w + 1) * N * kTile * kTile + at];
        }
        const int entry = list[i];
        float h = 0.0f;  // behind the last row: what the second product's sum ends on
        if (r < a.inner) {
            if constexpr (sizeof(typename W::E) == 1) {
                const float* f = a.gate_up_scale[rank] + (int64_t)local * 2 * a.inner + r;
                gs *= f[0];
                us *= f[a.inner];
            }
            if constexpr (sizeof(typename X::E) == 1) {
                int32_t t;
                const int xr = rank_of(a.entries, entry, &t);
                const float f = a.x_scale[xr][t / a.top_k];
                gs *= f;
                us *= f;
            }
            h = gs / (1.0f + expf(-gs)) * us;
        }
        const int64_t to = (int64_t)entry * a.hidden_row + r;
        if constexpr (sizeof(typename W::E) == 4) {
            reinterpret_cast<float*>(a.hidden)[to] = h;
        } else {
            two_bf16(h, reinterpret_cast<uint16_t*>(a.hidden) + to, reinterpret_cast<uint16_t*>(a.hidden + a.hidden_plane) + to);
        }
    }
}

// blockIdx.x: kTile rows of the hidden layer; blockIdx.y: the n-th expert named.
template <class X, class W>
__global__ __launch_bounds__(kUpWaves * kWave) void moe_up_kernel(MoeArgs a) {
    __shared__ uint32_t words[kMaxWords];
    __shared__ uint16_t list[RC_MAX_MOE_ENTRIES];
    __shared__ int count;
    __shared__ float parts[kUpWaves * 2 * 4 * kTile * kTile];
    constexpr int kThreads = kUpWaves * kWave, kMost = RC_MAX_MOE_ENTRIES / kThreads;
    const int32_t total = a.entries.total();
    const int num_words = (a.num_experts + 31) / 32;
    if (threadIdx.x < kMaxWords) words[threadIdx.x] = 0;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    int e[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        const int32_t i = threadIdx.x + j * kThreads;
        e[j] = i < total ? expert_of(a, i) : -1;
        if (e[j] >= 0) atomicOr(&words[e[j] / 32], 1u << (e[j] % 32));
    }
    __syncthreads();
    const int expert = nth_expert(words, num_words, blockIdx.y);
    if (expert < 0) return;
#pragma unroll
    for (int j = 0; j < kMost; ++j)  // in any order
        if (e[j] == expert) list[atomicAdd(&count, 1)] = (uint16_t)(threadIdx.x + j * kThreads);
    __syncthreads();
    const int n = __builtin_amdgcn_readfirstlane(count);
    if (n <= kTile) {
        up_tiles<X, W, 1>(a, expert, list, 0, n, parts);
    } else if (n <= 2 * kTile) {
        up_tiles<X, W, 2>(a, expert, list, 0, n, parts);
    } else {
        for (int first = 0; first < n; first += 4 * kTile) up_tiles<X, W, 4>(a, expert, list, first, n, parts);
    }
}

// One part of D times the hidden values of N tiles of an expert's entries, into
// `sums` ([entry][row]).
template <class W, int N>
__device__ __forceinline__ void down_tiles(const MoeArgs& a, int expert, const uint16_t* list, int first, int count, int s0, int s1,
                                           float* sums) {
    using M = Down<W>;
    constexpr int kAhead = N == 4 ? 2 : N == 2 ? 4 : 8;
    const int lane = lane_id(), sub = lane / kTile;
    const int rank = expert / a.per_rank, local = expert - rank * a.per_rank;
    const int tile = blockIdx.x * kTile, row = min(tile + lane % kTile, a.width - 1);
    const int64_t K = a.inner;
    const typename W::E* down = (const typename W::E*)a.down[rank] + ((int64_t)local * a.width + row) * K;
    const uint8_t* h[N];
    int entry[N];
    constexpr int kSize = M::kWide ? 4 : 2;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = first + n * kTile + lane % kTile;
        entry[n] = i < count ? list[i] : -1;
        h[n] = a.hidden + ((int64_t)list[i < count ? i : 0] * a.hidden_row + sub * (M::kK / 4)) * kSize;
    }
    f32x4 c[N] = {};
    const int full = min(s1, (int)K / M::kK), mine = sub * (M::kK / 4);
    int s = s0;
    auto hidden = [&](int n, int step, u32x4* hi, u32x4* lo) {
#pragma unroll
        for (int v = 0; v < M::kH; ++v) {
            const uint8_t* p = h[n] + (int64_t)step * M::kK * kSize + v * 16;
            hi[v] = *reinterpret_cast<const u32x4*>(p);
            if constexpr (!M::kWide) lo[v] = *reinterpret_cast<const u32x4*>(p + a.hidden_plane);
        }
    };
    for (; s + kAhead <= full; s += kAhead) {
        u32x4 w[kAhead], hi[kAhead][N][M::kH], lo[kAhead][N][M::kH];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) w[j] = load_row<W, true>(down, (s + j) * M::kK + mine, 0);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int n = 0; n < N; ++n) hidden(n, s + j, hi[j][n], lo[j][n]);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int n = 0; n < N; ++n) c[n] = M::mma(w[j], hi[j][n], lo[j][n], c[n]);
    }
    for (; s < s1; ++s) {
        const u32x4 w = load_row<W, false>(down, s * M::kK + mine, (int)K);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            u32x4 hi[M::kH], lo[M::kH];
            hidden(n, s, hi, lo);
            c[n] = M::mma(w, hi, lo, c[n]);
        }
    }
    f32x4 scale = {1, 1, 1, 1};
    if constexpr (sizeof(typename W::E) == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) scale[i] = a.down_scale[rank][(int64_t)local * a.width + min(tile + sub * 4 + i, a.width - 1)];
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (entry[n] >= 0) *reinterpret_cast<f32x4*>(sums + entry[n] * kTile + sub * 4) = c[n] * scale;
}

// blockIdx.x: kTile columns of the output, for all tokens.
template <class W>
__global__ __launch_bounds__(kDownWaves * kWave) void moe_down_kernel(MoeArgs a) {
    extern __shared__ float sums[];  // [part][entry][column]
    __shared__ int start[RC_MAX_EXPERTS];
    __shared__ int many[RC_MAX_EXPERTS];
    __shared__ uint16_t list[RC_MAX_MOE_ENTRIES], named[RC_MAX_EXPERTS];
    __shared__ int carry[2][kDownWaves];
    constexpr int kThreads = kDownWaves * kWave, kMost = RC_MAX_MOE_ENTRIES / kThreads, kEach = RC_MAX_EXPERTS / kThreads;
    const int32_t total = a.entries.total();
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    // a counting sort of the entries by their expert
#pragma unroll
    for (int j = 0; j < kEach; ++j) many[threadIdx.x + j * kThreads] = 0;
    __syncthreads();
    int e[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        const int32_t i = threadIdx.x + j * kThreads;
        e[j] = i < total ? expert_of(a, i) : -1;
        if (e[j] >= 0) atomicAdd(&many[e[j]], 1);
    }
    __syncthreads();
    int own[kEach], sum = 0, some = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        own[j] = many[threadIdx.x * kEach + j];
        sum += own[j];
        some += own[j] > 0;
    }
    int before = sum, first = some;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int v = __shfl_up(before, d), w = __shfl_up(first, d);
        if (lane >= d) before += v, first += w;
    }
    if (lane == kWave - 1) carry[0][wave] = before, carry[1][wave] = first;
    __syncthreads();
    int experts = 0;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) {
        if (w < wave) before += carry[0][w], first += carry[1][w];
        experts += carry[1][w];
    }
    before -= sum;
    first -= some;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        start[threadIdx.x * kEach + j] = before;
        before += own[j];
        if (own[j]) named[first++] = (uint16_t)(threadIdx.x * kEach + j);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMost; ++j)  // within an expert in any order; start ends as each expert's end
        if (e[j] >= 0) list[atomicAdd(&start[e[j]], 1)] = (uint16_t)(threadIdx.x + j * kThreads);
    __syncthreads();
    // experts, or parts of their sums where they are few, to the waves in turn
    using M = Down<W>;
    const int steps = (a.inner + M::kK - 1) / M::kK;
    const int splits = experts ? max(1, min(min(a.splits, steps), (4 * kDownWaves + experts - 1) / experts)) : 1;
    const int each = (steps + splits - 1) / splits;
    for (int item = wave; item < experts * splits; item += kDownWaves) {
        const int expert = __builtin_amdgcn_readfirstlane(named[item / splits]), part = item % splits;
        const int n = __builtin_amdgcn_readfirstlane(many[expert]), s0 = part * each, s1 = min(s0 + each, steps);
        const uint16_t* mine = list + start[expert] - n;
        float* to = sums + part * total * kTile;
        if (n <= kTile) {
            down_tiles<W, 1>(a, expert, mine, 0, n, s0, s1, to);
        } else if (n <= 2 * kTile) {
            down_tiles<W, 2>(a, expert, mine, 0, n, s0, s1, to);
        } else {
            for (int f = 0; f < n; f += 4 * kTile) down_tiles<W, 4>(a, expert, mine, f, n, s0, s1, to);
        }
    }
    __syncthreads();
    const int tokens = total / a.top_k;
    for (int at = threadIdx.x; at < tokens * kTile; at += kThreads) {
        const int token = at / kTile, column = blockIdx.x * kTile + at % kTile;
        if (column >= a.width) continue;
        int32_t local;
        const int rank = rank_of(a.entries, token * a.top_k, &local);
        float y = 0.0f;
        for (int k = 0; k < a.top_k; ++k) {
            const int x = a.experts[rank][local + k];
            if (x < 0 || x >= a.num_experts) continue;
            float v = 0.0f;
            for (int p = 0; p < splits; ++p) v += sums[(p * total + token * a.top_k + k) * kTile + at % kTile];
            y = __builtin_fmaf(a.weights[rank][local + k], v, y);
        }
        const int64_t to = (int64_t)(local / a.top_k) * a.width + column;
        if (a.out_dtype == RC_F32) static_cast<float*>(a.y[rank])[to] = y;
        else if (a.out_dtype == RC_F16) static_cast<F16::E*>(a.y[rank])[to] = F16::store(y);
        else static_cast<BF16::E*>(a.y[rank])[to] = BF16::store(y);
    }
}

template <class X, class W>
int run(const MoeArgs& a, hipStream_t s) {
    const int experts = a.num_experts < a.entries.total() ? a.num_experts : a.entries.total();
    moe_up_kernel<X, W><<<dim3(a.hidden_row / kTile, experts), kUpWaves * kWave, 0, s>>>(a);
    const size_t lds = (size_t)a.splits * a.entries.total() * kTile * sizeof(float);
    moe_down_kernel<W><<<(a.width + kTile - 1) / kTile, kDownWaves * kWave, lds, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int launch_moe(const MoeArgs& a, int dtype, int weight_dtype, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == RC_F32) return run<F32, F32>(a, s);
    if (dtype == RC_E4M3) return run<E4M3, E4M3>(a, s);
    if (weight_dtype == RC_E4M3) return dtype == RC_F16 ? run<F16, E4M3>(a, s) : run<BF16, E4M3>(a, s);
    return dtype == RC_F16 ? run<F16, F16>(a, s) : run<BF16, BF16>(a, s);
}

}  // namespace rc
