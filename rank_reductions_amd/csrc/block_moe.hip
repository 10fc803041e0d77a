// A mixture-of-experts layer for a few tokens.
//
// The first kernel computes silu(G x) * (U x) for every (token, expert) entry, the
// second D times that, the third the weighted sum over a token's experts.  With
// few tokens the time is that of reading the chosen experts' weights, so each
// weight is read once, by one wave, straight into the registers that the matrix
// instructions take: 16 rows of weights by 16 entries, 64 bytes of each row at a
// time.  Entries of an expert share its weights' pass; a lane's column of the
// product is one entry, so an entry's result does not hang on which others stand
// beside it.  One token of 4096 on 8 experts (302 MB of bfloat16 weights) takes 72
// us, 4.2 TB/s; 64 tokens on 64 experts in 8 bits (1.2 GB) 273 us, 4.4 TB/s; 256
// tokens, bfloat16 (2.4 GB), 550 to 583 us, 4.2 to 4.4 TB/s, where a large copy
// reaches 6.7.  A kernel that holds every token's sum for its columns does without
// the third, but reads the hidden values once for each 16 columns: 190 us in place
// of 100 for 64 tokens.
#include "blocks_impl.h"

namespace rc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4a1 __attribute__((ext_vector_type(4), aligned(1)));

struct E4M3 {
    using E = uint8_t;
    static constexpr int n = 16;
};

__device__ __forceinline__ u32x4 load_bytes(const uint8_t* p) { return *reinterpret_cast<const u32x4a1*>(p); }

// v moved down by `bytes` >= 0, zeros from above.
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int bytes) {
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    const int bits = 8 * (bytes & 7);
    if (bytes >= 16) lo = hi = 0;
    if (bytes >= 8) lo = hi, hi = 0;
    lo = lo >> bits | (bits ? hi << (64 - bits) : 0);
    hi >>= bits;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// 16 bytes of a row of `size` bytes from byte `at` on, zeros behind its end: those
// at its end moved down, without a branch unless the row is shorter.
__device__ __forceinline__ u32x4 load_end(const uint8_t* row, int at, int size) {
    if (size >= 16) {
        const int from = min(at, size - 16);
        return shift_down(load_bytes(row + from), at - from);
    }
    u32x4 v = {0, 0, 0, 0};
    for (int i = 0; i < 16 && at + i < size; ++i) v[i / 4] |= (uint32_t)row[at + i] << (8 * (i % 4));
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

// Parts bfloat16 numbers whose sum is nearest to v: two within 2^-16 of it, three
// at v itself.  Those after the first are zero where it is not finite.
template <int Parts>
__device__ __forceinline__ void as_bf16_parts(float v, uint16_t* part) {
#pragma unroll
    for (int i = 0; i < Parts; ++i) {
        const __bf16 h = (__bf16)v;
        const float f = (float)h;
        part[i] = __builtin_bit_cast(uint16_t, h);
        v = __builtin_isfinite(f) ? v - f : 0.0f;
    }
}

// The first product's step: kK elements of a row's sum, of which each of the
// four lanes that share a row takes a quarter.
template <class X, class W>
struct Up {
    static constexpr int kK = 64 / (int)sizeof(typename W::E);
    static constexpr int kX = kK / 4 * (int)sizeof(typename X::E) / 16;  // 16-byte vectors of x
    struct Frag {
        u32x4 x[kX];
    };
    __device__ __forceinline__ static f32x4 mma(u32x4 w, const Frag& f, f32x4 c) {
        const u32x4* x = f.x;
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

// The second product's: the hidden values are float32, or Parts bfloat16 each (two,
// off by a 32nd of a float16's half step at most, less of a bfloat16's; three for
// float32 outputs), and the weights taken as bfloat16 (float16 ones, of 11 bits, as the sum
// of two: hidden values may pass float16's range).
template <class W, int Parts>
struct Down {
    static constexpr int kK = 64 / (int)sizeof(typename W::E);
    static constexpr bool kWide = sizeof(typename W::E) == 4;
    static constexpr int kParts = kWide ? 1 : Parts;
    static constexpr int kH = kWide ? 1 : kK / 32;  // 16-byte vectors of one kind of hidden value
    struct Frag {
        u32x4 h[kParts][kH];
    };
    __device__ __forceinline__ static f32x4 mma(u32x4 w, const Frag& f, f32x4 c) {
        if constexpr (kWide) {
            return mma_f32(w, f.h[0][0], c);
        } else if constexpr (sizeof(typename W::E) == 1) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u32x4 v = as_bf16(w, i);
#pragma unroll
                for (int p = 0; p < Parts; ++p) c = mma_bf16(v, f.h[p][i], c);
            }
            return c;
        } else if constexpr (__is_same(W, F16)) {
            float e[8], l[8];
            F16::unpack(w, e);
            const u32x4 first = BF16::pack(e);
            float g[8];
            BF16::unpack(first, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = __builtin_isfinite(g[i]) ? e[i] - g[i] : 0.0f;
            const u32x4 second = BF16::pack(l);
            c = mma_bf16(second, f.h[0][0], mma_bf16(first, f.h[0][0], c));
            return mma_bf16(second, f.h[1][0], mma_bf16(first, f.h[1][0], c));
        } else {
            return mma_bf16(w, f.h[1][0], mma_bf16(w, f.h[0][0], c));
        }
    }
};

constexpr int kTile = 16;  // rows of weights, and entries, of a product
constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxWords = RC_MAX_EXPERTS / 32;

// An expert that entries name: its entries are list[first .. first + count).
// The first kernel writes them for the second.
struct Named {
    int32_t expert, first, count, pad;
};
__device__ __forceinline__ Named* named_of(const MoeArgs& a) { return reinterpret_cast<Named*>(a.lists); }
__device__ __forceinline__ uint16_t* list_of(const MoeArgs& a) {
    return reinterpret_cast<uint16_t*>(a.lists + sizeof(Named) * min(a.num_experts, a.entries.total()));
}

// The expert of entry i, -1 for none.
__device__ __forceinline__ int expert_of(const MoeArgs& a, int32_t i) {
    int32_t local;
    const int rank = rank_at(a.entries, i, &local);
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

// This wave's part of a sum of `steps` steps: a quarter, in multiples of `whole`.  That
// is the steps in flight of one tile of entries, also with more tiles: an entry's sum
// is cut alike however many others stand beside it.
__device__ __forceinline__ void part_of(int steps, int whole, int* s0, int* s1) {
    const int each = ((steps + kWaves - 1) / kWaves + whole - 1) / whole * whole;
    *s0 = threadIdx.x / kWave * each;
    *s1 = min(*s0 + each, steps);
}

// Sums over the steps [s0, s1) of Rows row tiles by N tiles of entries: c[row
// tile][entry tile].  A step is 64 bytes of a row of weights, of which the four
// lanes that share it take 16 each.  w: this lane's row of each row tile, of
// `size` bytes; other(n, step, frag, full): the entries' side of a step;
// zeros behind the sum's end where the step is not full.
template <class M, int Rows, int N, int Ahead, class Other>
__device__ __forceinline__ void sums_of(const uint8_t* const* w, int s0, int s1, int size, f32x4 (&c)[Rows][N], Other other) {
    const int mine = lane_id() / kTile * 16, whole = min(s1, size / 64);
    auto use = [&](const u32x4 (&v)[Rows], const typename M::Frag (&f)[N]) {
#pragma unroll
        for (int r = 0; r < Rows; ++r)
#pragma unroll
            for (int n = 0; n < N; ++n) c[r][n] = M::mma(v[r], f[n], c[r][n]);
    };
    for (int s = s0; s < whole; s += Ahead) {
        u32x4 v[Ahead][Rows];
        typename M::Frag f[Ahead][N];
#pragma unroll
        for (int j = 0; j < Ahead; ++j) {
            const int at = min(s + j, whole - 1);  // what is read twice is used once
#pragma unroll
            for (int r = 0; r < Rows; ++r) v[j][r] = load_bytes(w[r] + at * 64 + mine);
#pragma unroll
            for (int n = 0; n < N; ++n) other(n, at, f[j][n], true);
        }
#pragma unroll
        for (int j = 0; j < Ahead; ++j)
            if (s + j < whole) use(v[j], f[j]);
    }
    if (whole < s1 && s0 < s1) {  // a step that the row fills in part
        u32x4 v[Rows];
        typename M::Frag f[N];
#pragma unroll
        for (int r = 0; r < Rows; ++r) v[r] = load_end(w[r], whole * 64 + mine, size);
#pragma unroll
        for (int n = 0; n < N; ++n) other(n, whole, f[n], false);
        use(v, f);
    }
}

// ---- the same sums where an expert has many entries: the entries' side is read
// once by the workgroup, through LDS, and each of its waves has rows of its own.
constexpr int kManyWaves = 8;
constexpr int kManyThreads = kManyWaves * kWave;

// Bytes a step takes of an entry, in kPlanes rows of their own.
template <int Bytes, int Planes, int N>
struct Stage {
    static constexpr int kStage = Bytes * N > 512 ? 65536 : 32768;       // bytes of a part; two at a time
    static constexpr int kFit = kStage / (Bytes * N * kTile);
    static constexpr int kSteps = kFit >= 16 ? 16 : kFit >= 8 ? 8 : kFit >= 4 ? 4 : kFit;  // of a part
    static constexpr int kPlane = Bytes / Planes;                        // bytes of a step in a row
    static constexpr int kRow = kSteps * kPlane + 16;                    // rows 16 bytes apart in the banks
    static constexpr int kSize = kRow * Planes * N * kTile;              // of one of the two buffers
    static constexpr int kUnits = kSteps * kPlane / 16;                  // 16-byte pieces of a row
    static constexpr int kMine = kUnits * Planes * N * kTile / kManyThreads;
    // nearly as registers allow: 31 of the first kernel's are spilled with 16-bit rows
    // and 8-bit weights, 25 to 33 of the second's with 16-bit weights and 10 with
    // float32 outputs of 8-bit rows, none elsewhere
    static constexpr int kAhead = N < 8 && kSteps >= 8 ? 4 : kSteps >= 4 ? 2 : 1;
    static_assert(kSteps >= 2 && kMine * kManyThreads == kUnits * Planes * N * kTile, "parts");
};

// A barrier that waits for LDS only: what is on its way from memory stays so.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// src: the entries' rows, of `row_size` bytes, that this thread brings pieces of.  get(buffer, step of the part, n, frag): the entries'
// side of a step out of LDS.
template <class M, int Rows, int N, class S, class Get>
__device__ __forceinline__ void staged_sums(const uint8_t* const* w, int size, const uint8_t* const* src, int row_size, uint8_t* lds,
                                            f32x4 (&c)[Rows][N], Get get) {
    constexpr int kAhead = S::kAhead;
    const int mine = lane_id() / kTile * 16, whole = size / 64, steps = (size + 63) / 64;
    auto load = [&](u32x4 (&v)[kAhead][Rows], int s) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int at = min(s + j, whole - 1);  // what is read twice is used once
#pragma unroll
            for (int r = 0; r < Rows; ++r) v[j][r] = load_bytes(w[r] + at * 64 + mine);
        }
    };
    auto use_step = [&](const u32x4 (&v)[Rows], const uint8_t* from, int at) {
        typename M::Frag f[N];
#pragma unroll
        for (int n = 0; n < N; ++n) get(from, at, n, f[n]);
#pragma unroll
        for (int r = 0; r < Rows; ++r)
#pragma unroll
            for (int n = 0; n < N; ++n) c[r][n] = M::mma(v[r], f[n], c[r][n]);
    };
    auto use = [&](const u32x4 (&v)[kAhead][Rows], const uint8_t* from, int at, int s) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (s + j < whole) use_step(v[j], from, at + j);
    };
    const int unit = threadIdx.x % S::kUnits * 16;
    u32x4 held[S::kMine];
    auto fetch = [&](int part) {
        const int from = min(part * S::kUnits * 16 + unit, row_size - 16);
#pragma unroll
        for (int i = 0; i < S::kMine; ++i) held[i] = load_bytes(src[i] + from);
    };
    auto put = [&](uint8_t* to, int part) {
        const int at = part * S::kUnits * 16 + unit, behind = at - min(at, row_size - 16);
#pragma unroll
        for (int i = 0; i < S::kMine; ++i)
            *reinterpret_cast<u32x4*>(to + (threadIdx.x + i * kManyThreads) / S::kUnits * S::kRow + unit) = shift_down(held[i], behind);
    };
    u32x4 w0[kAhead][Rows], w1[kAhead][Rows];
    const int parts = (steps + S::kSteps - 1) / S::kSteps;
    fetch(0);
    load(w0, 0);
    __syncthreads();  // the buffers may still be read
    put(lds, 0);
    lds_barrier();
    for (int p = 0; p < parts; ++p) {
        const uint8_t* from = lds + (p & 1) * S::kSize;
        fetch(min(p + 1, parts - 1));
#pragma unroll
        for (int at = 0; at < S::kSteps; at += 2 * kAhead) {
            const int s = p * S::kSteps + at;
            load(w1, s + kAhead);
            use(w0, from, at, s);
            load(w0, s + 2 * kAhead);
            use(w1, from, at + kAhead, s + kAhead);
        }
        if (p + 1 < parts) put(lds + (~p & 1) * S::kSize, p + 1);
        lds_barrier();
    }
    if (whole < steps) {  // a step that the row fills in part
        u32x4 v[Rows];
#pragma unroll
        for (int r = 0; r < Rows; ++r) v[r] = load_end(w[r], whole * 64 + mine, size);
        use_step(v, lds + ((parts - 1) & 1) * S::kSize, whole - (parts - 1) * S::kSteps);
    }
}

// The hidden value of one entry and row from the two sums.
template <class X, class W>
__device__ __forceinline__ float hidden_of(const MoeArgs& a, int rank, int local, int row, float x_scale, float g, float u) {
    if (row >= a.inner) return 0.0f;  // what the second product's sum ends on
    if constexpr (sizeof(typename W::E) == 1) {
        const float* f = a.gate_up_scale[rank] + (int64_t)local * 2 * a.inner + row;
        g *= f[0];
        u *= f[a.inner];
    }
    if constexpr (sizeof(typename X::E) == 1) {
        g *= x_scale;
        u *= x_scale;
    }
    return g / (1.0f + expf(-g)) * u;
}
template <class X>
__device__ __forceinline__ float scale_of(const MoeArgs& a, int entry) {
    if constexpr (sizeof(typename X::E) > 1) return 1.0f;
    int32_t t;
    const int rank = rank_at(a.entries, entry, &t);
    return a.x_scale[rank][t / a.top_k];
}

// The p-th bfloat16 numbers of the hidden values; float32 outputs of 8-bit rows have a third.
template <class X>
constexpr int kMostParts = sizeof(typename X::E) == 1 ? 3 : 2;
__device__ __forceinline__ uint16_t* hidden_part(const MoeArgs& a, int p) { return reinterpret_cast<uint16_t*>(a.hidden + p * a.hidden_plane); }

// The hidden values of this lane's rows and entries, from the sums with G and with U.
template <class X, class W, int N>
__device__ __forceinline__ void write_hidden(const MoeArgs& a, int rank, int local, const uint16_t* list, int first, int count, int tile,
                                             const f32x4 (&c)[2][N]) {
    const int lane = lane_id(), row = tile + lane / kTile * 4;
    if (row >= a.hidden_row) return;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = first + n * kTile + lane % kTile;
        if (i >= count) continue;
        const int entry = list[i];
        const float x_scale = scale_of<X>(a, entry);
        f32x4 h;
#pragma unroll
        for (int v = 0; v < 4; ++v) h[v] = hidden_of<X, W>(a, rank, local, row + v, x_scale, c[0][n][v], c[1][n][v]);
        const int64_t to = (int64_t)entry * a.hidden_row + row;
        if constexpr (sizeof(typename W::E) == 4) {
            *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.hidden) + to) = h;
        } else {
            uint16_t part[4][kMostParts<X>];
#pragma unroll
            for (int v = 0; v < 4; ++v) as_bf16_parts<kMostParts<X>>(h[v], part[v]);
#pragma unroll
            for (int p = 0; p < kMostParts<X>; ++p)
                if (p < 2 || a.out_dtype == RC_F32)
                    *reinterpret_cast<u16x4*>(hidden_part(a, p) + to) = u16x4{part[0][p], part[1][p], part[2][p], part[3][p]};
        }
    }
}

// Where an entry's row of x begins.
template <class X>
__device__ __forceinline__ const uint8_t* row_of(const MoeArgs& a, int entry) {
    int32_t at;
    const int r = rank_at(a.entries, entry, &at);
    return static_cast<const uint8_t*>(a.x[r]) + (int64_t)(at / a.top_k) * a.width * (int)sizeof(typename X::E);
}
// This lane's row of G and of U.
template <class W>
__device__ __forceinline__ void up_rows(const MoeArgs& a, int rank, int local, int tile, const uint8_t** w) {
    const int64_t size = (int64_t)a.width * (int)sizeof(typename W::E), row = min(tile + lane_id() % kTile, a.inner - 1);
    w[0] = static_cast<const uint8_t*>(a.gate_up[rank]) + ((int64_t)local * 2 * a.inner + row) * size;
    w[1] = w[0] + a.inner * size;
}
// This lane's rows of D.
template <class W, int Rows>
__device__ __forceinline__ void down_rows(const MoeArgs& a, int rank, int local, int tile, const uint8_t** w) {
    const int64_t size = (int64_t)a.inner * (int)sizeof(typename W::E);
#pragma unroll
    for (int r = 0; r < Rows; ++r)
        w[r] = static_cast<const uint8_t*>(a.down[rank]) + ((int64_t)local * a.width + min(tile + r * kTile + lane_id() % kTile, a.width - 1)) * size;
}

// G x and U x of N tiles of entries through LDS, a tile of rows of each a wave.
template <class X, class W, int N>
__device__ __forceinline__ void up_many(const MoeArgs& a, int expert, const uint16_t* list, int first, int count, uint8_t* lds) {
    using M = Up<X, W>;
    using S = Stage<M::kX * 64, 1, N>;
    constexpr int Rows = 2, kSize = sizeof(typename X::E);
    const int lane = lane_id(), sub = lane / kTile;
    const int rank = expert / a.per_rank, local = expert - rank * a.per_rank;
    const int tile = (blockIdx.x * kManyWaves + threadIdx.x / kWave) * kTile;
    const int size = a.width * (int)sizeof(typename W::E);
    const uint8_t* w[Rows];
    up_rows<W>(a, rank, local, tile, w);
    const uint8_t* src[S::kMine];
#pragma unroll
    for (int i = 0; i < S::kMine; ++i) {
        const int row = (threadIdx.x + i * kManyThreads) / S::kUnits;
        src[i] = row_of<X>(a, list[first + row < count ? first + row : 0]);
    }
    f32x4 c[Rows][N] = {};
    staged_sums<M, Rows, N, S>(w, size, src, a.width * kSize, lds, c, [&](const uint8_t* from, int step, int n, typename M::Frag& f) {
#pragma unroll
        for (int v = 0; v < M::kX; ++v)
            f.x[v] = *reinterpret_cast<const u32x4*>(from + (n * kTile + lane % kTile) * S::kRow + step * S::kPlane + (sub * M::kX + v) * 16);
    });
    write_hidden<X, W, N>(a, rank, local, list, first, count, tile, c);
}

// G x and U x for a tile of rows of each and N tiles of entries, the sums cut over
// the workgroup's waves, then the hidden values.
template <class X, class W, int N>
__device__ __forceinline__ void up_tiles(const MoeArgs& a, int expert, const uint16_t* list, int first, int count, float* parts) {
    using M = Up<X, W>;
    constexpr int Rows = 2, kFirst = 6, kAhead = N == 4 ? 2 : N == 1 ? kFirst : 4;  // as registers allow; four: 6% slower for 16 tokens on 4 of 32
    const int lane = lane_id(), wave = threadIdx.x / kWave, sub = lane / kTile;
    const int rank = expert / a.per_rank, local = expert - rank * a.per_rank;
    const int tile = blockIdx.x * kTile;
    const int size = a.width * (int)sizeof(typename W::E), x_size = a.width * (int)sizeof(typename X::E);
    const uint8_t* w[Rows];
    up_rows<W>(a, rank, local, tile, w);
    const uint8_t* x[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {  // columns behind the last entry repeat the first, and are dropped
        const int i = first + n * kTile + lane % kTile;
        x[n] = row_of<X>(a, list[i < count ? i : 0]);
    }
    f32x4 c[Rows][N] = {};
    int s0, s1;
    part_of((size + 63) / 64, kFirst, &s0, &s1);
    sums_of<M, Rows, N, kAhead>(w, s0, s1, size, c, [&](int n, int step, typename M::Frag& f, bool full) {
        const int at = (step * 4 + sub) * M::kX * 16;
#pragma unroll
        for (int v = 0; v < M::kX; ++v) f.x[v] = full ? load_bytes(x[n] + at + v * 16) : load_end(x[n], at + v * 16, x_size);
    });
    // [wave][gate, up][entry][row]
    constexpr int kPart = N * kTile * kTile;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < Rows; ++r)
#pragma unroll
        for (int n = 0; n < N; ++n)
            *reinterpret_cast<f32x4*>(parts + (2 * wave + r) * kPart + (n * kTile + lane % kTile) * kTile + sub * 4) = c[r][n];
    __syncthreads();
    for (int at = threadIdx.x; at < kPart; at += kThreads) {
        const int i = first + at / kTile, row = tile + at % kTile;
        if (i >= count) continue;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            g += parts[(2 * v) * kPart + at];
            u += parts[(2 * v + 1) * kPart + at];
        }
        const int entry = list[i];
        const float h = hidden_of<X, W>(a, rank, local, row, scale_of<X>(a, entry), g, u);
        const int64_t to = (int64_t)entry * a.hidden_row + row;
        if constexpr (sizeof(typename W::E) == 4) {
            reinterpret_cast<float*>(a.hidden)[to] = h;
        } else {
            uint16_t part[kMostParts<X>];
            as_bf16_parts<kMostParts<X>>(h, part);
#pragma unroll
            for (int p = 0; p < kMostParts<X>; ++p)
                if (p < 2 || a.out_dtype == RC_F32) hidden_part(a, p)[to] = part[p];
        }
    }
}

// The blockIdx.y-th expert that entries name and its entries, in order (workgroups
// that share an expert's entries go by the same list); -1 if there are no more.  The
// first workgroup of each writes them for the second kernel.  The whole workgroup
// of Threads calls.
template <int Threads>
__device__ __forceinline__ int find_expert(const MoeArgs& a, uint16_t* list, int* count) {
    constexpr int kMost = RC_MAX_MOE_ENTRIES / Threads, kStrips = RC_MAX_MOE_ENTRIES / kWave;
    __shared__ uint32_t words[kMaxWords];
    __shared__ int many[kStrips], before;  // of each 64 entries
    const int32_t total = a.entries.total();
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    if (threadIdx.x < kMaxWords) words[threadIdx.x] = 0;
    if (threadIdx.x == 0) before = 0;
    __syncthreads();
    int e[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        const int32_t i = threadIdx.x + j * Threads;
        e[j] = -1;
        if (j * Threads >= total) continue;
        if (i < total) e[j] = expert_of(a, i);
        if (e[j] >= 0) atomicOr(&words[e[j] / 32], 1u << (e[j] % 32));
    }
    __syncthreads();
    const int expert = nth_expert(words, (a.num_experts + 31) / 32, blockIdx.y);
    const bool writes = blockIdx.x == 0 && blockIdx.z == 0;
    if (expert < 0) {
        if (writes && threadIdx.x == 0) named_of(a)[blockIdx.y] = Named{-1, 0, 0, 0};
        return -1;
    }
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        if (j * Threads >= total) continue;
        const uint64_t here = __ballot(e[j] == expert), less = __ballot(e[j] >= 0 && e[j] < expert);
        if (lane == 0) {
            many[j * (Threads / kWave) + wave] = __popcll(here);
            if (writes) atomicAdd(&before, __popcll(less));
        }
    }
    __syncthreads();
    const int strips = (total + Threads - 1) / Threads * (Threads / kWave);  // those that were counted
    int own = lane < strips ? many[lane] : 0, upto = own;
#pragma unroll
    for (int d = 1; d < kStrips; d *= 2) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    const int n = __builtin_amdgcn_readlane(upto, kStrips - 1);
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        if (j * Threads >= total) continue;
        const int strip = __builtin_amdgcn_readfirstlane(j * (Threads / kWave) + wave);
        const int first = __builtin_amdgcn_readlane(upto - own, strip);
        const uint64_t here = __ballot(e[j] == expert);
        if (e[j] == expert) list[first + __popcll(here & ((1ull << lane) - 1))] = (uint16_t)(threadIdx.x + j * Threads);
    }
    __syncthreads();
    if (writes) {
        if (threadIdx.x == 0) named_of(a)[blockIdx.y] = Named{expert, before, n, 0};
        for (int i = threadIdx.x; i < n; i += Threads) list_of(a)[before + i] = list[i];
    }
    *count = n;
    return expert;
}

// blockIdx.x: a tile of rows of the hidden layer; blockIdx.y: the n-th expert
// named; blockIdx.z: every gridDim.z-th 64 of many entries.
template <class X, class W>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a) {
    __shared__ uint16_t list[RC_MAX_MOE_ENTRIES];
    __shared__ __align__(16) float parts[kWaves * 2 * 4 * kTile * kTile];
    int n;
    const int expert = find_expert<kThreads>(a, list, &n);
    if (expert < 0) return;
    if (n <= 2 * kTile && blockIdx.z) return;
    if (n <= kTile) {
        up_tiles<X, W, 1>(a, expert, list, 0, n, parts);
    } else if (n <= 2 * kTile) {
        up_tiles<X, W, 2>(a, expert, list, 0, n, parts);
    } else {
        for (int first = blockIdx.z * 4 * kTile; first < n; first += gridDim.z * 4 * kTile) up_tiles<X, W, 4>(a, expert, list, first, n, parts);
    }
}

// Tiles of entries at most, nearly as registers allow.
template <class W>
constexpr int kDownMost = Down<W, 2>::kH == 2 ? 4 : 8;

// blockIdx.x: kManyWaves tiles of rows.
template <class X, class W>
__global__ __launch_bounds__(kManyThreads) void moe_up_many_kernel(MoeArgs a) {
    using M = Up<X, W>;
    __shared__ uint16_t list[RC_MAX_MOE_ENTRIES];
    __shared__ __align__(16) uint8_t lds[2 * Stage<M::kX * 64, 1, 8>::kSize];
    int n;
    const int expert = find_expert<kManyThreads>(a, list, &n);
    if (expert < 0) return;
    if (n <= kTile) {
        up_many<X, W, 1>(a, expert, list, 0, n, lds);
    } else if (n <= 2 * kTile) {
        up_many<X, W, 2>(a, expert, list, 0, n, lds);
    } else if (n <= 4 * kTile) {
        up_many<X, W, 4>(a, expert, list, 0, n, lds);
    } else {
        for (int first = 0; first < n; first += 8 * kTile) up_many<X, W, 8>(a, expert, list, first, n, lds);
    }
}

// This lane's rows of D times the hidden values of its entries.
template <class W, int Rows, int N>
__device__ __forceinline__ void write_products(const MoeArgs& a, int rank, int local, int tile, const int (&entry)[N], f32x4 (&c)[Rows][N]) {
    const int sub = lane_id() / kTile;
#pragma unroll
    for (int r = 0; r < Rows; ++r) {
        const int at = tile + r * kTile + sub * 4;
        if (at >= a.width) continue;
        if constexpr (sizeof(typename W::E) == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float scale = a.down_scale[rank][(int64_t)local * a.width + min(at + i, a.width - 1)];
#pragma unroll
                for (int n = 0; n < N; ++n) c[r][n][i] *= scale;
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n)  // a row of products has room for whole tiles
            if (entry[n] >= 0) *reinterpret_cast<f32x4*>(a.products + (int64_t)entry[n] * a.product_row + at) = c[r][n];
    }
}

// D times the hidden values of N tiles of an expert's entries, for two tiles of
// rows, the sums cut over the workgroup's waves.
template <class W, int Parts, int N>
__device__ __forceinline__ void down_tiles(const MoeArgs& a, const Named& e, int first, float* parts) {
    using M = Down<W, Parts>;
    constexpr int Rows = 2, kFirst = M::kH == 2 ? 4 : __is_same(W, F16) ? 6 : 12;  // as registers allow
    constexpr int kAhead = N == 1 ? kFirst : M::kH == 2 ? 4 / N : N == 4 ? 2 : 4;
    const int lane = lane_id(), sub = lane / kTile;
    const int rank = e.expert / a.per_rank, local = e.expert - rank * a.per_rank;
    const int wave = threadIdx.x / kWave, tile = blockIdx.x * Rows * kTile;
    const int size = a.inner * (int)sizeof(typename W::E);
    const uint8_t* w[Rows];
    down_rows<W, Rows>(a, rank, local, tile, w);
    const uint16_t* list = list_of(a) + e.first;
    const uint8_t* h[N];
    int entry[N];
    constexpr int kSize = M::kWide ? 4 : 2;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = first + n * kTile + lane % kTile;
        entry[n] = i < e.count ? list[i] : -1;
        h[n] = a.hidden + ((int64_t)list[i < e.count ? i : 0] * a.hidden_row + sub * (M::kK / 4)) * kSize;
    }
    f32x4 c[Rows][N] = {};
    int s0, s1;
    part_of((size + 63) / 64, kFirst, &s0, &s1);
    sums_of<M, Rows, N, kAhead>(w, s0, s1, size, c, [&](int n, int step, typename M::Frag& f, bool) {
#pragma unroll
        for (int v = 0; v < M::kH; ++v) {
            const uint8_t* at = h[n] + step * M::kK * kSize + v * 16;
#pragma unroll
            for (int p = 0; p < M::kParts; ++p) f.h[p][v] = *reinterpret_cast<const u32x4*>(at + p * a.hidden_plane);
        }
    });
    constexpr int kPart = Rows * N * kTile * kTile;
    __syncthreads();
    if (wave > 0) {
#pragma unroll
        for (int r = 0; r < Rows; ++r)
#pragma unroll
            for (int n = 0; n < N; ++n)
                *reinterpret_cast<f32x4*>(parts + (wave - 1) * kPart + ((r * N + n) * kWave + lane) * 4) = c[r][n];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int r = 0; r < Rows; ++r)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int v = 0; v < kWaves - 1; ++v) c[r][n] += *reinterpret_cast<f32x4*>(parts + v * kPart + ((r * N + n) * kWave + lane) * 4);
    write_products<W, Rows, N>(a, rank, local, tile, entry, c);
}

// The same through LDS, two tiles of rows a wave.
template <class W, int Parts, int N>
__device__ __forceinline__ void down_many(const MoeArgs& a, const Named& e, int first, uint8_t* lds) {
    using M = Down<W, Parts>;
    constexpr int Rows = 2, kSize = M::kWide ? 4 : 2;
    using S = Stage<64 * M::kH * M::kParts, M::kParts, N>;
    static_assert(S::kSize <= Stage<64 * M::kH * M::kParts, M::kParts, kDownMost<W>>::kSize, "the kernel's LDS");
    const int lane = lane_id(), sub = lane / kTile;
    const int rank = e.expert / a.per_rank, local = e.expert - rank * a.per_rank;
    const int tile = (blockIdx.x * kManyWaves + threadIdx.x / kWave) * Rows * kTile;
    const int size = a.inner * (int)sizeof(typename W::E);
    const uint8_t* w[Rows];
    down_rows<W, Rows>(a, rank, local, tile, w);
    const uint16_t* list = list_of(a) + e.first;
    int entry[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = first + n * kTile + lane % kTile;
        entry[n] = i < e.count ? list[i] : -1;
    }
    const uint8_t* src[S::kMine];
#pragma unroll
    for (int k = 0; k < S::kMine; ++k) {
        const int row = (threadIdx.x + k * kManyThreads) / S::kUnits, i = first + row % (N * kTile);
        src[k] = a.hidden + row / (N * kTile) * a.hidden_plane + (int64_t)list[i < e.count ? i : 0] * a.hidden_row * kSize;
    }
    f32x4 c[Rows][N] = {};
    staged_sums<M, Rows, N, S>(w, size, src, a.hidden_row * kSize, lds, c, [&](const uint8_t* from, int step, int n, typename M::Frag& f) {
#pragma unroll
        for (int v = 0; v < M::kH; ++v) {
            const uint8_t* at = from + (n * kTile + lane % kTile) * S::kRow + step * S::kPlane + (sub * M::kH + v) * 16;
#pragma unroll
            for (int p = 0; p < M::kParts; ++p) f.h[p][v] = *reinterpret_cast<const u32x4*>(at + p * N * kTile * S::kRow);
        }
    });
    write_products<W, Rows, N>(a, rank, local, tile, entry, c);
}

// blockIdx.x: two tiles of output columns; blockIdx.y: the n-th expert named.
template <class W, int Parts>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
    __shared__ __align__(16) float parts[(kWaves - 1) * 2 * 4 * kTile * kTile];
    const Named e = named_of(a)[blockIdx.y];
    if (e.expert < 0 || (e.count <= 2 * kTile && blockIdx.z)) return;
    if (e.count <= kTile) {
        down_tiles<W, Parts, 1>(a, e, 0, parts);
    } else if (e.count <= 2 * kTile) {
        down_tiles<W, Parts, 2>(a, e, 0, parts);
    } else {
        for (int first = blockIdx.z * 4 * kTile; first < e.count; first += gridDim.z * 4 * kTile) down_tiles<W, Parts, 4>(a, e, first, parts);
    }
}

// blockIdx.x: kManyWaves times two tiles of output columns.
template <class W, int Parts>
__global__ __launch_bounds__(kManyThreads) void moe_down_many_kernel(MoeArgs a) {
    using M = Down<W, Parts>;
    constexpr int kMost = kDownMost<W>;
    __shared__ __align__(16) uint8_t lds[2 * Stage<64 * M::kH * M::kParts, M::kParts, kMost>::kSize];
    const Named e = named_of(a)[blockIdx.y];
    if (e.expert < 0) return;
    if (e.count <= kTile) {
        down_many<W, Parts, 1>(a, e, 0, lds);
    } else if (e.count <= 2 * kTile) {
        down_many<W, Parts, 2>(a, e, 0, lds);
    } else if (e.count <= 4 * kTile) {
        down_many<W, Parts, 4>(a, e, 0, lds);
    } else {
        for (int first = 0; first < e.count; first += kMost * kTile) down_many<W, Parts, kMost>(a, e, first, lds);
    }
}

// Four columns of a token: the weighted sum of its experts' products, in order.
__global__ __launch_bounds__(kThreads) void moe_join_kernel(MoeArgs a) {
    const int token = blockIdx.y, column = (blockIdx.x * kThreads + threadIdx.x) * 4;
    if (column >= a.width) return;
    int32_t local;
    const int rank = rank_at(a.entries, token * a.top_k, &local);
    f32x4 y = {0, 0, 0, 0};
    constexpr int kAhead = 8;
    for (int k0 = 0; k0 < a.top_k; k0 += kAhead) {
        bool named[kAhead];
        float f[kAhead];
        f32x4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = min(k0 + j, a.top_k - 1), x = a.experts[rank][local + k];
            named[j] = k0 + j < a.top_k && x >= 0 && x < a.num_experts;
            f[j] = a.weights[rank][local + k];
            // there whether an expert is named or not
            v[j] = *reinterpret_cast<const f32x4*>(a.products + (int64_t)(token * a.top_k + k) * a.product_row + column);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = named[j] ? __builtin_fmaf(f[j], v[j][i], y[i]) : y[i];
    }
    const int64_t to = (int64_t)(local / a.top_k) * a.width + column;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (column + i >= a.width) continue;
        if (a.out_dtype == RC_F32) static_cast<float*>(a.y[rank])[to + i] = y[i];
        else if (a.out_dtype == RC_F16) static_cast<F16::E*>(a.y[rank])[to + i] = F16::store(y[i]);
        else static_cast<BF16::E*>(a.y[rank])[to + i] = BF16::store(y[i]);
    }
}

unsigned groups(int64_t n, int of) { return (unsigned)((n + of - 1) / of); }

// Through LDS where an expert has four entries or more on the average and there
// are workgroups for half of the CUs: waves that share their entries then read
// them once (64 tokens on 8 of 64 experts each, 8-bit weights: 279 us, and 352
// without; 256 tokens, bfloat16: 543 and 892; 32 on 4 of 16: 140 and 152), but wait
// for each other and are fewer (16 on 8 of 64: 383 and 362; 16 on 2 of 8: 117 and
// 74; all timed at 4096 x 1536).  Without, entries past 64 to an expert go to
// workgroups of their own (1024 tokens on two experts).  Rows have to hold one step.
template <class X, class W, int Parts = 2>
int run(const MoeArgs& a, hipStream_t s) {
    const int total = a.entries.total(), experts = min(a.num_experts, total);
    const dim3 up(groups(a.hidden_row, kManyWaves * kTile), experts), down(groups(a.width, kManyWaves * 2 * kTile), experts);
    if (total >= 4 * experts && (int)up.x * experts >= 128 && a.width >= 64 && a.inner >= 64) {
        moe_up_many_kernel<X, W><<<up, kManyThreads, 0, s>>>(a);
        moe_down_many_kernel<W, Parts><<<down, kManyThreads, 0, s>>>(a);
    } else {
        const unsigned z = groups(total, experts * 4 * kTile);
        moe_up_kernel<X, W><<<dim3(a.hidden_row / kTile, experts, z), kThreads, 0, s>>>(a);
        moe_down_kernel<W, Parts><<<dim3(groups(a.width, 2 * kTile), experts, z), kThreads, 0, s>>>(a);
    }
    moe_join_kernel<<<dim3(groups(a.width, 4 * kThreads), total / a.top_k), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int launch_moe(const MoeArgs& a, int dtype, int weight_dtype, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == RC_F32) return run<F32, F32>(a, s);
    if (dtype == RC_E4M3) return a.out_dtype == RC_F32 ? run<E4M3, E4M3, 3>(a, s) : run<E4M3, E4M3>(a, s);
    if (weight_dtype == RC_E4M3) return dtype == RC_F16 ? run<F16, E4M3>(a, s) : run<BF16, E4M3>(a, s);
    return dtype == RC_F16 ? run<F16, F16>(a, s) : run<BF16, BF16>(a, s);
}

}  // namespace rc
