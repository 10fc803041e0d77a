// Gradient norms and the AdamW step of many tensors at once.
//
// Both stream through memory and do a few operations for each element, so a
// launch covers as many tensors as its arguments can name: each workgroup takes
// one chunk of one tensor.  The step's tensors stand in a table on the GPU, made
// once; only the gradients, which a program may allocate anew, are arguments.
// Two ranks' 405 million float32 elements take 2155 us (11.3 GB at 5.3 TB/s; half of
// it is written), in bfloat16 with states of 8 bits 1353 us (6.5 GB at 4.8) and
// their norms 164 (0.8 GB at 4.9; 8 GB at 5.8).  A few small tensors wait for
// launches: 6 us the step, 6 and 2 the norms, 2.5 the factors.
#include "blocks_impl.h"

namespace rc {
namespace {

typedef uint32_t u32x4b __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2b __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32b __attribute__((aligned(1)));

// Four elements from `at` on; with Full all are there, else zeros behind `count`.
template <class T, bool Full>
__device__ __forceinline__ void load4(const void* from, int64_t at, int64_t count, float* f) {
    const typename T::E* p = static_cast<const typename T::E*>(from) + at;
    if (Full || at + 4 <= count) {
        if constexpr (T::n == 4) {
            T::unpack(*reinterpret_cast<const u32x4b*>(p), f);
        } else {
            const u32x2b v = *reinterpret_cast<const u32x2b*>(p);
            float g[8];
            T::unpack(u32x4{v[0], v[1], 0, 0}, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = g[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = at + i < count ? T::load(p[i]) : 0.0f;
    }
}
template <class T, bool Full>
__device__ __forceinline__ void store4(void* to, int64_t at, int64_t count, const float* f) {
    typename T::E* p = static_cast<typename T::E*>(to) + at;
    if (Full || at + 4 <= count) {
        if constexpr (T::n == 4) {
            *reinterpret_cast<u32x4b*>(p) = T::pack(f);
        } else {
            const float g[8] = {f[0], f[1], f[2], f[3], 0, 0, 0, 0};
            const u32x4 v = T::pack(g);
            *reinterpret_cast<u32x2b*>(p) = u32x2b{v[0], v[1]};
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i < count) p[i] = T::store(f[i]);
    }
}
template <bool Full>
__device__ __forceinline__ uint32_t load_codes(const void* from, int64_t at, int64_t count) {
    const uint8_t* p = static_cast<const uint8_t*>(from) + at;
    if (Full || at + 4 <= count) return *reinterpret_cast<const u32b*>(p);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (at + i < count) c |= (uint32_t)p[i] << (8 * i);
    return c;
}
template <bool Full>
__device__ __forceinline__ void store_codes(void* to, int64_t at, int64_t count, uint32_t c) {
    uint8_t* p = static_cast<uint8_t*>(to) + at;
    if (Full || at + 4 <= count) {
        *reinterpret_cast<u32b*>(p) = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (at + i < count) p[i] = (uint8_t)(c >> (8 * i));
}
__device__ __forceinline__ void values_of(uint32_t c, float scale, float* f) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    f[0] = lo[0] * scale;
    f[1] = lo[1] * scale;
    f[2] = hi[0] * scale;
    f[3] = hi[1] * scale;
}

__device__ __forceinline__ const void* address_of(uint64_t tagged) { return reinterpret_cast<const void*>(tagged & 0xffffffffffffffull); }
__device__ __forceinline__ int type_of(uint64_t tagged) { return (int)(tagged >> 56); }

// ---------------------------------------------------------------- gradient norms

constexpr int kThreads = 256;

__device__ __forceinline__ double join_sum(double v) {
    __shared__ double at[kThreads / kWave];
#pragma unroll
    for (int d = kWave / 2; d > 0; d /= 2) v += __shfl_xor(v, d);
    if (lane_id() == 0) at[threadIdx.x / kWave] = v;
    __syncthreads();
    return (at[0] + at[1]) + (at[2] + at[3]);
}

// Squares are exact in 64 bits for 16-bit elements, and neither small nor large
// ones leave its range.
template <class T>
__device__ __forceinline__ double squares(const void* grad, int64_t from, int64_t to) {
    double sum = 0.0;
    constexpr int kAhead = 4;
    int64_t at = from + 4 * threadIdx.x;
    for (; at - 4 * threadIdx.x + 4 * kThreads * kAhead <= to; at += 4 * kThreads * kAhead) {
        float f[kAhead][4];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) load4<T, true>(grad, at + 4 * kThreads * k, to, f[k]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = __builtin_fma((double)f[k][i], (double)f[k][i], sum);
    }
    for (; at < to; at += 4 * kThreads) {
        float f[4];
        load4<T, false>(grad, at, to, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = __builtin_fma((double)f[i], (double)f[i], sum);
    }
    return sum;
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(GradNormArgs a) {
    const int32_t chunk = blockIdx.x;
    int lo = 0, hi = a.n - 1;  // the last gradient whose first chunk is not past this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.first[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    const int64_t from = (int64_t)(chunk - a.first[lo]) * kNormChunk, to = min((int64_t)a.count[lo], from + kNormChunk);
    const void* grad = address_of(a.grad[lo]);
    const int type = type_of(a.grad[lo]);
    double sum = type == RC_F32 ? squares<F32>(grad, from, to) : type == RC_F16 ? squares<F16>(grad, from, to) : squares<BF16>(grad, from, to);
    sum = join_sum(sum);
    if (threadIdx.x == 0) a.partial[chunk] = sum;
}

__global__ __launch_bounds__(kThreads) void grad_norm_join_kernel(GradNormJoin a) {
    const int rank = blockIdx.x;
    const int64_t from = a.over_all ? 0 : a.first[rank], to = a.over_all ? a.first[a.nranks] : a.first[rank + 1];
    double sum = 0.0;
    int64_t i = from + threadIdx.x;
    for (; i + 7 * kThreads < to; i += 8 * kThreads) {
        double v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = a.partial[i + j * kThreads];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[j];
    }
    for (; i < to; i += kThreads) sum += a.partial[i];
    sum = join_sum(sum);
    if (threadIdx.x == 0) a.norms[rank] = (float)sqrt(sum);
}

// ---------------------------------------------------------------- AdamW

// 32 bits scrambled: products with odd numbers from the binary digits of the
// golden ratio and of the roots of 2 and 3, each spread down by a shift.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x *= 0x9E3779B9u;
    x = (x ^ (x >> 15)) * 0x6A09E667u;
    x = (x ^ (x >> 13)) * 0xBB67AE85u;
    return x ^ (x >> 16);
}

constexpr uint32_t kOfMeans = 0x6A09E667u;  // sets the chances of m apart from those of the root of v

// One lane for each rank: its factors, its step counted.
__global__ __launch_bounds__(kWave) void adamw_begin_kernel(AdamwBegin a) {
    const int r = threadIdx.x;
    if (r >= a.nranks) return;
    const float norm = a.norms ? a.norms[r] : 0.0f;
    const bool fine = isfinite(norm);
    const int32_t t = a.steps[r] + (fine ? 1 : 0);
    const double lr = a.lr_on_gpu ? (double)*a.lr_on_gpu : a.lr;
    double grad = a.grad_scale;
    const double size = (double)norm * fabs(a.grad_scale);
    if (a.max_norm > 0.0 && size > a.max_norm) grad *= a.max_norm / size;
    AdamwFactors f{};
    f.grad = (float)grad;
    f.keep = (float)(1.0 - lr * a.weight_decay);
    f.rate = (float)(lr / (1.0 - pow(a.beta1, (double)t)));
    f.root = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)t)));
    f.key = mix(mix((uint32_t)t) + a.seed);
    f.skip = !fine;
    a.table->factors[r] = f;
    a.steps_out[r] = t;
}

// The exponent's bits of x >= 0 among e4m3 values, whose distance is 2^-3 of theirs:
// values below 2^-6 lie as far apart as those above.
__device__ __forceinline__ uint32_t octave(float x) { return max(__builtin_bit_cast(uint32_t, x) >> 23, 127u - 6); }

// Values in [0, 448] as e4m3, each rounded up with the chance `u` / 2^16 <= its
// distance from the value below.
__device__ __forceinline__ float by_chance(float x, uint32_t u) {
    x = x > kE4M3Most ? kE4M3Most : x;
    const uint32_t e = octave(x);
    const float step = __builtin_bit_cast(float, (e - 3) << 23), per = __builtin_bit_cast(float, (257 - e) << 23);
    const float q = floorf(__builtin_fmaf(x, per, (float)u * 0x1p-16f)) * step;
    return q > kE4M3Most ? kE4M3Most : q;
}
// The same, zero to zero and others to no less than 2^-9.
__device__ __forceinline__ float root_by_chance(float x, uint32_t u) {
    const float c = by_chance(x, u);
    return x > 0.0f && c < 0x1p-9f ? 0x1p-9f : c;
}

// Four means m after a step, times what takes their block to e4m3, as what is to be
// rounded to nearest.  The `idle` ones (a bit each: their gradients were below the
// eighth of the smallest codes they had) whose decay, `rest` = 1 - beta1 of them, is
// less than half the distance of codes are rounded here, by chance: to nearest they
// would stay for ever where others hold the block's scale, and move their parameters
// the further the more the root that divides them has decayed.
__device__ __forceinline__ void round_means(const float* m, uint32_t idle, float rest, float mf, uint32_t key, float* q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = m[i] * mf;
    if (!__any(idle != 0)) return;
    const uint32_t u = mix(key), w = mix(key + 1);
    const uint32_t chance[4] = {u & 0xffff, u >> 16, w & 0xffff, w >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = fabsf(q[i]), half = __builtin_bit_cast(float, (octave(y) - 4) << 23);
        if ((idle >> i & 1) && rest * y < half) q[i] = copysignf(by_chance(y, chance[i]), q[i]);
    }
}

// One step of the chunk [from, to) of a parameter with a gradient: four elements a
// lane, so that a wave holds a block of 256, and two blocks ahead, which leaves
// registers for eight waves a SIMD, for seven with states of 8 bits.
template <class P, class G, int Bits, bool Full>
__device__ __forceinline__ void step_chunk(const AdamwArgs& a, const AdamwEntry& e, const AdamwEntry& o, const void* grad,
                                           const AdamwFactors& c, int64_t from, int64_t to) {
    constexpr int kAhead = 2, kRound = 4 * kThreads;
    static_assert(kAdamwLeast % (kAhead * kRound) == 0, "whole rounds");
    for (int64_t base = from; base < to; base += kRound * kAhead) {
        float p[kAhead][4], g[kAhead][4], m[kAhead][4], v[kAhead][4];
        uint32_t mc[kAhead], vc[kAhead];
        float ms[kAhead], vs[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t at = base + kRound * k + 4 * threadIdx.x, block = at / RC_ADAMW_BLOCK;
            load4<G, Full>(grad, at, to, g[k]);
            load4<F32, Full>(P::n == 4 ? e.param : e.master, at, to, p[k]);
            if constexpr (Bits == 32) {
                load4<F32, Full>(e.m, at, to, m[k]);
                load4<F32, Full>(e.v, at, to, v[k]);
            } else {
                const bool there = Full || block * RC_ADAMW_BLOCK < to;
                mc[k] = load_codes<Full>(e.m, at, to);
                vc[k] = load_codes<Full>(e.v, at, to);
                ms[k] = there ? e.m_scale[block] : 0.0f;
                vs[k] = there ? e.v_scale[block] : 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t at = base + kRound * k + 4 * threadIdx.x, block = at / RC_ADAMW_BLOCK;
            if constexpr (Bits == 8) {
                values_of(mc[k], ms[k], m[k]);
                values_of(vc[k], vs[k], v[k]);
            }
            float r[4];
            uint32_t idle = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = g[k][i] * c.grad;
                if constexpr (Bits == 8) {
                    idle |= (uint32_t)(fabsf(x) < ms[k] * 0x1p-6f) << i;
                    v[k][i] *= v[k][i];
                }
                m[k][i] = a.beta1 * m[k][i] + a.rest1 * x;
                v[k][i] = a.beta2 * v[k][i] + a.rest2 * (x * x);
                r[i] = sqrtf(v[k][i]);
                p[k][i] = p[k][i] * c.keep - c.rate * m[k][i] / (r[i] * c.root + a.eps);
            }
            if constexpr (P::n == 4) {
                store4<F32, Full>(o.param, at, to, p[k]);
            } else {
                store4<F32, Full>(o.master, at, to, p[k]);
                store4<P, Full>(o.param, at, to, p[k]);
            }
            if constexpr (Bits == 32) {
                store4<F32, Full>(o.m, at, to, m[k]);
                store4<F32, Full>(o.v, at, to, v[k]);
            } else {
                // a wave holds one block
                float mm = 0.0f, rr = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) mm = fmaxf(mm, fabsf(m[k][i])), rr = fmaxf(rr, r[i]);
                mm = wave_max(mm);
                rr = wave_max(rr);
                const float mf = e4m3_factor(mm), rf = e4m3_factor(rr);
                // the chances of elements 2i and 2i + 1 are the halves of one number
                const uint64_t pair = (uint64_t)at >> 1;
                const uint32_t place = (uint32_t)pair + 0xBB67AE85u * (uint32_t)(pair >> 32);
                const uint32_t u = mix(c.key + place), w = mix(c.key + place + 1);
                float q[4];
                round_means(m[k], idle, a.rest1, mf, (c.key ^ kOfMeans) + place, q);
                store_codes<Full>(o.m, at, to, e4m3_of(q[0], q[1], q[2], q[3]));
                store_codes<Full>(o.v, at, to, e4m3_of(root_by_chance(r[0] * rf, u & 0xffff), root_by_chance(r[1] * rf, u >> 16),
                                                       root_by_chance(r[2] * rf, w & 0xffff), root_by_chance(r[3] * rf, w >> 16)));
                if (lane_id() == 0 && (Full || at < to)) {
                    o.m_scale[block] = e4m3_scale(mm);
                    o.v_scale[block] = e4m3_scale(rr);
                }
            }
        }
    }
}

// Elements [from, to) of size `size` as they are.
__device__ __forceinline__ void copy_chunk(const void* src, void* dst, int64_t from, int64_t to, int size) {
    const uint8_t* s = static_cast<const uint8_t*>(src);
    uint8_t* d = static_cast<uint8_t*>(dst);
    if (size == 4) {
        for (int64_t i = from + threadIdx.x; i < to; i += kThreads) reinterpret_cast<uint32_t*>(d)[i] = reinterpret_cast<const uint32_t*>(s)[i];
    } else if (size == 2) {
        for (int64_t i = from + threadIdx.x; i < to; i += kThreads) reinterpret_cast<uint16_t*>(d)[i] = reinterpret_cast<const uint16_t*>(s)[i];
    } else {
        for (int64_t i = from + threadIdx.x; i < to; i += kThreads) d[i] = s[i];
    }
}

template <class P, class G, int Bits>
__device__ __forceinline__ void step_any(const AdamwArgs& a, const AdamwEntry& e, const AdamwEntry& o, const void* grad,
                                         const AdamwFactors& c, int64_t from) {
    if (from + a.chunk <= e.count) step_chunk<P, G, Bits, true>(a, e, o, grad, c, from, from + a.chunk);
    else step_chunk<P, G, Bits, false>(a, e, o, grad, c, from, e.count);
}

template <int Bits>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
    const int64_t chunk = group_index();
    if (chunk >= a.chunks) return;
    const uint8_t* table = reinterpret_cast<const uint8_t*>(a.table);
    const int32_t t = reinterpret_cast<const int32_t*>(table + a.chunks_at)[a.first_chunk + chunk];
    const AdamwEntry& e = reinterpret_cast<const AdamwEntry*>(table + a.entries_at)[t];
    const AdamwEntry& o = reinterpret_cast<const AdamwEntry*>(reinterpret_cast<const uint8_t*>(a.out) + a.entries_at)[t];
    const AdamwFactors c = a.table->factors[e.rank];
    const int64_t from = (a.first_chunk + chunk - e.first_chunk) * a.chunk;
    const void* grad = address_of(a.grad[t - a.first]);
    const int type = type_of(a.grad[t - a.first]);
    if (c.skip || !grad) {
        if (a.out == a.table) return;
        const int64_t to = min(e.count, from + a.chunk);
        copy_chunk(e.param, o.param, from, to, e.dtype == RC_F32 ? 4 : 2);
        if (e.dtype != RC_F32) copy_chunk(e.master, o.master, from, to, 4);
        copy_chunk(e.m, o.m, from, to, Bits / 8);
        copy_chunk(e.v, o.v, from, to, Bits / 8);
        if constexpr (Bits == 8) {
            const int64_t b0 = from / RC_ADAMW_BLOCK, b1 = (to + RC_ADAMW_BLOCK - 1) / RC_ADAMW_BLOCK;
            copy_chunk(e.m_scale, o.m_scale, b0, b1, 4);
            copy_chunk(e.v_scale, o.v_scale, b0, b1, 4);
        }
        return;
    }
    if (e.dtype == RC_F32) step_any<F32, F32, Bits>(a, e, o, grad, c, from);
    else if (e.dtype == RC_F16 && type == RC_F32) step_any<F16, F32, Bits>(a, e, o, grad, c, from);
    else if (e.dtype == RC_F16) step_any<F16, F16, Bits>(a, e, o, grad, c, from);
    else if (type == RC_F32) step_any<BF16, F32, Bits>(a, e, o, grad, c, from);
    else step_any<BF16, BF16, Bits>(a, e, o, grad, c, from);
}

}  // namespace

int launch_grad_norm(const GradNormArgs& a, void* stream) {
    grad_norm_kernel<<<a.chunks, kThreads, 0, (hipStream_t)stream>>>(a);
    return hipGetLastError();
}
int launch_grad_norm_join(const GradNormJoin& a, void* stream) {
    grad_norm_join_kernel<<<a.nranks, kThreads, 0, (hipStream_t)stream>>>(a);
    return hipGetLastError();
}
int launch_adamw_begin(const AdamwBegin& a, void* stream) {
    adamw_begin_kernel<<<1, kWave, 0, (hipStream_t)stream>>>(a);
    return hipGetLastError();
}
int launch_adamw(const AdamwArgs& a, int bits, void* stream) {
    const dim3 grid = grid_of(a.chunks);
    if (bits == 32) adamw_kernel<32><<<grid, kThreads, 0, (hipStream_t)stream>>>(a);
    else adamw_kernel<8><<<grid, kThreads, 0, (hipStream_t)stream>>>(a);
    return hipGetLastError();
}

}  // namespace rc
