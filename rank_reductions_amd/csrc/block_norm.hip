// Root-mean-square norm of rows with the residual's addition, its output in
// the rows' type or in 8 bits, and its gradient.  Compiled once per row type.
//
// Forward: s = x + residual (rounded to the rows' type and stored: what the
// gradient and the next layer read), y = s / sqrt(mean(s^2) + eps) * w.  A row
// stays in registers between the sum of its squares and its output, so every
// byte moves once.  Gradient, with n = s / sqrt(...) and dn = dy * w:
// dx = (dn - n * mean(dn * n)) / sqrt(...) + d_sum; dw = the sum over rows of
// dy * n, held in registers by a workgroup over the rows it takes, then added
// up over the workgroups in order.
// Both stream: 16384 rows of 4096 bf16 with a residual take 85 us forward (537 MB,
// some from the last-level cache, at 6.2 TB/s) and 122 back (4.5 TB/s: a row waits
// for its two sums; rows of more than 16384 elements spill 90 to 143 registers); 6404
// rows of 5003 float16 to 8 bits 58 us (3.9 TB/s).
#include "blocks_impl.h"

#ifndef RC_ROW_TYPE
#error "RC_ROW_TYPE: F32, F16 or BF16"
#endif

namespace rc {
namespace {

// One 16-byte vector of a row of `width` elements, from element `at` on; zeros
// behind the row's end.
template <class T>
__device__ __forceinline__ u32x4 load_part(const typename T::E* row, int64_t at, int64_t width) {
    u32x4 v = {0, 0, 0, 0};
    if (at + T::n <= width) {
        v = load16<T>(row + at);
    } else if (at < width) {
        float f[T::n];
#pragma unroll
        for (int i = 0; i < T::n; ++i) f[i] = at + i < width ? T::load(row[at + i]) : 0.0f;
        v = T::pack(f);
    }
    return v;
}
template <class T>
__device__ __forceinline__ void store_part(typename T::E* row, int64_t at, int64_t width, const float* f) {
    if (at + T::n <= width) {
        store16<T>(row + at, T::pack(f));
    } else if (at < width) {
#pragma unroll
        for (int i = 0; i < T::n; ++i)
            if (at + i < width) row[at + i] = T::store(f[i]);
    }
}
// N floats of type W (a row's own type or float32) from element `at` on.
template <class W, int N>
__device__ __forceinline__ void load_floats(const typename W::E* row, int64_t at, int64_t width, float* f) {
#pragma unroll
    for (int i = 0; i < N; i += W::n) W::unpack(load_part<W>(row, at + i, width), f + i);
}
typedef uint32_t u32x2b __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32b __attribute__((aligned(1)));
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t at, int64_t width, const float* f) {
    uint32_t c[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) c[i] = e4m3_of(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    if (at + N <= width) {
        if constexpr (N == 8) {
            const u32x2b v = {c[0], c[1]};
            *reinterpret_cast<u32x2b*>(row + at) = v;
        } else {
            *reinterpret_cast<u32b*>(row + at) = c[0];
        }
    } else if (at < width) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (at + i < width) row[at + i] = (uint8_t)(c[i / 4] >> (8 * (i % 4)));
    }
}

// Joins the waves of a row; `at`: one slot of LDS for each wave.  All threads call.
template <int Waves, class F>
__device__ __forceinline__ float join_waves(float v, float* at, F f) {
    if constexpr (Waves == 1) return v;
    const int wave = threadIdx.x / kWave;
    if (lane_id() == 0) at[wave] = v;
    __syncthreads();
    float t = at[0];
#pragma unroll
    for (int w = 1; w < Waves; ++w) t = f(t, at[w]);
    return t;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }

// Waves: waves of a row; V: vectors of a row that each lane holds.
template <class T, class W, int Waves, int V>
__global__ __launch_bounds__(Waves == 1 ? 256 : Waves * kWave) void rms_norm_kernel(NormArgs a) {
    __shared__ float joined[2][Waves];
    constexpr int kThreads = Waves * kWave, N = T::n;
    const int at = Waves == 1 ? lane_id() : threadIdx.x;
    const int64_t row = Waves == 1 ? group_index() * (256 / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) : group_index();
    if (row >= a.tokens.total()) return;
    int32_t t;
    const int rank = rank_at(a.tokens, (int32_t)row, &t);
    const int64_t width = a.width, from = t * width;
    u32x4 raw[V], more[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        raw[j] = load_part<T>((const typename T::E*)a.x[rank] + from, (int64_t)(at + j * kThreads) * N, width);
    if (a.has_residual) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            more[j] = load_part<T>((const typename T::E*)a.residual[rank] + from, (int64_t)(at + j * kThreads) * N, width);
    }
    float s[V * N];
    float square = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float* f = s + j * N;
        T::unpack(raw[j], f);
        if (a.has_residual) {
            float r[N];
            T::unpack(more[j], r);
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] += r[i];
            store_part<T>((typename T::E*)a.sum[rank] + from, (int64_t)(at + j * kThreads) * N, width, f);
            // the norm is that of the sum as it is stored
            T::unpack(T::pack(f), f);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) square = __builtin_fmaf(f[i], f[i], square);
    }
    square = join_waves<Waves>(wave_sum(square), joined[0], add);
    const float factor = 1.0f / sqrtf(square / (float)width + a.eps);
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float* f = s + j * N;
        const int64_t e = (int64_t)(at + j * kThreads) * N;
        float w[N];
        load_floats<W, N>((const typename W::E*)a.weight[rank], e, width, w);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = f[i] * factor * w[i];
        if (!a.quantize) {
            store_part<T>((typename T::E*)a.y[rank] + from, e, width, f);
        } else {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(f[i]));
            if (a.group) {
                m = lanes_max(m, a.group / N);
                const float to = e4m3_factor(m);
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] *= to;
                store_codes<N>((uint8_t*)a.y[rank] + from, e, width, f);
                if (e % a.group == 0 && e < width) a.scale[rank][(int64_t)t * a.groups + e / a.group] = e4m3_scale(m);
            } else {
                most = fmaxf(most, m);
            }
        }
    }
    if (a.quantize && !a.group) {
        most = join_waves<Waves>(wave_max(most), joined[1], fmaxf);
        const float to = e4m3_factor(most);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float* f = s + j * N;
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] *= to;
            store_codes<N>((uint8_t*)a.y[rank] + from, (int64_t)(at + j * kThreads) * N, width, f);
        }
        if (at == 0) a.scale[rank][t] = e4m3_scale(most);
    }
}

// A workgroup keeps its part of dw in registers, so few workgroups, 512 in all,
// keep the parts' memory small (8 MB of 546 at 4096 columns); with eight waves of
// one vector 120 us in place of 126 with four of two.
//
// The gradient for the rows t = part, part + parts, ... of a rank (a workgroup
// is four waves with a row each, or `Waves` on one row).
template <class T, class W, int Waves, int V>
__global__ __launch_bounds__(Waves == 1 ? 256 : Waves * kWave) void rms_norm_grad_kernel(NormArgs a) {
    constexpr int kThreads = Waves * kWave, N = T::n, kRows = Waves == 1 ? 4 : 1;
    __shared__ float joined[2][2][Waves];
    __shared__ float rows[kRows == 1 ? 1 : 3 * kWave * V * N];
    const int at = Waves == 1 ? lane_id() : threadIdx.x, wave = threadIdx.x / kWave;
    int32_t part;
    const int rank = rank_at(a.parts, (int32_t)blockIdx.x, &part);
    const int32_t parts = a.parts.first[rank + 1] - a.parts.first[rank];
    const int32_t tokens = a.tokens.first[rank + 1] - a.tokens.first[rank];
    const int64_t width = a.width;
    float dw[V * N] = {};
    int turn = 0;
    for (int64_t t = (int64_t)part * kRows + (kRows == 1 ? 0 : wave); t < tokens; t += (int64_t)parts * kRows, turn ^= 1) {
        const int64_t from = t * width;
        u32x4 s[V], g[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t e = (int64_t)(at + j * kThreads) * N;
            s[j] = load_part<T>((const typename T::E*)a.x[rank] + from, e, width);
            g[j] = load_part<T>((const typename T::E*)a.d_y[rank] + from, e, width);
        }
        float square = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float f[N], d[N], w[N];
            T::unpack(s[j], f);
            T::unpack(g[j], d);
            load_floats<W, N>((const typename W::E*)a.weight[rank], (int64_t)(at + j * kThreads) * N, width, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                square = __builtin_fmaf(f[i], f[i], square);
                dot = __builtin_fmaf(d[i] * w[i], f[i], dot);
            }
        }
        square = wave_sum(square);
        dot = wave_sum(dot);
        if constexpr (Waves > 1) {  // two rows in turn use the two halves: one barrier a row
            if (lane_id() == 0) joined[turn][0][wave] = square, joined[turn][1][wave] = dot;
            __syncthreads();
            square = dot = 0.0f;
#pragma unroll
            for (int i = 0; i < Waves; ++i) square += joined[turn][0][i], dot += joined[turn][1][i];
        }
        const float factor = 1.0f / sqrtf(square / (float)width + a.eps);
        const float back = dot * factor / (float)width * factor;  // mean(dn * n) / sqrt(...), but for s's own factor
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t e = (int64_t)(at + j * kThreads) * N;
            float f[N], d[N], w[N], more[N];
            T::unpack(s[j], f);
            T::unpack(g[j], d);
            load_floats<W, N>((const typename W::E*)a.weight[rank], e, width, w);
            if (a.has_residual) T::unpack(load_part<T>((const typename T::E*)a.residual[rank] + from, e, width), more);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float n = f[i] * factor;
                dw[j * N + i] = __builtin_fmaf(d[i], n, dw[j * N + i]);
                f[i] = factor * (d[i] * w[i]) - n * back;
                if (a.has_residual) f[i] += more[i];
            }
            store_part<T>((typename T::E*)a.y[rank] + from, e, width, f);
        }
    }
    if constexpr (kRows > 1) {  // the four waves' sums, in order
        if (wave > 0) {
#pragma unroll
            for (int j = 0; j < V * N; ++j) rows[((wave - 1) * V * N + j) * kWave + at] = dw[j];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int j = 0; j < V * N; ++j)
            for (int w = 0; w < 3; ++w) dw[j] += rows[(w * V * N + j) * kWave + at];
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < N; i += 4)
            store_part<F32>(a.partial + (int64_t)blockIdx.x * width, (int64_t)(at + j * kThreads) * N + i, width, dw + j * N + i);
}

// Each column's parts: eight runs of consecutive ones, then the runs in order.
constexpr int kColumnLanes = 32, kColumnRuns = 8;
template <class W>
__global__ __launch_bounds__(kColumnLanes * kColumnRuns) void norm_columns_kernel(NormArgs a) {
    __shared__ float sums[kColumnRuns][kColumnLanes];
    const int rank = blockIdx.y, lane = threadIdx.x % kColumnLanes, run = threadIdx.x / kColumnLanes;
    const int64_t c = (int64_t)blockIdx.x * kColumnLanes + lane;
    const int32_t first = a.parts.first[rank], parts = a.parts.first[rank + 1] - first;
    const int32_t each = (parts + kColumnRuns - 1) / kColumnRuns;
    float sum = 0.0f;
    if (c < a.width)
        for (int32_t p = run * each; p < min((run + 1) * each, parts); ++p) sum += a.partial[(int64_t)(first + p) * a.width + c];
    sums[run][lane] = sum;
    __syncthreads();
    if (run || c >= a.width) return;
#pragma unroll
    for (int k = 1; k < kColumnRuns; ++k) sum += sums[k][lane];
    ((typename W::E*)a.d_weight[rank])[c] = W::store(sum);
}

template <class T, class W, int Waves, int V>
int run_norm(const NormArgs& a, hipStream_t s) {
    const int64_t rows = a.tokens.total();
    rms_norm_kernel<T, W, Waves, V><<<grid_of(Waves == 1 ? (rows + 3) / 4 : rows), Waves == 1 ? 256 : Waves * kWave, 0, s>>>(a);
    return hipGetLastError();
}

// Short rows take a wave each, longer ones four to sixteen waves with a few
// vectors a lane (16384 rows of 4096 bf16: 84 us with four waves of two vectors,
// 105 with one of eight; 64 rows: 4.4 and 7.6 us), in steps that leave few lanes idle
// (4096 rows of 17000: 118 us with three vectors a lane, 127 with four; of 24576: 153
// and 159).
template <class T, class W>
int norm_of(const NormArgs& a, hipStream_t s) {
    const int64_t vectors = (a.width + T::n - 1) / T::n;
    if (vectors <= 64) return run_norm<T, W, 1, 1>(a, s);
    if (vectors <= 128) return run_norm<T, W, 1, 2>(a, s);
    if (vectors <= 256) return run_norm<T, W, 4, 1>(a, s);
    if (vectors <= 512) return run_norm<T, W, 4, 2>(a, s);
    if (vectors <= 768) return run_norm<T, W, 4, 3>(a, s);
    if (vectors <= 1024) return run_norm<T, W, 4, 4>(a, s);
    if (vectors <= 1536) return run_norm<T, W, 8, 3>(a, s);
    if (vectors <= 2048) return run_norm<T, W, 8, 4>(a, s);
    if (vectors <= 3 * 1024) return run_norm<T, W, 16, 3>(a, s);
    if constexpr (T::n == 4)
        if (vectors > 4096) return run_norm<T, W, 16, 8>(a, s);
    return run_norm<T, W, 16, 4>(a, s);
}

template <class T, class W, int Waves, int V>
int run_grad(const NormArgs& a, hipStream_t s) {
    if (a.parts.total())
        rms_norm_grad_kernel<T, W, Waves, V><<<a.parts.total(), Waves == 1 ? 256 : Waves * kWave, 0, s>>>(a);
    const dim3 grid((unsigned)((a.width + kColumnLanes - 1) / kColumnLanes), (unsigned)a.parts.nranks);
    norm_columns_kernel<W><<<grid, kColumnLanes * kColumnRuns, 0, s>>>(a);
    return hipGetLastError();
}

template <class T, class W>
int grad_of(const NormArgs& a, hipStream_t s) {
    const int64_t vectors = (a.width + T::n - 1) / T::n;
    if (vectors <= 64) return run_grad<T, W, 1, 1>(a, s);
    if (vectors <= 128) return run_grad<T, W, 1, 2>(a, s);
    if (vectors <= 256) return run_grad<T, W, 4, 1>(a, s);
    if (vectors <= 512) return run_grad<T, W, 8, 1>(a, s);
    if (vectors <= 1024) return run_grad<T, W, 8, 2>(a, s);
    if (vectors <= 2048) return run_grad<T, W, 16, 2>(a, s);
    if constexpr (T::n == 4)
        if (vectors > 4096) return run_grad<T, W, 16, 8>(a, s);
    return run_grad<T, W, 16, 4>(a, s);
}

}  // namespace

#define RC_JOIN_(a, b) a##b
#define RC_JOIN(a, b) RC_JOIN_(a, b)
int RC_JOIN(launch_rms_norm_, RC_ROW_TYPE)(const NormArgs& a, int weight_dtype, void* stream) {
    using T = RC_ROW_TYPE;
    if (weight_dtype == RC_F32) return norm_of<T, F32>(a, (hipStream_t)stream);
    return norm_of<T, T>(a, (hipStream_t)stream);
}
int RC_JOIN(launch_rms_norm_grad_, RC_ROW_TYPE)(const NormArgs& a, int weight_dtype, void* stream) {
    using T = RC_ROW_TYPE;
    if (weight_dtype == RC_F32) return grad_of<T, F32>(a, (hipStream_t)stream);
    return grad_of<T, T>(a, (hipStream_t)stream);
}

}  // namespace rc
