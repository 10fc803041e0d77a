// Device helpers shared by the row-exchange kernels (gfx950, wave64).
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include "rows.h"

namespace rc {
namespace {

constexpr int kWave = 64;

// A 16-byte vector at any element-aligned address: gfx950 global accesses
// need no alignment beyond the element's, so rows of odd widths take the same
// wide instructions.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4m __attribute__((ext_vector_type(4), aligned(2)));

// Element types: E is the storage, n the elements of a 16-byte vector.
struct F32 {
    using E = float;
    static constexpr int n = 4;
    __device__ __forceinline__ static float load(E v) { return v; }
    __device__ __forceinline__ static E store(float v) { return v; }
    __device__ __forceinline__ static void unpack(u32x4 v, float* f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = v[i];  // not the vector's element itself, which a bit cast would take from its start
            f[i] = __builtin_bit_cast(float, u);
        }
    }
    __device__ __forceinline__ static u32x4 pack(const float* f) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint32_t, f[i]);
        return v;
    }
};

struct F16 {
    using E = _Float16;
    static constexpr int n = 8;
    __device__ __forceinline__ static float load(E v) { return (float)v; }
    __device__ __forceinline__ static E store(float v) { return (_Float16)v; }
    __device__ __forceinline__ static void unpack(u32x4 v, float* f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[i / 2] >> (16 * (i % 2))));
    }
    __device__ __forceinline__ static u32x4 pack(const float* f) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[2 * i]) |
                   (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[2 * i + 1]) << 16;
        return v;
    }
};

struct BF16 {
    using E = uint16_t;
    static constexpr int n = 8;
    __device__ __forceinline__ static float load(E v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
    __device__ __forceinline__ static E store(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
    __device__ __forceinline__ static void unpack(u32x4 v, float* f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
            f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static u32x4 pack(const float* f) {
        typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf2 p = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
            v[i] = __builtin_bit_cast(uint32_t, p);
        }
        return v;
    }
};

template <class T>
__device__ __forceinline__ u32x4 load16(const typename T::E* p) {
    return *reinterpret_cast<const u32x4m*>(p);
}
template <class T>
__device__ __forceinline__ void store16(typename T::E* p, u32x4 v) {
    *reinterpret_cast<u32x4m*>(p) = v;
}

// A store that goes past the caches, for what is not read again soon.
template <class T>
__device__ __forceinline__ void store16_past(typename T::E* p, u32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4m*>(p));
}

// The rank whose span holds item i (spans may be empty), and the item's index within it.
__device__ __forceinline__ int rank_of(const RankSpans& s, int32_t i, int32_t* local) {
    int r = 0;
    int32_t base = 0;
    for (int k = 1; k < s.nranks; ++k) {
        const bool past = i >= s.first[k];
        r = past ? k : r;
        base = past ? s.first[k] : base;
    }
    *local = i - base;
    return r;
}

// Workgroups in sequence over a grid of two dimensions: a launch may hold no
// more than 2^32 threads along one.
constexpr int64_t kGridWide = int64_t(1) << 20;
inline dim3 grid_of(int64_t groups, int64_t z = 1) {
    return dim3((unsigned)(groups < kGridWide ? groups : kGridWide), (unsigned)((groups + kGridWide - 1) / kGridWide), (unsigned)z);
}
__device__ __forceinline__ int64_t group_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// A value that all lanes hold alike.
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// LDS written by this wave's lanes may be read by its other lanes behind it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

#define RC_BY_TYPE(fn, ...)                                    \
    (dtype == RC_F32 ? fn<F32>(__VA_ARGS__)                    \
     : dtype == RC_F16 ? fn<F16>(__VA_ARGS__) : fn<BF16>(__VA_ARGS__))

__device__ __forceinline__ int lane_id() { return threadIdx.x & (kWave - 1); }

}  // namespace
}  // namespace rc
