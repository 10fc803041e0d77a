// Device helpers shared by the block operators' kernels (gfx950, wave64).
#pragma once

#include "rows_impl.h"

#include "blocks.h"

namespace rc {
namespace {

constexpr float kE4M3Most = 448.0f;
// A row, group or block whose largest value is below this is held as zeros: the
// factor that takes it to 448 stays below 2^126, the scale is a normal number.
constexpr float kLeast = 0x1p-117f;

template <int Ctrl>
__device__ __forceinline__ float dpp(float v) {
    const int i = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, Ctrl, 0xf, 0xf, true));
}
constexpr int kSwap1 = 0xb1, kSwap2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;

// The sum over the wave's lanes, alike in all of them: pairs, quads, eights and
// sixteens, then the four sixteens.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<kSwap1>(v);
    v += dpp<kSwap2>(v);
    v += dpp<kHalfMirror>(v);
    v += dpp<kMirror>(v);
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// The largest value of each run of `lanes` lanes (a power of two), alike in all
// of them; values that are no number count as none.
__device__ __forceinline__ float lanes_max(float v, int lanes) {
    if (lanes > 1) v = fmaxf(v, dpp<kSwap1>(v));
    if (lanes > 2) v = fmaxf(v, dpp<kSwap2>(v));
    if (lanes > 4) v = fmaxf(v, dpp<kHalfMirror>(v));
    if (lanes > 8) v = fmaxf(v, dpp<kMirror>(v));
    if (lanes > 16) v = fmaxf(v, __shfl_xor(v, 16));
    if (lanes > 32) v = fmaxf(v, __shfl_xor(v, 32));
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
    v = lanes_max(v, 16);
    return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}

// rank_of without a loop: spans past the last rank begin at the total.
__device__ __forceinline__ int rank_at(const RankSpans& s, int32_t i, int32_t* local) {
    int r = 0;
    int32_t base = 0;
#pragma unroll
    for (int k = 1; k < kMaxRanks; ++k) {
        const bool past = i >= s.first[k];
        r = past ? k : r;
        base = past ? s.first[k] : base;
    }
    *local = i - base;
    return r;
}

// Four values as e4m3, to nearest even.
__device__ __forceinline__ uint32_t e4m3_of(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// What takes a largest value to 448, and the scale that takes it back.
__device__ __forceinline__ float e4m3_factor(float most) { return most < kLeast ? 0.0f : kE4M3Most / most; }
__device__ __forceinline__ float e4m3_scale(float most) { return most < kLeast ? 0.0f : most / kE4M3Most; }

}  // namespace
}  // namespace rc
