// Block operators: what stands around a mixture-of-experts block and behind a
// gradient sync (root-mean-square norm, the experts' products of a few tokens,
// gradient norms and the AdamW step).  Argument blocks shared by the argument
// checks (blocks.cpp) and the kernels (block_*.hip).  Plain C++.
#pragma once

#include <cstdint>

#include "rows.h"

namespace rc {

// ---------------------------------------------------------------- norm
struct NormArgs {
    const void* x[kMaxRanks];        // rows; gradient: the rows that were normalised
    const void* residual[kMaxRanks]; // gradient: d_sums
    const void* weight[kMaxRanks];
    void* y[kMaxRanks];              // gradient: d_xs
    float* scale[kMaxRanks];
    void* sum[kMaxRanks];
    const void* d_y[kMaxRanks];      // gradient
    void* d_weight[kMaxRanks];       // gradient
    float* partial;                  // gradient: [parts of all ranks][width]
    RankSpans tokens;
    RankSpans parts;                 // gradient: workgroups of each rank
    int64_t width;
    int32_t has_residual;
    int32_t quantize;
    int32_t group;                   // elements that share a scale; 0: a row
    int32_t groups;                  // scales of a row
    float eps;
};

int launch_rms_norm_F32(const NormArgs& a, int weight_dtype, void* stream);
int launch_rms_norm_F16(const NormArgs& a, int weight_dtype, void* stream);
int launch_rms_norm_BF16(const NormArgs& a, int weight_dtype, void* stream);
inline int launch_rms_norm(const NormArgs& a, int dtype, int weight_dtype, void* stream) {
    return dtype == RC_F32 ? launch_rms_norm_F32(a, weight_dtype, stream)
         : dtype == RC_F16 ? launch_rms_norm_F16(a, weight_dtype, stream) : launch_rms_norm_BF16(a, weight_dtype, stream);
}
int launch_rms_norm_grad_F32(const NormArgs& a, int weight_dtype, void* stream);
int launch_rms_norm_grad_F16(const NormArgs& a, int weight_dtype, void* stream);
int launch_rms_norm_grad_BF16(const NormArgs& a, int weight_dtype, void* stream);
inline int launch_rms_norm_grad(const NormArgs& a, int dtype, int weight_dtype, void* stream) {
    return dtype == RC_F32 ? launch_rms_norm_grad_F32(a, weight_dtype, stream)
         : dtype == RC_F16 ? launch_rms_norm_grad_F16(a, weight_dtype, stream)
                           : launch_rms_norm_grad_BF16(a, weight_dtype, stream);
}

// Workgroups of each rank that sum its weights' gradient.
RankSpans norm_parts(const RankSpans& tokens);

}  // namespace rc
