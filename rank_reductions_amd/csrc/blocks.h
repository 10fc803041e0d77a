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

// ---------------------------------------------------------------- experts
struct MoeArgs {
    const void* x[kMaxRanks];
    const float* x_scale[kMaxRanks];
    const int32_t* experts[kMaxRanks];
    const float* weights[kMaxRanks];
    const void* gate_up[kMaxRanks];
    const float* gate_up_scale[kMaxRanks];
    const void* down[kMaxRanks];
    const float* down_scale[kMaxRanks];
    void* y[kMaxRanks];
    RankSpans entries;       // (token, k) of all ranks
    uint8_t* hidden;         // silu(G x) * (U x) of every entry: [entries][hidden_row], float32, or bfloat16 two or three times
    int64_t hidden_plane;    // bytes of all entries' first bfloat16 numbers
    int64_t hidden_bytes;    // of all
    float* products;         // D times the hidden values: [entries][product_row]
    uint8_t* lists;          // the experts named, and their entries
    int32_t hidden_row;      // elements, a multiple of 64
    int32_t product_row;     // elements, a multiple of 16
    int32_t num_experts;
    int32_t per_rank;
    int32_t top_k;
    int32_t width;
    int32_t inner;
    int32_t out_dtype;
};
static_assert(sizeof(MoeArgs) <= 4096, "kernel arguments");
int launch_moe(const MoeArgs& a, int dtype, int weight_dtype, void* stream);

// ---------------------------------------------------------------- gradient norms
constexpr int64_t kNormChunk = 32768;  // elements of a workgroup
constexpr int kNormList = 250;         // pieces of a launch: kernel arguments hold 4096 bytes
constexpr int64_t kNormPiece = int64_t(1) << 30;  // elements of a piece at most: whole chunks

struct GradNormArgs {
    uint64_t grad[kNormList];  // addresses; the top byte is the type
    int32_t count[kNormList];
    int32_t first[kNormList];  // the piece's first chunk within the launch
    int32_t n;
    int32_t chunks;
    double* partial;           // the launch's first chunk
};
struct GradNormJoin {
    const double* partial;
    float* norms;
    int64_t first[kMaxRanks + 1];  // chunks of each rank
    int32_t nranks;
    int32_t over_all;
};
int launch_grad_norm(const GradNormArgs& a, void* stream);
int launch_grad_norm_join(const GradNormJoin& a, void* stream);

// ---------------------------------------------------------------- AdamW
// Elements of a workgroup: the most that still give 2048 workgroups, or the least.
constexpr int64_t kAdamwLeast = 2048, kAdamwMost = 8192;
constexpr int kAdamwList = 440;        // parameters of a launch

struct AdamwEntry {
    void* param;
    float* master;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    int64_t count;
    int64_t first_chunk;
    int32_t dtype;
    int32_t rank;
};
// What a rank's elements are computed with, written at each step's start.
struct AdamwFactors {
    float grad;    // of the gradient
    float keep;    // 1 - lr * weight_decay
    float rate;    // lr / (1 - beta1^t)
    float root;    // 1 / sqrt(1 - beta2^t)
    uint32_t key;  // of the roundings
    int32_t skip;
    int32_t pad[2];
};
// A table: this, then the entries, the entry of each chunk, and on the host's
// side alone the spans of all buffers in order.
struct AdamwHeader {
    uint64_t magic;
    int64_t bytes;
    int32_t nranks;
    int32_t bits;
    int32_t first[kMaxRanks + 1];  // parameters of each rank
    int32_t spans;
    int64_t chunks;
    int64_t chunk;  // elements
    int64_t entries_at, chunks_at, spans_at;  // byte offsets
    AdamwFactors factors[kMaxRanks];
};
struct AdamwSpan {
    uint64_t lo, hi;
};
constexpr uint64_t kAdamwMagic = 0x6164616d77746231ull;

struct AdamwBegin {
    AdamwHeader* table;
    double lr, beta1, beta2, weight_decay, max_norm, grad_scale;
    const float* lr_on_gpu;
    const float* norms;
    const int32_t* steps;
    int32_t* steps_out;
    uint32_t seed;
    int32_t nranks;
};
struct AdamwArgs {
    uint64_t grad[kAdamwList];  // addresses; the top byte is the type
    const AdamwHeader* table;
    const AdamwHeader* out;
    int64_t entries_at, chunks_at;
    int32_t first;              // the launch's first parameter
    int32_t pad;
    int64_t first_chunk, chunks, chunk;
    float beta1, rest1, beta2, rest2, eps;
};
static_assert(sizeof(GradNormArgs) <= 4096 && sizeof(AdamwArgs) <= 4096, "kernel arguments");
int launch_adamw_begin(const AdamwBegin& a, void* stream);
int launch_adamw(const AdamwArgs& a, int bits, void* stream);

}  // namespace rc
