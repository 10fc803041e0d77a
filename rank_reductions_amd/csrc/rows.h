// Row exchanges: operators that move rows between the logical ranks by an
// index computed on the GPU (expert routing, dispatch and combine, the
// sharded embedding lookup and its gradient).  Argument blocks shared by the
// argument checks (rows.cpp) and the kernels (rows_*.hip).  Plain C++.
#pragma once

#include <cstdint>
#include <functional>

#include "rc_internal.h"

namespace rc {

// Bytes of a row operator's element type; 0 for a type it does not have.
inline int64_t row_element_size(int dtype) {
    return dtype == RC_F32 ? 4 : dtype == RC_F16 || dtype == RC_BF16 ? 2 : 0;
}

// Items of all ranks counted in one sequence: rank r's are [first[r],
// first[r + 1]); entries past the last rank repeat the total.
struct RankSpans {
    int32_t first[kMaxRanks + 1];
    int32_t nranks;
    constexpr int32_t total() const { return first[kMaxRanks]; }
};

// ---------------------------------------------------------------- routing
struct RouteArgs {
    const void* logits[kMaxRanks];
    float* weights[kMaxRanks];      // route: out
    int32_t* experts[kMaxRanks];    // route: out; gradient: in
    const float* d_weights[kMaxRanks];  // gradient: in
    void* d_logits[kMaxRanks];          // gradient: out
    RankSpans tokens;
    const float* bias;
    int32_t num_experts;
    int32_t top_k;
    int32_t sigmoid;
    int32_t groups;
    int32_t top_groups;
    int32_t top2;         // a group's score is the sum of its two best
    int32_t renormalize;
    float scale;
    int32_t group_size;   // num_experts / groups
    int32_t group_lanes;  // lanes of a token that share a group
    int32_t vec;          // every row starts on a 4-element boundary, and so does every group
    int32_t bias_vec;     // and the bias
    int32_t staged;       // rows go through LDS
};

// ---------------------------------------------------------------- counting sort
// Entries per workgroup of the sort kernels, and the most digits one pass
// tells apart.
constexpr int kSortBlock = 1024;
constexpr int kSortBins = 1024;

// One pass of a stable counting sort over `spans.total()` entries cut into
// blocks of kSortBlock, each within one rank's entries.
struct SortPass {
    RankSpans spans;       // entries of each rank
    RankSpans blocks;      // blocks of each rank
    const void* ids[kMaxRanks];  // keys of the first pass (experts, token ids)
    int32_t id64;          // ids are 64-bit
    int64_t key_limit;     // ids outside [0, key_limit) get the key key_limit
    int32_t drop;          // entries with that key have no place
    const int32_t* keys;   // later passes: keys and values in the order of the pass before
    const int32_t* vals;
    int32_t* out_keys;
    int32_t* out_vals;
    int32_t shift;
    int32_t bits;
    int32_t bins;          // digits in use
    int32_t* hist;         // [blocks][bins] counts; scanned: sums of the blocks before, then bins totals
    int32_t scanned;
    uint8_t* named;        // embedding gradient: a byte per table row, one if a key names it
};

struct PlanArgs {
    SortPass sort;
    int32_t* slots[kMaxRanks];
    int32_t* offsets[kMaxRanks];
    int32_t* counts[kMaxRanks];
    int64_t capacity[kMaxRanks];
    int32_t num_experts;
    int32_t per_rank;  // experts of each rank
};

// ---------------------------------------------------------------- row moves
struct ExchangeArgs {
    const void* in[kMaxRanks];      // dispatch: xs; combine: rows; gradient: rows
    void* out[kMaxRanks];           // dispatch: rows; combine: outs; gradient: d_rows
    const void* d_out[kMaxRanks];   // gradient
    const float* weights[kMaxRanks];
    float* d_weights[kMaxRanks];
    const int32_t* experts[kMaxRanks];
    const int32_t* slots[kMaxRanks];
    int64_t capacity[kMaxRanks];
    RankSpans tokens;
    int64_t width;
    int32_t num_experts;
    int32_t per_rank;
    int32_t top_k;
    int32_t weighted;
    int32_t chunks;  // pieces of a row, one wave each
};

// ---------------------------------------------------------------- embedding
struct EmbeddingArgs {
    const void* ids[kMaxRanks];
    const void* table[kMaxRanks];
    void* out[kMaxRanks];
    RankSpans tokens;
    int64_t vocab;
    int64_t shard;   // rows of a full shard, ceil(vocab / ranks)
    int64_t width;
    float scale;
    int32_t id64;
    int32_t chunks;
};

// Sorted entries per piece of a long sum (see rows_embedding.hip).
constexpr int kPiece = 64;

struct EmbeddingGradArgs {
    const void* d_out[kMaxRanks];
    void* table[kMaxRanks];
    RankSpans tokens;
    const int32_t* keys;   // sorted ids; vocab for those outside the table
    const int32_t* vals;   // position in the sequence of all ranks' tokens
    const uint8_t* named;  // [vocab], one for a row that some token names
    float* partial;        // [blocks of kPiece entries][2][width]
    int64_t vocab;
    int64_t shard;
    int64_t width;
    float scale;
    int32_t accumulate;
    int32_t window;        // sorted entries per workgroup, a power of two up to kPiece
    int32_t windows;
    int32_t fill_rows;     // table rows per workgroup that clears those no id names, a power of two up to 64
    int32_t fill_groups;
    int32_t spacing;       // the first workgroups at multiples of this clear rows; 0: those behind the windows do
};

// ---------------------------------------------------------------- launches (rows_*.hip)
// Each returns a hipError_t as int; the session's device is current.
int launch_route_F32(const RouteArgs& a, void* stream);
int launch_route_F16(const RouteArgs& a, void* stream);
int launch_route_BF16(const RouteArgs& a, void* stream);
int launch_route_grad_F32(const RouteArgs& a, void* stream);
int launch_route_grad_F16(const RouteArgs& a, void* stream);
int launch_route_grad_BF16(const RouteArgs& a, void* stream);
inline int launch_route(const RouteArgs& a, int dtype, void* stream) {
    return dtype == RC_F32 ? launch_route_F32(a, stream)
         : dtype == RC_F16 ? launch_route_F16(a, stream) : launch_route_BF16(a, stream);
}
inline int launch_route_grad(const RouteArgs& a, int dtype, void* stream) {
    return dtype == RC_F32 ? launch_route_grad_F32(a, stream)
         : dtype == RC_F16 ? launch_route_grad_F16(a, stream) : launch_route_grad_BF16(a, stream);
}
int launch_plan(PlanArgs a, void* workspace, void* stream);
int launch_dispatch(const ExchangeArgs& a, int dtype, void* stream);
int launch_combine(const ExchangeArgs& a, int dtype, void* stream);
int launch_combine_grad(const ExchangeArgs& a, int dtype, void* stream);
int launch_embedding(const EmbeddingArgs& a, int dtype, void* stream);
// Sorts the ids, then sums; `sort` holds the ids (spans, ids, id64).
int launch_embedding_grad(EmbeddingGradArgs a, SortPass sort, int dtype, int grad_dtype, void* workspace,
                          void* stream);

// Workspace bytes of the two sorting operators.
int64_t plan_workspace_bytes(const RankSpans& entries, int num_experts);
int64_t embedding_grad_workspace_bytes(const RankSpans& tokens, int64_t vocab, int64_t width);

// Blocks of kSortBlock entries for each rank.
RankSpans sort_blocks(const RankSpans& entries);

}  // namespace rc
