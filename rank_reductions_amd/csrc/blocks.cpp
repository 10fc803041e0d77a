// Entry points and argument checks of the block operators.  Host-only C++; the
// kernels are reached through the launch_* functions of blocks.h.  Everything
// is checked before anything is enqueued.
#include "blocks.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "rows_check.h"

namespace rc {
namespace {

constexpr int64_t kMaxElements = int64_t(1) << 38;  // of a tensor
constexpr int64_t kMaxNormChunks = kMaxElements / kNormChunk;  // of a launch: 2^31 threads
constexpr int64_t kMaxTensors = int64_t(1) << 24;   // of all ranks

Error check_workspace(const char* what, const void* workspace, int64_t have, int64_t need_bytes, Buffers* b) {
    if (have < need_bytes) return bad(what, fmt("workspace of %lld bytes, needs %lld", have, need_bytes));
    b->write(workspace, need_bytes, 1, "workspace", 0);
    if (need_bytes && reinterpret_cast<uintptr_t>(workspace) % 16) return bad(what, "misaligned workspace");
    return {};
}

// ---------------------------------------------------------------- norm

Error check_norm(const char* what, int R, const rc_norm_desc* d, NormArgs* a) {
    RC_TRY(check_desc(what, d, "rc_norm_desc"));
    if (!row_element_size(d->dtype)) return bad(what, fmt("unknown dtype %lld", d->dtype));
    if (d->weight_dtype != RC_F32 && d->weight_dtype != d->dtype)
        return bad(what, fmt("weight_dtype %lld is neither RC_F32 nor dtype", d->weight_dtype));
    if (d->width < 1 || d->width > RC_MAX_NORM_WIDTH) return bad(what, fmt("width %lld outside [1, 32768]", d->width));
    if (!(d->eps >= 0) || !std::isfinite(d->eps)) return bad(what, "eps is not a number of at least 0");
    if (d->quantize != RC_QUANTIZE_NONE && d->quantize != RC_QUANTIZE_E4M3) return bad(what, "unknown quantize");
    if (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128 && d->group != 256)
        return bad(what, fmt("group %lld is none of 0, 32, 64, 128 and 256", d->group));
    RC_TRY(spans_of(what, R, d->tokens, 1, &a->tokens));
    a->width = d->width;
    a->eps = d->eps;
    a->quantize = d->quantize;
    a->group = d->group;
    a->groups = d->group ? (int32_t)((d->width + d->group - 1) / d->group) : 1;
    return {};
}

// ---------------------------------------------------------------- experts

int64_t any_element_size(int dtype) { return dtype == RC_E4M3 ? 1 : row_element_size(dtype); }

Error check_moe(const char* what, int R, const rc_moe_desc* d, MoeArgs* a, int64_t* workspace) {
    RC_TRY(check_desc(what, d, "rc_moe_desc"));
    if (!any_element_size(d->dtype)) return bad(what, fmt("unknown dtype %lld", d->dtype));
    if (d->weight_dtype != d->dtype && (d->weight_dtype != RC_E4M3 || d->dtype == RC_F32))
        return bad(what, fmt("weight_dtype %lld for rows of dtype %lld", d->weight_dtype, d->dtype));
    if (d->dtype == RC_E4M3 ? !row_element_size(d->out_dtype) : d->out_dtype != d->dtype)
        return bad(what, fmt("out_dtype %lld for rows of dtype %lld", d->out_dtype, d->dtype));
    if (d->num_experts < 1 || d->num_experts > RC_MAX_EXPERTS || d->num_experts % R)
        return bad(what, fmt("num_experts %lld outside [1, 1024] or not divisible by the %lld ranks", d->num_experts, R));
    if (d->top_k < 1 || d->top_k > RC_MAX_TOP_K) return bad(what, fmt("top_k %lld outside [1, 16]", d->top_k));
    if (d->width < 1 || d->width > RC_MAX_MOE_WIDTH) return bad(what, fmt("width %lld outside [1, 65536]", d->width));
    if (d->inner < 1 || d->inner > RC_MAX_MOE_WIDTH) return bad(what, fmt("inner %lld outside [1, 65536]", d->inner));
    RC_TRY(spans_of(what, R, d->tokens, d->top_k, &a->entries));
    const int64_t n = a->entries.total();
    if (n > RC_MAX_MOE_ENTRIES)
        return bad(what, fmt("%lld tokens times %lld choices: more than 2048 (a dispatch takes any number)", n / d->top_k, d->top_k));
    a->num_experts = d->num_experts;
    a->per_rank = d->num_experts / R;
    a->top_k = d->top_k;
    a->width = (int32_t)d->width;
    a->inner = (int32_t)d->inner;
    a->out_dtype = d->out_dtype;
    a->hidden_row = (int32_t)((d->inner + 63) / 64 * 64);
    a->hidden_plane = n * a->hidden_row * 2;
    // float32 outputs of 8-bit rows: three bfloat16 numbers to a hidden value
    a->hidden_bytes = a->hidden_plane * (d->dtype == RC_E4M3 && d->out_dtype == RC_F32 ? 3 : 2);
    a->product_row = (int32_t)((d->width + 15) / 16 * 16);
    // the hidden values, the products, the lists
    const int64_t experts = std::min<int64_t>(n, d->num_experts);
    *workspace = a->hidden_bytes + n * a->product_row * 4 + experts * 16 + (n * 2 + 15) / 16 * 16;
    return {};
}

// ---------------------------------------------------------------- gradients

// One gradient's fields; *has: whether there is one.
Error check_grad(const char* what, const rc_grad& g, int rank, int i, bool* has) {
    *has = g.grad != nullptr && g.count > 0;
    auto wrong = [&](const std::string& how) { return bad(what, fmt("rank %lld, gradient %lld: ", rank, i) + how); };
    if (g.count < 0 || g.count > kMaxElements) return wrong(fmt("a count of %lld", g.count));
    if (!g.grad && g.count) return wrong("NULL");
    if (!*has) return {};
    const int64_t es = row_element_size(g.dtype);
    if (!es) return wrong(fmt("unknown dtype %lld", g.dtype));
    if (reinterpret_cast<uintptr_t>(g.grad) % (uintptr_t)es) return wrong("misaligned");
    if (reinterpret_cast<uintptr_t>(g.grad) >> 56) return wrong("no address of a GPU buffer");  // the byte holds the type
    return {};
}

template <class T>
Error check_lists(const char* what, int R, const int* n, const T* const* lists, const char* name) {
    RC_TRY(need(what, n, "counts"));
    RC_TRY(need(what, lists, name));
    int64_t all = 0;
    for (int r = 0; r < R; ++r) {
        if (n[r] < 0 || (all += n[r]) > kMaxTensors) return bad(what, fmt("rank %lld: %lld tensors", r, n[r]));
        if (n[r] && !lists[r]) return bad(what, fmt("rank %lld: NULL ", r) + name);
    }
    return {};
}

int64_t pieces(int64_t count, int64_t of) { return (count + of - 1) / of; }

Error check_grad_norm(const char* what, int R, const rc_grad_norm_desc* d, const int* n, const rc_grad* const* grads,
                      GradNormJoin* join) {
    RC_TRY(check_desc(what, d, "rc_grad_norm_desc"));
    RC_TRY(check_lists(what, R, n, grads, "gradients"));
    int64_t chunks = 0;
    for (int r = 0; r < R; ++r) {
        join->first[r] = chunks;
        for (int i = 0; i < n[r]; ++i) {
            bool has;
            RC_TRY(check_grad(what, grads[r][i], r, i, &has));
            if (has) chunks += pieces(grads[r][i].count, kNormChunk);
        }
    }
    for (int r = R; r <= kMaxRanks; ++r) join->first[r] = chunks;
    join->nranks = R;
    join->over_all = d->over_all != 0;
    return {};
}

// ---------------------------------------------------------------- AdamW

template <class T>
const T* part(const AdamwHeader* h, int64_t at) {
    return reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(h) + at);
}

// The first span that ends behind `lo`, if it starts before `hi`.
bool in_spans(const AdamwHeader* h, uint64_t lo, uint64_t hi) {
    const AdamwSpan *s = part<AdamwSpan>(h, h->spans_at), *end = s + h->spans;
    s = std::upper_bound(s, end, lo, [](uint64_t v, const AdamwSpan& x) { return v < x.hi; });
    return s != end && s->lo < hi;
}

Error check_table(const char* what, int R, const void* table, const void* on_gpu, const char* name) {
    RC_TRY(need(what, table, name));
    RC_TRY(need(what, on_gpu, name));
    const auto* h = static_cast<const AdamwHeader*>(table);
    if (reinterpret_cast<uintptr_t>(table) % 8 || h->magic != kAdamwMagic)
        return bad(what, std::string(name) + " was not written by rc_adamw_table");
    if (reinterpret_cast<uintptr_t>(on_gpu) % 16) return bad(what, std::string("misaligned ") + name);
    if (h->nranks != R) return bad(what, std::string(name) + fmt(" of %lld ranks, the session has %lld", h->nranks, R));
    return {};
}

Error same_parameters(const char* what, const AdamwHeader* a, const AdamwHeader* b) {
    bool same = a->bits == b->bits && a->chunks == b->chunks && a->entries_at == b->entries_at && a->chunks_at == b->chunks_at &&
                std::equal(a->first, a->first + kMaxRanks + 1, b->first);
    const auto *e = part<AdamwEntry>(a, a->entries_at), *o = part<AdamwEntry>(b, b->entries_at);
    for (int32_t i = 0; same && i < a->first[kMaxRanks]; ++i) same = e[i].count == o[i].count && e[i].dtype == o[i].dtype;
    if (!same) return bad(what, "the tables' parameters differ");
    const AdamwSpan *x = part<AdamwSpan>(a, a->spans_at), *y = part<AdamwSpan>(b, b->spans_at);
    for (int32_t i = 0, j = 0; i < a->spans && j < b->spans;) {
        if (x[i].lo < y[j].hi && y[j].lo < x[i].hi) return bad(what, "the tables share a buffer");
        if (x[i].hi <= y[j].hi) ++i;
        else ++j;
    }
    return {};
}

Error check_adamw(const char* what, const rc_adamw_desc* d) {
    RC_TRY(check_desc(what, d, "rc_adamw_desc"));
    if (!(d->lr >= 0) || !std::isfinite(d->lr)) return bad(what, "lr is not a number of at least 0");
    if (!(d->beta1 >= 0 && d->beta1 < 1) || !(d->beta2 >= 0 && d->beta2 < 1)) return bad(what, "a beta outside [0, 1)");
    if (!(d->eps >= 0) || !std::isfinite(d->eps)) return bad(what, "eps is not a number of at least 0");
    if (!std::isfinite(d->weight_decay)) return bad(what, "weight_decay is not finite");
    if (!(d->max_norm >= 0)) return bad(what, "max_norm is not a number of at least 0");
    if (d->max_norm > 0 && !d->norms) return bad(what, "max_norm without norms");
    if (!std::isfinite(d->grad_scale)) return bad(what, "grad_scale is not finite");
    return {};
}

}  // namespace

// 512 workgroups over all ranks, by their tokens: two for each CU, and their
// partial sums small beside the rows.
RankSpans norm_parts(const RankSpans& tokens) {
    constexpr int64_t kParts = 512;
    RankSpans p{};
    p.nranks = tokens.nranks;
    const int64_t total = tokens.total();
    int32_t sum = 0;
    for (int r = 0; r < kMaxRanks; ++r) {
        p.first[r] = sum;
        const int64_t n = (int64_t)tokens.first[r + 1] - tokens.first[r];
        if (n) sum += (int32_t)std::min(n, (kParts * n + total - 1) / total);
    }
    p.first[kMaxRanks] = sum;
    return p;
}

}  // namespace rc

using namespace rc;

extern "C" {

int rc_rms_norm(const rc_norm_desc* desc, const void* const* xs, const void* const* residuals,
                const void* const* weights, void* const* ys, float* const* scales, void* const* sums, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "rms_norm";
        NormArgs a{};
        RC_TRY(check_norm(what, R, desc, &a));
        RC_TRY(need(what, xs, "xs"));
        RC_TRY(need(what, weights, "weights"));
        RC_TRY(need(what, ys, "ys"));
        if (a.quantize) RC_TRY(need(what, scales, "scales"));
        if (!residuals != !sums) return bad(what, "residuals and sums are given together");
        a.has_residual = residuals != nullptr;
        const int64_t es = row_element_size(desc->dtype), ws = row_element_size(desc->weight_dtype);
        Buffers b(what);
        for (int r = 0; r < R; ++r) {
            const int64_t n = desc->tokens[r] * a.width;
            if (a.quantize || ys[r] != xs[r]) b.read(xs[r], n, es, "xs", r);
            if (desc->tokens[r]) b.read(weights[r], a.width, ws, "weights", r);
            b.write(ys[r], n, a.quantize ? 1 : es, "ys", r);
            if (a.quantize) b.write(scales[r], desc->tokens[r] * a.groups, 4, "scales", r);
            if (a.has_residual) {
                if (sums[r] != residuals[r]) b.read(residuals[r], n, es, "residuals", r);
                b.write(sums[r], n, es, "sums", r);
                a.residual[r] = residuals[r];
                a.sum[r] = sums[r];
            }
            a.x[r] = xs[r];
            a.weight[r] = weights[r];
            a.y[r] = ys[r];
            a.scale[r] = a.quantize ? scales[r] : nullptr;
        }
        RC_TRY(b.check());
        if (validate_only || !a.tokens.total()) return {};
        return device_run([&] { return launch_rms_norm(a, desc->dtype, desc->weight_dtype, stream); });
    });
}

int rc_rms_norm_grad_workspace(const rc_norm_desc* desc, int64_t* bytes) {
    return whole_call([&](int R, bool) -> Error {
        const char* what = "rms_norm_grad_workspace";
        NormArgs a{};
        RC_TRY(check_norm(what, R, desc, &a));
        RC_TRY(need(what, bytes, "bytes"));
        *bytes = norm_parts(a.tokens).total() * a.width * 4;
        return {};
    });
}

int rc_rms_norm_grad(const rc_norm_desc* desc, const void* const* d_ys, const void* const* sums,
                     const void* const* weights, const void* const* d_sums, void* const* d_xs, void* const* d_weights,
                     void* workspace, int64_t workspace_bytes, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "rms_norm_grad";
        NormArgs a{};
        RC_TRY(check_norm(what, R, desc, &a));
        RC_TRY(need(what, d_ys, "d_ys"));
        RC_TRY(need(what, sums, "sums"));
        RC_TRY(need(what, weights, "weights"));
        RC_TRY(need(what, d_xs, "d_xs"));
        RC_TRY(need(what, d_weights, "d_weights"));
        a.parts = norm_parts(a.tokens);
        a.has_residual = d_sums != nullptr;
        a.partial = static_cast<float*>(workspace);
        const int64_t es = row_element_size(desc->dtype), ws = row_element_size(desc->weight_dtype);
        Buffers b(what);
        RC_TRY(check_workspace(what, workspace, workspace_bytes, a.parts.total() * a.width * 4, &b));
        for (int r = 0; r < R; ++r) {
            const int64_t n = desc->tokens[r] * a.width;
            if (d_xs[r] != d_ys[r]) b.read(d_ys[r], n, es, "d_ys", r);
            b.read(sums[r], n, es, "sums", r);
            if (desc->tokens[r]) b.read(weights[r], a.width, ws, "weights", r);
            if (d_sums && d_sums[r] != d_xs[r]) b.read(d_sums[r], n, es, "d_sums", r);
            b.write(d_xs[r], n, es, "d_xs", r);
            b.write(d_weights[r], a.width, ws, "d_weights", r);
            a.d_y[r] = d_ys[r];
            a.x[r] = sums[r];
            a.weight[r] = weights[r];
            a.residual[r] = d_sums ? d_sums[r] : nullptr;
            a.y[r] = d_xs[r];
            a.d_weight[r] = d_weights[r];
        }
        RC_TRY(b.check());
        if (validate_only) return {};
        return device_run([&] { return launch_rms_norm_grad(a, desc->dtype, desc->weight_dtype, stream); });
    });
}

int rc_moe_layer_workspace(const rc_moe_desc* desc, int64_t* bytes) {
    return whole_call([&](int R, bool) -> Error {
        const char* what = "moe_layer_workspace";
        MoeArgs a{};
        int64_t ws = 0;
        RC_TRY(check_moe(what, R, desc, &a, &ws));
        RC_TRY(need(what, bytes, "bytes"));
        *bytes = ws;
        return {};
    });
}

int rc_moe_layer(const rc_moe_desc* desc, const void* const* xs, const float* const* scales,
                 const int32_t* const* experts, const float* const* weights, const void* const* gate_up,
                 const float* const* gate_up_scales, const void* const* down, const float* const* down_scales,
                 void* const* ys, void* workspace, int64_t workspace_bytes, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "moe_layer";
        MoeArgs a{};
        int64_t ws = 0;
        RC_TRY(check_moe(what, R, desc, &a, &ws));
        RC_TRY(need(what, xs, "xs"));
        RC_TRY(need(what, experts, "experts"));
        RC_TRY(need(what, weights, "weights"));
        RC_TRY(need(what, gate_up, "gate_up"));
        RC_TRY(need(what, down, "down"));
        RC_TRY(need(what, ys, "ys"));
        const bool rows8 = desc->dtype == RC_E4M3, weights8 = desc->weight_dtype == RC_E4M3;
        if (rows8 != (scales != nullptr)) return bad(what, "scales are given with 8-bit rows, and only then");
        if (weights8 != (gate_up_scales != nullptr) || weights8 != (down_scales != nullptr))
            return bad(what, "scales of the weights are given with 8-bit weights, and only then");
        Buffers b(what);
        RC_TRY(check_workspace(what, workspace, workspace_bytes, ws, &b));
        const int64_t xe = any_element_size(desc->dtype), we = any_element_size(desc->weight_dtype);
        const int64_t H = desc->width, I = desc->inner, per = a.per_rank, K = desc->top_k;
        for (int r = 0; r < R; ++r) {
            const int64_t n = desc->tokens[r];
            b.read(xs[r], n * H, xe, "xs", r);
            if (rows8) b.read(scales[r], n, 4, "scales", r);
            b.read(experts[r], n * K, 4, "experts", r);
            b.read(weights[r], n * K, 4, "weights", r);
            if (a.entries.total()) {
                b.read(gate_up[r], per * 2 * I * H, we, "gate_up", r);
                b.read(down[r], per * H * I, we, "down", r);
                if (weights8) b.read(gate_up_scales[r], per * 2 * I, 4, "gate_up_scales", r);
                if (weights8) b.read(down_scales[r], per * H, 4, "down_scales", r);
            }
            b.write(ys[r], n * H, row_element_size(desc->out_dtype), "ys", r);
            a.x[r] = xs[r];
            a.x_scale[r] = rows8 ? scales[r] : nullptr;
            a.experts[r] = experts[r];
            a.weights[r] = weights[r];
            a.gate_up[r] = gate_up[r];
            a.gate_up_scale[r] = weights8 ? gate_up_scales[r] : nullptr;
            a.down[r] = down[r];
            a.down_scale[r] = weights8 ? down_scales[r] : nullptr;
            a.y[r] = ys[r];
        }
        RC_TRY(b.check());
        const int64_t n = a.entries.total();
        a.hidden = static_cast<uint8_t*>(workspace);
        a.products = reinterpret_cast<float*>(a.hidden + a.hidden_bytes);
        a.lists = reinterpret_cast<uint8_t*>(a.products + n * a.product_row);
        if (validate_only || !a.entries.total()) return {};
        return device_run([&] { return launch_moe(a, desc->dtype, desc->weight_dtype, stream); });
    });
}

int rc_grad_norm_workspace(const rc_grad_norm_desc* desc, const int* num_grads, const rc_grad* const* grads,
                           int64_t* bytes) {
    return whole_call([&](int R, bool) -> Error {
        const char* what = "grad_norm_workspace";
        GradNormJoin join{};
        RC_TRY(check_grad_norm(what, R, desc, num_grads, grads, &join));
        RC_TRY(need(what, bytes, "bytes"));
        *bytes = join.first[kMaxRanks] * 8;
        return {};
    });
}

int rc_grad_norm(const rc_grad_norm_desc* desc, const int* num_grads, const rc_grad* const* grads, float* norms,
                 void* workspace, int64_t workspace_bytes, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "grad_norm";
        GradNormJoin join{};
        RC_TRY(check_grad_norm(what, R, desc, num_grads, grads, &join));
        Buffers b(what);
        RC_TRY(check_workspace(what, workspace, workspace_bytes, join.first[kMaxRanks] * 8, &b));
        b.write(norms, R, 4, "norms", 0);
        for (int r = 0; r < R; ++r)
            for (int i = 0; i < num_grads[r]; ++i)
                b.read(grads[r][i].grad, grads[r][i].count, std::max<int64_t>(1, row_element_size(grads[r][i].dtype)), "gradient", r);
        RC_TRY(b.check());
        if (validate_only) return {};
        join.partial = static_cast<const double*>(workspace);
        join.norms = norms;
        return device_run([&] {
            GradNormArgs a{};
            int64_t done = 0;
            auto flush = [&] {
                a.partial = static_cast<double*>(workspace) + done;
                const int e = a.n ? launch_grad_norm(a, stream) : 0;
                done += a.chunks;
                a.n = a.chunks = 0;
                return e;
            };
            for (int r = 0; r < R; ++r)
                for (int i = 0; i < num_grads[r]; ++i) {
                    const rc_grad& g = grads[r][i];
                    if (!g.grad || !g.count) continue;
                    for (int64_t at = 0; at < g.count; at += kNormPiece) {
                        const int64_t count = std::min(g.count - at, kNormPiece), chunks = pieces(count, kNormChunk);
                        if (a.n == kNormList || a.chunks + chunks > kMaxNormChunks)
                            if (const int e = flush()) return e;
                        a.grad[a.n] = (reinterpret_cast<uint64_t>(g.grad) + (uint64_t)(at * row_element_size(g.dtype))) | (uint64_t)g.dtype << 56;
                        a.count[a.n] = (int32_t)count;
                        a.first[a.n++] = a.chunks;
                        a.chunks += (int32_t)chunks;
                    }
                }
            if (const int e = flush()) return e;
            return launch_grad_norm_join(join, stream);
        });
    });
}

int rc_adamw_table(const rc_adamw_table_desc* desc, const int* num_params, const rc_adamw_param* const* params, void* table,
                   int64_t* bytes) {
    return whole_call([&](int R, bool) -> Error {
        const char* what = "adamw_table";
        RC_TRY(check_desc(what, desc, "rc_adamw_table_desc"));
        const int state_bits = desc->state_bits;
        if (state_bits != 32 && state_bits != 8) return bad(what, fmt("states of %lld bits, not 32 or 8", state_bits));
        RC_TRY(check_lists(what, R, num_params, params, "params"));
        RC_TRY(need(what, bytes, "bytes"));
        AdamwHeader h{};
        h.magic = kAdamwMagic;
        h.nranks = R;
        h.bits = state_bits;
        std::vector<AdamwEntry> entries;
        std::vector<AdamwSpan> spans;
        Buffers b(what);
        int64_t elements = 0;
        for (int r = 0; r < R; ++r)
            for (int i = 0; i < num_params[r]; ++i)
                elements += std::min(std::max<int64_t>(0, params[r][i].count), kMaxElements);
        h.chunk = kAdamwMost;
        while (h.chunk > kAdamwLeast && elements / h.chunk < 2048) h.chunk /= 2;
        for (int r = 0; r < R; ++r) {
            h.first[r] = (int32_t)entries.size();
            for (int i = 0; i < num_params[r]; ++i) {
                const rc_adamw_param& p = params[r][i];
                const std::string where = fmt("rank %lld, parameter %lld: ", r, i);
                const int64_t es = row_element_size(p.dtype), blocks = pieces(p.count, RC_ADAMW_BLOCK);
                if (p.count < 0 || p.count > kMaxElements) return bad(what, where + fmt("a count of %lld", p.count));
                if (!es) return bad(what, where + fmt("unknown dtype %lld", p.dtype));
                auto add = [&](const void* at, int64_t count, int64_t size, const char* name) {
                    b.write(at, count, size, name, r);
                    if (count)
                        spans.push_back({reinterpret_cast<uintptr_t>(at), reinterpret_cast<uintptr_t>(at) + (uint64_t)(count * size)});
                };
                add(p.param, p.count, es, "param");
                if (p.dtype != RC_F32) add(p.master, p.count, 4, "master");
                add(p.m, p.count, state_bits / 8, "m");
                add(p.v, p.count, state_bits / 8, "v");
                if (state_bits == 8) {
                    add(p.m_scale, blocks, 4, "m_scale");
                    add(p.v_scale, blocks, 4, "v_scale");
                }
                entries.push_back({p.param, p.master, p.m, p.v, p.m_scale, p.v_scale, p.count, h.chunks, p.dtype, r});
                h.chunks += pieces(p.count, h.chunk);
                if (h.chunks > kMaxItems) return bad(what, "too many elements for one table");
            }
        }
        RC_TRY(b.check());
        for (int r = R; r <= kMaxRanks; ++r) h.first[r] = (int32_t)entries.size();
        // spans in order, those that touch as one
        std::sort(spans.begin(), spans.end(), [](const AdamwSpan& x, const AdamwSpan& y) { return x.lo < y.lo; });
        size_t kept = 0;
        for (size_t i = 0; i < spans.size(); ++i) {
            if (kept && spans[kept - 1].hi >= spans[i].lo) spans[kept - 1].hi = spans[i].hi;
            else spans[kept++] = spans[i];
        }
        h.spans = (int32_t)kept;
        h.entries_at = (int64_t)sizeof h;
        h.chunks_at = h.entries_at + (int64_t)(entries.size() * sizeof(AdamwEntry));
        h.spans_at = (h.chunks_at + h.chunks * 4 + 15) / 16 * 16;
        h.bytes = h.spans_at + (int64_t)(kept * sizeof(AdamwSpan));
        if (!table) {
            *bytes = h.bytes;
            return {};
        }
        if (*bytes < h.bytes) return bad(what, fmt("a table of %lld bytes, needs %lld", *bytes, h.bytes));
        if (reinterpret_cast<uintptr_t>(table) % 8) return bad(what, "misaligned table");
        uint8_t* at = static_cast<uint8_t*>(table);
        std::memcpy(at, &h, sizeof h);
        if (!entries.empty()) std::memcpy(at + h.entries_at, entries.data(), entries.size() * sizeof(AdamwEntry));
        auto* map = reinterpret_cast<int32_t*>(at + h.chunks_at);
        for (size_t i = 0; i < entries.size(); ++i) map = std::fill_n(map, pieces(entries[i].count, h.chunk), (int32_t)i);
        std::fill(reinterpret_cast<uint8_t*>(map), at + h.spans_at, uint8_t(0));
        if (kept) std::memcpy(at + h.spans_at, spans.data(), kept * sizeof(AdamwSpan));
        return {};
    });
}

int rc_adamw_step(const rc_adamw_desc* desc, const void* table, void* table_on_gpu, const void* out_table,
                  const void* out_table_on_gpu, const rc_grad* const* grads, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "adamw_step";
        RC_TRY(check_adamw(what, desc));
        RC_TRY(check_table(what, R, table, table_on_gpu, "table"));
        RC_TRY(check_table(what, R, out_table, out_table_on_gpu, "out_table"));
        RC_TRY(need(what, grads, "gradients"));
        const auto *from = static_cast<const AdamwHeader*>(table), *to = static_cast<const AdamwHeader*>(out_table);
        const bool in_place = table_on_gpu == out_table_on_gpu;
        if (in_place != (table == out_table)) return bad(what, "the tables on the host and on the GPU do not belong together");
        if (!in_place) RC_TRY(same_parameters(what, from, to));
        Buffers b(what);
        auto small = [&](const void* p, int64_t n, const char* name, bool out) -> Error {
            if (out) b.write(p, n, 4, name, 0);
            else b.read(p, n, 4, name, 0);
            const auto lo = reinterpret_cast<uintptr_t>(p);
            const uint64_t hi = lo + (uint64_t)n * 4;
            if (in_spans(to, lo, hi) || (out && in_spans(from, lo, hi))) return bad(what, std::string(name) + " overlap a parameter's buffers");
            return {};
        };
        if (desc->steps != desc->steps_out) RC_TRY(small(desc->steps, R, "steps", false));
        RC_TRY(small(desc->steps_out, R, "steps_out", true));
        if (desc->norms) RC_TRY(small(desc->norms, R, "norms", false));
        if (desc->lr_on_gpu) RC_TRY(small(desc->lr_on_gpu, 1, "lr", false));
        b.write(table_on_gpu, from->bytes, 1, "table", 0);
        if (!in_place) b.read(out_table_on_gpu, to->bytes, 1, "out_table", 0);
        RC_TRY(b.check());
        // neither of the tables may be stepped over, nor a gradient written before it is read
        struct Small {
            uintptr_t lo, hi;
            const char* name;
        };
        const auto at = [](const void* p, int64_t bytes, const char* name) {
            return Small{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes, name};
        };
        const Small smalls[] = {at(table_on_gpu, from->bytes, "the table"), at(out_table_on_gpu, to->bytes, "the out_table"),
                                at(desc->steps_out, (int64_t)R * 4, "steps_out")};
        for (const Small& s : smalls)
            if (in_spans(to, s.lo, s.hi) || in_spans(from, s.lo, s.hi))
                return bad(what, std::string(s.name) + " overlaps a parameter's buffers");
        const AdamwEntry* entries = part<AdamwEntry>(from, from->entries_at);
        for (int r = 0; r < R; ++r) {
            const int n = from->first[r + 1] - from->first[r];
            if (n && !grads[r]) return bad(what, fmt("rank %lld: NULL gradients", r));
            for (int i = 0; i < n; ++i) {
                const rc_grad& g = grads[r][i];
                const AdamwEntry& e = entries[from->first[r] + i];
                bool has;
                RC_TRY(check_grad(what, g, r, i, &has));
                if (!has) continue;
                auto wrong = [&](const std::string& how) { return bad(what, fmt("rank %lld, gradient %lld: ", r, i) + how); };
                if (g.count != e.count) return wrong(fmt("%lld elements, the parameter has %lld", g.count, e.count));
                if (g.dtype != RC_F32 && g.dtype != e.dtype) return wrong(fmt("dtype %lld is neither RC_F32 nor the parameter's", g.dtype));
                const auto lo = reinterpret_cast<uintptr_t>(g.grad), hi = lo + (uintptr_t)(g.count * row_element_size(g.dtype));
                if (in_spans(to, lo, hi)) return wrong("overlaps a parameter's buffers");
                for (const Small& s : smalls)
                    if (lo < s.hi && s.lo < hi) return wrong(std::string("overlaps ") + s.name);
            }
        }
        if (validate_only) return {};
        return device_run([&] {
            AdamwBegin begin{static_cast<AdamwHeader*>(table_on_gpu), desc->lr, desc->beta1, desc->beta2, desc->weight_decay,
                             desc->max_norm, desc->grad_scale, desc->lr_on_gpu, desc->norms, desc->steps, desc->steps_out,
                             desc->seed, R};
            if (const int e = launch_adamw_begin(begin, stream)) return e;
            AdamwArgs a{};
            a.table = static_cast<const AdamwHeader*>(table_on_gpu);
            a.out = static_cast<const AdamwHeader*>(out_table_on_gpu);
            a.entries_at = from->entries_at;
            a.chunks_at = from->chunks_at;
            a.chunk = from->chunk;
            a.beta1 = (float)desc->beta1;
            a.rest1 = (float)(1.0 - desc->beta1);
            a.beta2 = (float)desc->beta2;
            a.rest2 = (float)(1.0 - desc->beta2);
            a.eps = (float)desc->eps;
            const int32_t all = from->first[kMaxRanks];
            for (int32_t first = 0; first < all; first += kAdamwList) {
                const int32_t end = std::min(all, first + kAdamwList);
                bool any = !in_place;
                for (int32_t i = first, r = 0; i < end; ++i) {
                    while (i >= from->first[r + 1]) ++r;
                    const rc_grad& g = grads[r][i - from->first[r]];
                    const bool has = g.grad && g.count;
                    any |= has;
                    a.grad[i - first] = has ? reinterpret_cast<uint64_t>(g.grad) | (uint64_t)g.dtype << 56 : 0;
                }
                a.first = first;
                a.first_chunk = entries[first].first_chunk;
                a.chunks = (end < all ? entries[end].first_chunk : from->chunks) - a.first_chunk;
                if (!any || !a.chunks) continue;
                if (const int e = launch_adamw(a, from->bits, stream)) return e;
            }
            return 0;
        });
    });
}

}  // extern "C"
