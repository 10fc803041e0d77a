// Entry points and argument checks of the block operators.  Host-only C++; the
// kernels are reached through the launch_* functions of blocks.h.  Everything
// is checked before anything is enqueued.
#include "blocks.h"

#include <algorithm>
#include <cmath>

#include "rows_check.h"

namespace rc {
namespace {

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

}  // extern "C"
