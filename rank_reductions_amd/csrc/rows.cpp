// Entry points and argument checks of the row exchanges (expert routing,
// dispatch and combine, the sharded embedding lookup and its gradient).
// Host-only C++; the kernels are reached through the launch_* functions of
// rows.h.  Everything is checked before anything is enqueued.
#include "rows.h"

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdio>
#include <string>
#include <vector>

namespace rc {
namespace {

constexpr int64_t kMaxItems = 0x7fffffff;              // counts fit 32 bits
constexpr int64_t kMaxWidth = int64_t(1) << 22;        // elements of a row
constexpr int64_t kMaxCapacity = 0x7fffffff;

std::string fmt(const char* f, long long a = 0, long long b = 0, long long c = 0) {
    char buf[256];
    std::snprintf(buf, sizeof buf, f, a, b, c);
    return buf;
}

Error bad(const char* what, const std::string& msg) {
    return Error{RC_ERR_INVALID_ARGUMENT, std::string(what) + ": " + msg};
}

// Collects a call's buffers: each must be there and aligned if it has
// elements, and no output may overlap another buffer.
class Buffers {
  public:
    explicit Buffers(const char* what) : what_(what) { at_.reserve(6 * kMaxRanks); }
    void read(const void* p, int64_t count, int64_t es, const char* name, int rank) { add(p, count, es, name, rank, false); }
    void write(const void* p, int64_t count, int64_t es, const char* name, int rank) { add(p, count, es, name, rank, true); }
    Error check() {
        if (err_.code) return err_;
        std::sort(at_.begin(), at_.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
        // the furthest ends of the writes, and of all buffers, before each
        const Span *w = nullptr, *any = nullptr;
        for (const Span& s : at_) {
            const Span* hit = w && w->hi > s.lo ? w : (s.out && any && any->hi > s.lo ? any : nullptr);
            if (hit)
                return bad(what_, std::string(hit->name) + fmt(" of rank %lld overlaps ", hit->rank) + s.name +
                                      fmt(" of rank %lld", s.rank));
            if (s.out && (!w || s.hi > w->hi)) w = &s;
            if (!any || s.hi > any->hi) any = &s;
        }
        return {};
    }

  private:
    struct Span {
        uintptr_t lo, hi;
        const char* name;
        int rank;
        bool out;
    };
    void add(const void* p, int64_t count, int64_t es, const char* name, int rank, bool out) {
        if (err_.code || count <= 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (!p) err_ = bad(what_, fmt("rank %lld: NULL ", rank) + name);
        else if (lo % (uintptr_t)es) err_ = bad(what_, fmt("rank %lld: misaligned ", rank) + name);
        else at_.push_back({lo, lo + (uintptr_t)(count * es), name, rank, out});
    }
    const char* what_;
    std::vector<Span> at_;
    Error err_;
};

// The ranks' counts times `each`, as spans.
Error spans_of(const char* what, int R, const int64_t* counts, int64_t each, RankSpans* out) {
    if (!counts) return bad(what, "NULL tokens");
    int64_t sum = 0;
    for (int r = 0; r < R; ++r) {
        if (counts[r] < 0) return bad(what, fmt("rank %lld: negative token count", r));
        if (counts[r] > kMaxItems || sum + counts[r] * each > kMaxItems)
            return bad(what, "more than 2^31 - 1 entries over all ranks");
        out->first[r] = (int32_t)sum;
        sum += counts[r] * each;
    }
    for (int r = R; r <= kMaxRanks; ++r) out->first[r] = (int32_t)sum;
    out->nranks = R;
    return {};
}

template <class P>
Error need(const char* what, P* p, const char* name) {
    return p ? Error{} : bad(what, std::string("NULL ") + name);
}

#define RC_TRY(expr)              \
    do {                          \
        Error rc_e_ = (expr);     \
        if (rc_e_.code) return rc_e_; \
    } while (0)

// A descriptor's size, and the session that its arrays were made for.
template <class D>
Error check_desc(const char* what, const D* d, const char* type) {
    RC_TRY(need(what, d, "desc"));
    if (d->struct_size == offsetof(D, session)) return {};
    if (d->struct_size != sizeof(D)) return bad(what, std::string("desc->struct_size must be sizeof(") + type + ")");
    if (d->session && d->session != session_id())
        return bad(what, "the session that the call was made for has been closed, and another is open");
    return {};
}

// ---------------------------------------------------------------- routing

Error check_route(const char* what, int R, const rc_route_desc* d, const int64_t* tokens, RouteArgs* a) {
    RC_TRY(check_desc(what, d, "rc_route_desc"));
    if (!row_element_size(d->dtype)) return bad(what, fmt("unknown dtype %lld", d->dtype));
    if (d->num_experts < 1 || d->num_experts > RC_MAX_EXPERTS) return bad(what, fmt("num_experts %lld outside [1, 1024]", d->num_experts));
    if (d->top_k < 1 || d->top_k > RC_MAX_TOP_K) return bad(what, fmt("top_k %lld outside [1, 16]", d->top_k));
    if (d->score != RC_SCORE_SOFTMAX && d->score != RC_SCORE_SIGMOID) return bad(what, "unknown score");
    if (d->num_groups < 1 || d->num_groups > RC_MAX_EXPERT_GROUPS || d->num_experts % d->num_groups)
        return bad(what, fmt("num_groups %lld outside [1, 64] or no divisor of num_experts", d->num_groups));
    if (d->top_groups < 1 || d->top_groups > d->num_groups) return bad(what, "top_groups outside [1, num_groups]");
    if (d->group_by != RC_GROUP_MAX && d->group_by != RC_GROUP_TOP2) return bad(what, "unknown group_by");
    if (d->top_k > d->top_groups * (d->num_experts / d->num_groups))
        return bad(what, fmt("top_k %lld exceeds the experts of top_groups groups", d->top_k));
    if (!std::isfinite(d->scale)) return bad(what, "scale is not finite");
    if (reinterpret_cast<uintptr_t>(d->bias) % 4) return bad(what, "misaligned bias");
    // entries are counted by token * num_experts at most in 64 bits; by token in 32
    RC_TRY(spans_of(what, R, tokens, 1, &a->tokens));
    a->bias = d->bias;
    a->num_experts = d->num_experts;
    a->top_k = d->top_k;
    a->sigmoid = d->score == RC_SCORE_SIGMOID;
    a->groups = d->num_groups;
    a->top_groups = d->top_groups;
    a->top2 = d->group_by == RC_GROUP_TOP2;
    a->renormalize = d->renormalize != 0;
    a->scale = d->scale;
    a->group_size = d->num_experts / d->num_groups;
    return {};
}

// Whether every rank's rows of num_experts elements start on 4-element boundaries.
bool rows_of_four(const void* const* p, const int64_t* tokens, int R, int64_t experts, int64_t es) {
    if (experts % 4) return false;
    for (int r = 0; r < R; ++r)
        if (tokens[r] && reinterpret_cast<uintptr_t>(p[r]) % (uintptr_t)(4 * es)) return false;
    return true;
}

// ---------------------------------------------------------------- exchange

struct Exchange {
    ExchangeArgs a{};
    RankSpans entries{};  // tokens * top_k
    int64_t es = 0;
};

Error check_exchange(const char* what, int R, const rc_exchange_desc* d, bool plan, Exchange* x) {
    RC_TRY(check_desc(what, d, "rc_exchange_desc"));
    x->es = row_element_size(d->dtype);
    if (!plan) {
        if (!x->es) return bad(what, fmt("unknown dtype %lld", d->dtype));
        if (d->width < 1 || d->width > kMaxWidth) return bad(what, fmt("width %lld outside [1, 2^22]", d->width));
    }
    if (d->num_experts < 1 || d->num_experts > RC_MAX_EXPERTS || d->num_experts % R)
        return bad(what, fmt("num_experts %lld outside [1, 1024] or not divisible by the %lld ranks", d->num_experts, R));
    if (d->top_k < 1 || d->top_k > RC_MAX_TOP_K) return bad(what, fmt("top_k %lld outside [1, 16]", d->top_k));
    RC_TRY(spans_of(what, R, d->tokens, 1, &x->a.tokens));
    RC_TRY(spans_of(what, R, d->tokens, d->top_k, &x->entries));
    RC_TRY(need(what, d->capacity, "capacity"));
    for (int r = 0; r < R; ++r) {
        if (d->capacity[r] < 0 || d->capacity[r] > kMaxCapacity)
            return bad(what, fmt("rank %lld: capacity outside [0, 2^31 - 1]", r));
        x->a.capacity[r] = d->capacity[r];
    }
    RC_TRY(need(what, d->experts, "experts"));
    RC_TRY(need(what, d->slots, "slots"));
    for (int r = 0; r < R; ++r) {
        x->a.experts[r] = d->experts[r];
        x->a.slots[r] = d->slots[r];
    }
    x->a.num_experts = d->num_experts;
    x->a.per_rank = d->num_experts / R;
    x->a.top_k = d->top_k;
    x->a.width = d->width;
    return {};
}

// The index buffers of a call that follows a plan.
void read_plan(const rc_exchange_desc* d, int R, Buffers* b) {
    for (int r = 0; r < R; ++r) {
        b->read(d->experts[r], d->tokens[r] * d->top_k, 4, "experts", r);
        b->read(d->slots[r], d->tokens[r] * d->top_k, 4, "slots", r);
    }
}

// ---------------------------------------------------------------- embedding

struct Embedding {
    RankSpans tokens{};
    int64_t es = 0, ges = 0, ides = 0, shard = 0;
    int64_t rows(int r, int64_t vocab) const { return std::max<int64_t>(0, std::min((r + 1) * shard, vocab) - r * shard); }
};

Error check_embedding(const char* what, int R, const rc_embedding_desc* d, bool grad, bool with_ids, Embedding* x) {
    RC_TRY(check_desc(what, d, "rc_embedding_desc"));
    x->es = row_element_size(d->dtype);
    if (!x->es) return bad(what, fmt("unknown dtype %lld", d->dtype));
    if (d->id_dtype != RC_I32 && d->id_dtype != RC_I64) return bad(what, fmt("unknown id_dtype %lld", d->id_dtype));
    x->ides = d->id_dtype == RC_I64 ? 8 : 4;
    if (grad) {
        if (d->grad_dtype != RC_F32 && d->grad_dtype != d->dtype)
            return bad(what, fmt("grad_dtype %lld is neither RC_F32 nor dtype", d->grad_dtype));
        x->ges = row_element_size(d->grad_dtype);
    }
    if (d->vocab < 1 || d->vocab > kMaxItems - 1) return bad(what, "vocab outside [1, 2^31 - 2]");
    if (d->width < 1 || d->width > kMaxWidth) return bad(what, fmt("width %lld outside [1, 2^22]", d->width));
    if (!std::isfinite(d->scale)) return bad(what, "scale is not finite");
    RC_TRY(spans_of(what, R, d->tokens, 1, &x->tokens));
    if (with_ids) RC_TRY(need(what, d->ids, "ids"));
    x->shard = (d->vocab + R - 1) / R;
    return {};
}

}  // namespace

RankSpans sort_blocks(const RankSpans& entries) {
    RankSpans b{};
    int32_t sum = 0;
    for (int r = 0; r < kMaxRanks; ++r) {
        b.first[r] = sum;
        sum += (int32_t)(((int64_t)entries.first[r + 1] - entries.first[r] + (kSortBlock - 1)) / kSortBlock);
    }
    b.first[kMaxRanks] = sum;
    b.nranks = entries.nranks;
    return b;
}

}  // namespace rc

using namespace rc;

extern "C" {

int rc_route(const rc_route_desc* desc, const int64_t* tokens, const void* const* logits, float* const* weights,
             int32_t* const* experts, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "route";
        RouteArgs a{};
        RC_TRY(check_route(what, R, desc, tokens, &a));
        RC_TRY(need(what, logits, "logits"));
        RC_TRY(need(what, weights, "weights"));
        RC_TRY(need(what, experts, "experts"));
        const int64_t es = row_element_size(desc->dtype), E = desc->num_experts, K = desc->top_k;
        Buffers b(what);
        if (a.tokens.total()) b.read(desc->bias, desc->bias ? E : 0, 4, "bias", 0);
        for (int r = 0; r < R; ++r) {
            b.read(logits[r], tokens[r] * E, es, "logits", r);
            b.write(weights[r], tokens[r] * K, 4, "weights", r);
            b.write(experts[r], tokens[r] * K, 4, "experts", r);
            a.logits[r] = logits[r];
            a.weights[r] = weights[r];
            a.experts[r] = experts[r];
        }
        RC_TRY(b.check());
        a.vec = rows_of_four(logits, tokens, R, E, es) && a.group_size % 4 == 0;
        a.bias_vec = a.group_size % 4 == 0 && reinterpret_cast<uintptr_t>(desc->bias) % 16 == 0;
        if (validate_only || !a.tokens.total()) return {};
        return device_run([&] { return launch_route(a, desc->dtype, stream); });
    });
}

int rc_route_grad(const rc_route_desc* desc, const int64_t* tokens, const void* const* logits,
                  const int32_t* const* experts, const float* const* d_weights, void* const* d_logits, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "route_grad";
        RouteArgs a{};
        RC_TRY(check_route(what, R, desc, tokens, &a));
        RC_TRY(need(what, logits, "logits"));
        RC_TRY(need(what, experts, "experts"));
        RC_TRY(need(what, d_weights, "d_weights"));
        RC_TRY(need(what, d_logits, "d_logits"));
        const int64_t es = row_element_size(desc->dtype), E = desc->num_experts, K = desc->top_k;
        Buffers b(what);
        for (int r = 0; r < R; ++r) {
            b.read(logits[r], tokens[r] * E, es, "logits", r);
            b.read(experts[r], tokens[r] * K, 4, "experts", r);
            b.read(d_weights[r], tokens[r] * K, 4, "d_weights", r);
            b.write(d_logits[r], tokens[r] * E, es, "d_logits", r);
            a.logits[r] = logits[r];
            a.experts[r] = const_cast<int32_t*>(experts[r]);
            a.d_weights[r] = d_weights[r];
            a.d_logits[r] = d_logits[r];
        }
        RC_TRY(b.check());
        a.vec = rows_of_four(logits, tokens, R, E, es) &&
                rows_of_four(const_cast<const void* const*>(d_logits), tokens, R, E, es);
        if (validate_only || !a.tokens.total()) return {};
        return device_run([&] { return launch_route_grad(a, desc->dtype, stream); });
    });
}

int rc_dispatch_plan_workspace(const rc_exchange_desc* desc, int64_t* bytes) {
    return whole_call([&](int R, bool) -> Error {
        const char* what = "dispatch_plan_workspace";
        Exchange x;
        RC_TRY(check_exchange(what, R, desc, true, &x));
        RC_TRY(need(what, bytes, "bytes"));
        *bytes = plan_workspace_bytes(x.entries, desc->num_experts);
        return {};
    });
}

int rc_dispatch_plan(const rc_exchange_desc* desc, int32_t* const* offsets, int32_t* const* counts, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "dispatch_plan";
        Exchange x;
        RC_TRY(check_exchange(what, R, desc, true, &x));
        RC_TRY(need(what, offsets, "offsets"));
        RC_TRY(need(what, counts, "counts"));
        const int64_t ws = plan_workspace_bytes(x.entries, desc->num_experts);
        if (workspace_bytes < ws) return bad(what, fmt("workspace of %lld bytes, needs %lld", workspace_bytes, ws));
        PlanArgs a{};
        Buffers b(what);
        b.write(workspace, ws, 1, "workspace", 0);
        if (ws && reinterpret_cast<uintptr_t>(workspace) % 16) return bad(what, "misaligned workspace");
        for (int r = 0; r < R; ++r) {
            const int64_t n = desc->tokens[r] * desc->top_k;
            b.read(desc->experts[r], n, 4, "experts", r);
            b.write(desc->slots[r], n, 4, "slots", r);
            b.write(offsets[r], x.a.per_rank + 1, 4, "offsets", r);
            b.write(counts[r], x.a.per_rank, 4, "counts", r);
            a.sort.ids[r] = desc->experts[r];
            a.slots[r] = desc->slots[r];
            a.offsets[r] = offsets[r];
            a.counts[r] = counts[r];
            a.capacity[r] = desc->capacity[r];
        }
        RC_TRY(b.check());
        a.sort.spans = x.entries;
        a.sort.key_limit = desc->num_experts;
        a.num_experts = desc->num_experts;
        a.per_rank = x.a.per_rank;
        if (validate_only) return {};
        return device_run([&] { return launch_plan(a, workspace, stream); });
    });
}

int rc_dispatch(const rc_exchange_desc* desc, const void* const* xs, void* const* rows, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "dispatch";
        Exchange x;
        RC_TRY(check_exchange(what, R, desc, false, &x));
        RC_TRY(need(what, xs, "xs"));
        RC_TRY(need(what, rows, "rows"));
        Buffers b(what);
        read_plan(desc, R, &b);
        for (int r = 0; r < R; ++r) {
            b.read(xs[r], desc->tokens[r] * desc->width, x.es, "xs", r);
            b.write(rows[r], desc->capacity[r] * desc->width, x.es, "rows", r);
            x.a.in[r] = xs[r];
            x.a.out[r] = rows[r];
        }
        RC_TRY(b.check());
        if (validate_only || !x.a.tokens.total()) return {};
        return device_run([&] { return launch_dispatch(x.a, desc->dtype, stream); });
    });
}

int rc_combine(const rc_exchange_desc* desc, const void* const* rows, const float* const* weights,
               void* const* outs, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "combine";
        Exchange x;
        RC_TRY(check_exchange(what, R, desc, false, &x));
        RC_TRY(need(what, rows, "rows"));
        RC_TRY(need(what, outs, "outs"));
        Buffers b(what);
        read_plan(desc, R, &b);
        for (int r = 0; r < R; ++r) {
            b.read(rows[r], desc->capacity[r] * desc->width, x.es, "rows", r);
            if (weights) b.read(weights[r], desc->tokens[r] * desc->top_k, 4, "weights", r);
            b.write(outs[r], desc->tokens[r] * desc->width, x.es, "outs", r);
            x.a.in[r] = rows[r];
            x.a.weights[r] = weights ? weights[r] : nullptr;
            x.a.out[r] = outs[r];
        }
        x.a.weighted = weights != nullptr;
        RC_TRY(b.check());
        if (validate_only || !x.a.tokens.total()) return {};
        return device_run([&] { return launch_combine(x.a, desc->dtype, stream); });
    });
}

int rc_combine_grad(const rc_exchange_desc* desc, const void* const* d_outs, const void* const* rows,
                    const float* const* weights, void* const* d_rows, float* const* d_weights, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "combine_grad";
        Exchange x;
        RC_TRY(check_exchange(what, R, desc, false, &x));
        RC_TRY(need(what, d_outs, "d_outs"));
        RC_TRY(need(what, rows, "rows"));
        RC_TRY(need(what, weights, "weights"));
        RC_TRY(need(what, d_rows, "d_rows"));
        RC_TRY(need(what, d_weights, "d_weights"));
        Buffers b(what);
        read_plan(desc, R, &b);
        for (int r = 0; r < R; ++r) {
            b.read(d_outs[r], desc->tokens[r] * desc->width, x.es, "d_outs", r);
            b.read(rows[r], desc->capacity[r] * desc->width, x.es, "rows", r);
            b.read(weights[r], desc->tokens[r] * desc->top_k, 4, "weights", r);
            b.write(d_rows[r], desc->capacity[r] * desc->width, x.es, "d_rows", r);
            b.write(d_weights[r], desc->tokens[r] * desc->top_k, 4, "d_weights", r);
            x.a.d_out[r] = d_outs[r];
            x.a.in[r] = rows[r];
            x.a.weights[r] = weights[r];
            x.a.out[r] = d_rows[r];
            x.a.d_weights[r] = d_weights[r];
        }
        x.a.weighted = 1;
        RC_TRY(b.check());
        if (validate_only || !x.a.tokens.total()) return {};
        return device_run([&] { return launch_combine_grad(x.a, desc->dtype, stream); });
    });
}

int rc_embedding(const rc_embedding_desc* desc, const void* const* tables, void* const* outs, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "embedding";
        Embedding x;
        RC_TRY(check_embedding(what, R, desc, false, true, &x));
        RC_TRY(need(what, tables, "tables"));
        RC_TRY(need(what, outs, "outs"));
        EmbeddingArgs a{};
        Buffers b(what);
        for (int r = 0; r < R; ++r) {
            b.read(desc->ids[r], desc->tokens[r], x.ides, "ids", r);
            b.read(tables[r], x.rows(r, desc->vocab) * desc->width, x.es, "table", r);
            b.write(outs[r], desc->tokens[r] * desc->width, x.es, "outs", r);
            a.ids[r] = desc->ids[r];
            a.table[r] = tables[r];
            a.out[r] = outs[r];
        }
        RC_TRY(b.check());
        a.tokens = x.tokens;
        a.vocab = desc->vocab;
        a.shard = x.shard;
        a.width = desc->width;
        a.scale = desc->scale;
        a.id64 = desc->id_dtype == RC_I64;
        if (validate_only || !a.tokens.total()) return {};
        return device_run([&] { return launch_embedding(a, desc->dtype, stream); });
    });
}

int rc_embedding_grad_workspace(const rc_embedding_desc* desc, int64_t* bytes) {
    return whole_call([&](int R, bool) -> Error {
        const char* what = "embedding_grad_workspace";
        Embedding x;
        RC_TRY(check_embedding(what, R, desc, true, false, &x));
        RC_TRY(need(what, bytes, "bytes"));
        *bytes = embedding_grad_workspace_bytes(x.tokens, desc->vocab, desc->width);
        return {};
    });
}

int rc_embedding_grad(const rc_embedding_desc* desc, const void* const* d_outs, void* const* d_tables,
                      void* workspace, int64_t workspace_bytes, void* stream) {
    return whole_call([&](int R, bool validate_only) -> Error {
        const char* what = "embedding_grad";
        Embedding x;
        RC_TRY(check_embedding(what, R, desc, true, true, &x));
        RC_TRY(need(what, d_outs, "d_outs"));
        RC_TRY(need(what, d_tables, "d_tables"));
        const int64_t ws = embedding_grad_workspace_bytes(x.tokens, desc->vocab, desc->width);
        if (workspace_bytes < ws) return bad(what, fmt("workspace of %lld bytes, needs %lld", workspace_bytes, ws));
        EmbeddingGradArgs a{};
        SortPass sort{};
        Buffers b(what);
        b.write(workspace, ws, 1, "workspace", 0);
        if (ws && reinterpret_cast<uintptr_t>(workspace) % 16) return bad(what, "misaligned workspace");
        for (int r = 0; r < R; ++r) {
            b.read(desc->ids[r], desc->tokens[r], x.ides, "ids", r);
            b.read(d_outs[r], desc->tokens[r] * desc->width, x.es, "d_outs", r);
            b.write(d_tables[r], x.rows(r, desc->vocab) * desc->width, x.ges, "d_tables", r);
            sort.ids[r] = desc->ids[r];
            a.d_out[r] = d_outs[r];
            a.table[r] = d_tables[r];
        }
        RC_TRY(b.check());
        sort.spans = x.tokens;
        sort.id64 = desc->id_dtype == RC_I64;
        sort.key_limit = desc->vocab;
        a.tokens = x.tokens;
        a.vocab = desc->vocab;
        a.shard = x.shard;
        a.width = desc->width;
        a.scale = desc->scale;
        a.accumulate = desc->accumulate != 0;
        if (validate_only || (a.accumulate && !a.tokens.total())) return {};
        return device_run(
            [&] { return launch_embedding_grad(a, sort, desc->dtype, desc->grad_dtype, workspace, stream); });
    });
}

}  // extern "C"
