// Host-only stress of the block operators' entry points (no GPU): several threads
// make random calls, most of them valid, some with one thing wrong.  The
// kernels are stubs that check what a launch may rely on; an AdamW table's copy on
// the GPU is the host's own, so the stub walks it as the kernel does.  Built with
// sanitizers by the tests; links blocks.cpp, rows.cpp, session.cpp, validate.cpp
// and plan.cpp.
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <thread>
#include <vector>

#include "blocks.h"
#include "rc.h"

namespace {
std::atomic<int> g_bad{0}, g_launched{0};

#define CHECK(x)                                                      \
    do {                                                              \
        if (!(x)) {                                                   \
            ++g_bad;                                                  \
            std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x);       \
        }                                                             \
    } while (0)

constexpr int R = 3;

void check_spans(const rc::RankSpans& s) {
    CHECK(s.nranks == R && s.first[0] == 0);
    for (int r = 0; r < rc::kMaxRanks; ++r) CHECK(s.first[r] <= s.first[r + 1]);
    CHECK(s.first[R] == s.total());
}
int norm_ok(const rc::NormArgs& a, bool grad) {
    check_spans(a.tokens);
    CHECK(a.width >= 1 && a.width <= RC_MAX_NORM_WIDTH);
    if (grad) {
        check_spans(a.parts);
        for (int r = 0; r < R; ++r) {
            const int n = a.tokens.first[r + 1] - a.tokens.first[r], p = a.parts.first[r + 1] - a.parts.first[r];
            CHECK(p <= n && (n == 0 || p > 0) && a.d_weight[r]);
        }
        CHECK(a.parts.total() <= 512 + R && (a.partial || !a.parts.total()));
    } else {
        CHECK(a.tokens.total() > 0 && (!a.group || a.groups == (a.width + a.group - 1) / a.group));
    }
    ++g_launched;
    return 0;
}
}  // namespace

namespace rc {
Error device_open(const Config&, DeviceInfo*) { return {}; }
Error device_launch(const LaunchPlan&, void*) { return Error{RC_ERR_DEVICE, "no device in this test"}; }
Error device_launch_batch(const BatchPlan&, void*) { return Error{RC_ERR_DEVICE, "no device in this test"}; }
size_t batch_table_bytes(const BatchPlan&) { return 0; }
Error device_launch_batch_static(const BatchPlan&, void*) { return Error{RC_ERR_DEVICE, "no device in this test"}; }
Error device_finish() { return {}; }
void device_reset() {}
Error device_event_create(void**) { return Error{RC_ERR_DEVICE, "no device in this test"}; }
void device_event_destroy(void*) {}
Error device_event_record(void*, void*) { return Error{RC_ERR_DEVICE, "no device in this test"}; }
Error device_stream_wait(void*, void*) { return Error{RC_ERR_DEVICE, "no device in this test"}; }
Error device_timer_start(void*, int*) { return Error{RC_ERR_DEVICE, "no device in this test"}; }
Error device_timer_stop(int, void*) { return Error{RC_ERR_DEVICE, "no device in this test"}; }
Error device_timer_read(int, bool* done, float*) {
    *done = false;
    return Error{RC_ERR_DEVICE, "no device in this test"};
}
Error device_stream_capturing(void*, bool* c) {
    *c = false;
    return Error{RC_ERR_DEVICE, "no device in this test"};
}
Error device_run(const std::function<int()>& launch) {
    const int e = launch();
    return e ? Error{RC_ERR_DEVICE, "launch"} : Error{};
}

int launch_rms_norm_F32(const NormArgs& a, int, void*) { return norm_ok(a, false); }
int launch_rms_norm_F16(const NormArgs& a, int, void*) { return norm_ok(a, false); }
int launch_rms_norm_BF16(const NormArgs& a, int, void*) { return norm_ok(a, false); }
int launch_rms_norm_grad_F32(const NormArgs& a, int, void*) { return norm_ok(a, true); }
int launch_rms_norm_grad_F16(const NormArgs& a, int, void*) { return norm_ok(a, true); }
int launch_rms_norm_grad_BF16(const NormArgs& a, int, void*) { return norm_ok(a, true); }

int launch_moe(const MoeArgs& a, int, int, void*) {
    check_spans(a.entries);
    const int n = a.entries.total();
    CHECK(n > 0 && n <= RC_MAX_MOE_ENTRIES && n % a.top_k == 0 && a.per_rank * R == a.num_experts);
    CHECK(a.hidden_row % 64 == 0 && a.hidden_row >= a.inner && a.product_row % 16 == 0 && a.product_row >= a.width);
    const auto at = reinterpret_cast<uintptr_t>(a.hidden);
    CHECK(at % 16 == 0 && a.hidden_plane == (int64_t)n * a.hidden_row * 2);
    CHECK(reinterpret_cast<uintptr_t>(a.products) == at + (uintptr_t)n * a.hidden_row * 4);
    CHECK(reinterpret_cast<uintptr_t>(a.lists) == reinterpret_cast<uintptr_t>(a.products) + (uintptr_t)n * a.product_row * 4);
    ++g_launched;
    return 0;
}

thread_local int64_t t_partials = 0;
int launch_grad_norm(const GradNormArgs& a, void*) {
    CHECK(a.n > 0 && a.n <= kNormList && a.chunks > 0);
    int64_t chunks = 0;
    for (int i = 0; i < a.n; ++i) {
        CHECK(a.first[i] == chunks && a.count[i] > 0 && (a.grad[i] & 0xffffffffffffffull));
        CHECK((a.grad[i] >> 56) == RC_F32 || (a.grad[i] >> 56) == RC_F16 || (a.grad[i] >> 56) == RC_BF16);
        chunks += (a.count[i] + kNormChunk - 1) / kNormChunk;
    }
    CHECK(chunks == a.chunks);
    t_partials += chunks;
    return 0;
}
int launch_grad_norm_join(const GradNormJoin& a, void*) {
    for (int r = 0; r < kMaxRanks; ++r) CHECK(a.first[r] <= a.first[r + 1]);
    CHECK(a.first[R] == t_partials && a.nranks == R);
    t_partials = 0;
    ++g_launched;
    return 0;
}
thread_local int64_t t_chunks = 0;
int launch_adamw_begin(const AdamwBegin& a, void*) {
    CHECK(a.nranks == R && a.table && a.steps && a.steps_out);
    t_chunks = 0;
    ++g_launched;
    return 0;
}
int launch_adamw(const AdamwArgs& a, int bits, void*) {
    CHECK(a.chunks > 0 && a.first_chunk >= t_chunks && (bits == 8 || bits == 32));
    const auto* base = reinterpret_cast<const uint8_t*>(a.table);
    const auto* entries = reinterpret_cast<const AdamwEntry*>(base + a.entries_at);
    const auto* out = reinterpret_cast<const AdamwEntry*>(reinterpret_cast<const uint8_t*>(a.out) + a.entries_at);
    const auto* map = reinterpret_cast<const int32_t*>(base + a.chunks_at);
    CHECK(a.chunk % RC_ADAMW_BLOCK == 0 && a.chunk >= kAdamwLeast && a.chunk <= kAdamwMost);
    for (int64_t c = a.first_chunk; c < a.first_chunk + a.chunks; ++c) {
        const int32_t t = map[c];
        CHECK(t >= a.first && t < a.first + kAdamwList && t < a.table->first[kMaxRanks]);
        const int64_t from = (c - entries[t].first_chunk) * a.chunk;
        CHECK(from >= 0 && from < entries[t].count && entries[t].rank >= 0 && entries[t].rank < R && out[t].count == entries[t].count);
    }
    t_chunks = a.first_chunk + a.chunks;
    return 0;
}

// of the row exchanges, which this test does not call
int launch_route_F32(const RouteArgs&, void*) { return 1; }
int launch_route_F16(const RouteArgs&, void*) { return 1; }
int launch_route_BF16(const RouteArgs&, void*) { return 1; }
int launch_route_grad_F32(const RouteArgs&, void*) { return 1; }
int launch_route_grad_F16(const RouteArgs&, void*) { return 1; }
int launch_route_grad_BF16(const RouteArgs&, void*) { return 1; }
int launch_plan(PlanArgs, void*, void*) { return 1; }
int launch_dispatch(const ExchangeArgs&, int, void*) { return 1; }
int launch_combine(const ExchangeArgs&, int, void*) { return 1; }
int launch_combine_grad(const ExchangeArgs&, int, void*) { return 1; }
int launch_embedding(const EmbeddingArgs&, int, void*) { return 1; }
int launch_embedding_grad(EmbeddingGradArgs, SortPass, int, int, void*, void*) { return 1; }
int64_t plan_workspace_bytes(const RankSpans&, int) { return 0; }
int64_t embedding_grad_workspace_bytes(const RankSpans&, int64_t, int64_t) { return 0; }
}  // namespace rc

namespace {

using Rng = std::mt19937_64;
int64_t pick(Rng& g, int64_t lo, int64_t hi) { return lo + (int64_t)(g() % (uint64_t)(hi - lo + 1)); }

// Addresses of buffers that do not overlap; never dereferenced.
struct Space {
    uintptr_t at = uintptr_t(1) << 40;
    void* take(int64_t bytes) {
        void* p = reinterpret_cast<void*>(at);
        at += ((uintptr_t)bytes + 255) / 256 * 256 + 256;
        return p;
    }
};

void check(int code, bool valid) {
    const char* err = rc_last_error();
    CHECK(code == RC_OK || code == RC_ERR_INVALID_ARGUMENT);
    CHECK((code == RC_OK) == (err[0] == '\0'));
    CHECK((code == RC_OK) == valid);
}

void norms(Rng& g, bool valid) {
    Space sp;
    const int types[] = {RC_F32, RC_F16, RC_BF16};
    int64_t tokens[R];
    for (int64_t& t : tokens) t = pick(g, 1, g() % 4 ? 50 : 100000000);
    rc_norm_desc d{};
    d.struct_size = sizeof d;
    d.dtype = types[g() % 3];
    d.weight_dtype = g() % 2 ? (int)RC_F32 : d.dtype;
    d.quantize = (int32_t)(g() % 2);
    d.group = g() % 2 ? 0 : 32 << (g() % 4);
    d.eps = 1e-6f;
    d.width = pick(g, 1, RC_MAX_NORM_WIDTH);
    d.tokens = tokens;
    const bool with = g() % 2;
    void* b[6][R];
    for (auto& list : b)
        for (int r = 0; r < R; ++r) list[r] = sp.take(tokens[r] * (d.width + 512) * 4);
    if (!valid) {
        switch (g() % 4) {
            case 0: d.width = g() % 2 ? 0 : RC_MAX_NORM_WIDTH + 1; break;
            case 1: tokens[g() % R] = g() % 2 ? -1 : INT64_MAX; break;
            case 2: b[3][g() % R] = nullptr; break;
            default: b[3][0] = b[2][1]; break;
        }
    }
    check(rc_rms_norm(&d, b[0], with ? b[1] : nullptr, b[2], b[3], reinterpret_cast<float* const*>(b[4]), with ? b[5] : nullptr, nullptr), valid);
    if (!valid) return;
    int64_t size = 0;
    check(rc_rms_norm_grad_workspace(&d, &size), true);
    void* ws = sp.take(size);
    check(rc_rms_norm_grad(&d, b[0], b[1], b[2], with ? b[3] : nullptr, b[4], b[5], ws, size, nullptr), true);
    check(rc_rms_norm_grad(&d, b[0], b[1], b[2], nullptr, b[4], b[5], ws, size - 1, nullptr), false);
}

void layers(Rng& g, bool valid) {
    Space sp;
    rc_moe_desc d{};
    const int kinds[][3] = {{RC_F32, RC_F32, RC_F32}, {RC_F16, RC_F16, RC_F16}, {RC_BF16, RC_BF16, RC_BF16}, {RC_BF16, RC_E4M3, RC_BF16}, {RC_E4M3, RC_E4M3, RC_F16}};
    const int* k = kinds[g() % 5];
    d.struct_size = sizeof d;
    d.dtype = k[0];
    d.weight_dtype = k[1];
    d.out_dtype = k[2];
    d.num_experts = R * (int32_t)pick(g, 1, RC_MAX_EXPERTS / R);
    d.top_k = (int32_t)pick(g, 1, RC_MAX_TOP_K);
    d.width = pick(g, 1, g() % 2 ? 100 : RC_MAX_MOE_WIDTH);
    d.inner = pick(g, 1, g() % 2 ? 100 : RC_MAX_MOE_WIDTH);
    int64_t tokens[R];
    for (int64_t& t : tokens) t = pick(g, 1, RC_MAX_MOE_ENTRIES / R / d.top_k);
    d.tokens = tokens;
    void* b[9][R];
    for (int r = 0; r < R; ++r) {
        for (int i : {0, 1, 2, 3, 8}) b[i][r] = sp.take(tokens[r] * (d.width + d.top_k) * 4);
        for (int i : {4, 5, 6, 7}) b[i][r] = sp.take((int64_t)d.num_experts / R * 2 * d.inner * d.width * 4 + d.num_experts * (2 * d.inner + d.width) * 4);
    }
    if (!valid) {
        switch (g() % 4) {
            case 0: d.num_experts += 1; break;
            case 1: tokens[g() % R] = g() % 2 ? RC_MAX_MOE_ENTRIES : INT64_MAX; if (d.top_k == 1) tokens[0] = tokens[1] = RC_MAX_MOE_ENTRIES; break;
            case 2: b[4][g() % R] = nullptr; break;
            default: b[8][0] = b[6][2]; break;
        }
    }
    int64_t size = 0;
    const int code = rc_moe_layer_workspace(&d, &size);
    if (valid) check(code, true);
    void* ws = sp.take(std::max<int64_t>(size, 1 << 20));
    auto f = [&](int i) { return reinterpret_cast<const float* const*>(b[i]); };
    const bool x8 = d.dtype == RC_E4M3, w8 = d.weight_dtype == RC_E4M3;
    auto call = [&](int64_t bytes) {
        return rc_moe_layer(&d, b[0], x8 ? f(1) : nullptr, reinterpret_cast<const int32_t* const*>(b[2]), f(3), b[4], w8 ? f(5) : nullptr, b[6],
                            w8 ? f(7) : nullptr, b[8], ws, bytes, nullptr);
    };
    check(call(std::max<int64_t>(size, 1 << 20)), valid);
    if (valid) check(call(size - 1), false);
}

void steps(Rng& g, bool valid) {
    Space sp;
    const int types[] = {RC_F32, RC_F16, RC_BF16};
    rc_adamw_table_desc t{};
    t.struct_size = sizeof t;
    t.state_bits = g() % 2 ? 8 : 32;
    int n[R];
    std::vector<rc_adamw_param> params[2][R];
    std::vector<rc_grad> grads[R];
    for (int r = 0; r < R; ++r) {
        n[r] = (int)pick(g, 0, g() % 3 ? 5 : 700);
        for (int i = 0; i < n[r]; ++i) {
            rc_adamw_param p{};
            p.count = pick(g, 0, g() % 8 ? 3000 : 3000000);
            p.dtype = types[g() % 3];
            for (auto& list : params) {
                p.param = sp.take(p.count * 4);
                p.master = static_cast<float*>(sp.take(p.count * 4));
                p.m = sp.take(p.count * 4);
                p.v = sp.take(p.count * 4);
                p.m_scale = static_cast<float*>(sp.take(p.count / 16 + 4));
                p.v_scale = static_cast<float*>(sp.take(p.count / 16 + 4));
                list[r].push_back(p);
            }
            rc_grad q{};
            if (p.count && g() % 4) q = {sp.take(p.count * 4), p.count, g() % 2 ? (int)RC_F32 : p.dtype, 0};
            grads[r].push_back(q);
        }
    }
    const rc_adamw_param* lists[2][R];
    const rc_grad* glists[R];
    for (int r = 0; r < R; ++r) {
        for (int k = 0; k < 2; ++k) lists[k][r] = params[k][r].data();
        glists[r] = grads[r].data();
    }
    std::vector<uint64_t> tables[2];
    for (int k = 0; k < 2; ++k) {
        int64_t size = 0;
        check(rc_adamw_table(&t, n, lists[k], nullptr, &size), true);
        tables[k].resize((size_t)size / 8 + 3);
        uint64_t* at = tables[k].data() + (reinterpret_cast<uintptr_t>(tables[k].data()) % 16 ? 1 : 0);
        check(rc_adamw_table(&t, n, lists[k], at, &size), true);
        size -= 1;
        check(rc_adamw_table(&t, n, lists[k], at, &size), false);
    }
    auto table = [&](int k) { return tables[k].data() + (reinterpret_cast<uintptr_t>(tables[k].data()) % 16 ? 1 : 0); };
    rc_adamw_desc d{};
    d.struct_size = sizeof d;
    d.lr = 1e-3;
    d.beta1 = 0.9;
    d.beta2 = 0.999;
    d.eps = 1e-8;
    d.grad_scale = 1;
    int32_t* counted = static_cast<int32_t*>(sp.take(64));
    d.steps = d.steps_out = counted;
    rc_grad_norm_desc gd{};
    gd.struct_size = sizeof gd;
    gd.over_all = (int32_t)(g() % 2);
    int64_t size = 0;
    check(rc_grad_norm_workspace(&gd, n, glists, &size), true);
    float* norm = static_cast<float*>(sp.take(64));
    check(rc_grad_norm(&gd, n, glists, norm, sp.take(size), size, nullptr), true);
    if (g() % 2) d.norms = norm, d.max_norm = 1;
    int spoiled = -1;
    for (int r = 0; r < R && !valid; ++r)
        if (n[r]) spoiled = r;
    if (spoiled >= 0) {
        const auto i = g() % grads[spoiled].size();
        switch (g() % 3) {
            case 0: grads[spoiled][i] = {sp.take(64), params[0][spoiled][i].count + 1, RC_F32, 0}; break;
            case 1: grads[spoiled][i] = {nullptr, 5, RC_F32, 0}; break;
            default: d.beta2 = 1.0; break;
        }
    }
    const int out = (int)(g() % 2);
    check(rc_adamw_step(&d, table(0), table(0), table(out), table(out), glists, nullptr), spoiled < 0);
}

void calls(int seed, int iters) {
    Rng g(seed);
    for (int i = 0; i < iters; ++i) {
        const bool valid = g() % 3 != 0;
        switch (g() % 3) {
            case 0: norms(g, valid); break;
            case 1: layers(g, valid); break;
            default: steps(g, valid); break;
        }
    }
}

}  // namespace

int main() {
    CHECK(rc_register(R, nullptr) == RC_OK);
    std::vector<std::thread> threads;
    for (int k = 0; k < 4; ++k) threads.emplace_back(calls, k + 1, 60);
    for (auto& t : threads) t.join();
    CHECK(g_launched > 80);
    CHECK(rc_reset() == RC_OK);
    std::printf("%d launches, %d bad results\n", g_launched.load(), g_bad.load());
    return g_bad != 0;
}
