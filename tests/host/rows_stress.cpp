// Host-only stress of the row exchanges' entry points (no GPU): several threads
// make random calls, most of them valid, some with one thing wrong, some with
// random fields.  The kernels are stubs that check what a launch may rely on.
// Built with sanitizers by the tests; links rows.cpp, session.cpp,
// validate.cpp and plan.cpp.
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <random>
#include <thread>
#include <vector>

#include "rc.h"
#include "rows.h"

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
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

void check_spans(const rc::RankSpans& s) {
    CHECK(s.nranks == R && s.first[0] == 0);
    for (int r = 0; r < rc::kMaxRanks; ++r) CHECK(s.first[r] <= s.first[r + 1]);
    CHECK(s.first[R] == s.total());
}
int route_ok(const rc::RouteArgs& a, size_t es) {
    check_spans(a.tokens);
    CHECK(a.tokens.total() > 0 && a.num_experts >= 1 && a.num_experts <= RC_MAX_EXPERTS);
    CHECK(a.top_k >= 1 && a.top_k <= RC_MAX_TOP_K && a.top_k <= a.num_experts);
    CHECK(a.groups >= 1 && a.groups <= RC_MAX_EXPERT_GROUPS && a.group_size * a.groups == a.num_experts);
    for (int r = 0; r < R; ++r) {
        if (a.tokens.first[r] == a.tokens.first[r + 1]) continue;
        CHECK(a.logits[r] && aligned(a.logits[r], a.vec ? 4 * es : es));
        if (a.d_weights[r]) CHECK(a.d_logits[r] && aligned(a.d_logits[r], a.vec ? 4 * es : es));
        else CHECK(a.weights[r] && a.experts[r]);
    }
    if (a.vec) CHECK(a.num_experts % 4 == 0);
    ++g_launched;
    return 0;
}
int exchange_ok(const rc::ExchangeArgs& a) {
    check_spans(a.tokens);
    CHECK(a.tokens.total() > 0 && a.width >= 1 && a.per_rank * R == a.num_experts);
    for (int r = 0; r < R; ++r) CHECK(a.capacity[r] >= 0 && a.capacity[r] <= std::numeric_limits<int32_t>::max());
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

int launch_route_F32(const RouteArgs& a, void*) { return route_ok(a, 4); }
int launch_route_F16(const RouteArgs& a, void*) { return route_ok(a, 2); }
int launch_route_BF16(const RouteArgs& a, void*) { return route_ok(a, 2); }
int launch_route_grad_F32(const RouteArgs& a, void*) { return route_ok(a, 4); }
int launch_route_grad_F16(const RouteArgs& a, void*) { return route_ok(a, 2); }
int launch_route_grad_BF16(const RouteArgs& a, void*) { return route_ok(a, 2); }
int launch_plan(PlanArgs a, void*, void*) {
    check_spans(a.sort.spans);
    const RankSpans b = sort_blocks(a.sort.spans);
    for (int r = 0; r < R; ++r) {
        const int64_t n = (int64_t)a.sort.spans.first[r + 1] - a.sort.spans.first[r];
        CHECK((int64_t)(b.first[r + 1] - b.first[r]) * kSortBlock >= n);
        CHECK(a.offsets[r] && a.counts[r] && (n == 0 || (a.slots[r] && a.sort.ids[r])));
    }
    ++g_launched;
    return 0;
}
int launch_dispatch(const ExchangeArgs& a, int, void*) { return exchange_ok(a); }
int launch_combine(const ExchangeArgs& a, int, void*) { return exchange_ok(a); }
int launch_combine_grad(const ExchangeArgs& a, int, void*) { return exchange_ok(a); }
int launch_embedding(const EmbeddingArgs& a, int, void*) {
    check_spans(a.tokens);
    CHECK(a.shard * R >= a.vocab && (a.shard - 1) * R < a.vocab && a.width >= 1);
    ++g_launched;
    return 0;
}
int launch_embedding_grad(EmbeddingGradArgs a, SortPass sort, int, int, void*, void*) {
    check_spans(a.tokens);
    CHECK(sort.key_limit == a.vocab && a.shard * R >= a.vocab && sort.spans.total() == a.tokens.total());
    ++g_launched;
    return 0;
}
int64_t plan_workspace_bytes(const RankSpans& entries, int num_experts) {
    return ((int64_t)sort_blocks(entries).total() + 1) * num_experts * 4;
}
int64_t embedding_grad_workspace_bytes(const RankSpans& tokens, int64_t vocab, int64_t width) {
    return tokens.total() ? vocab + (tokens.total() + kPiece - 1) / kPiece * 2 * width * 4 : 0;
}
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

// One of them loses its buffer, or its alignment, or lands on the other's.
template <class P>
void spoil(Rng& g, P** a, P** b) {
    const int r = (int)(g() % R);
    switch (g() % 3) {
        case 0: a[r] = nullptr; break;
        case 1: a[r] = reinterpret_cast<P*>(reinterpret_cast<uintptr_t>(a[r]) + 1); break;
        default: a[r] = b[(r + 1) % R]; break;
    }
}

void check(int code, bool valid) {
    const char* err = rc_last_error();
    CHECK(code == RC_OK || code == RC_ERR_INVALID_ARGUMENT);
    CHECK((code == RC_OK) == (err[0] == '\0'));
    if (valid) CHECK(code == RC_OK);
    else CHECK(code != RC_OK);
}

void calls(int seed, int iters) {
    Rng g(seed);
    const int types[] = {RC_F32, RC_F16, RC_BF16};
    for (int i = 0; i < iters; ++i) {
        Space sp;
        const bool valid = g() % 3 != 0;
        const int dtype = types[g() % 3];
        const int64_t es = dtype == RC_F32 ? 4 : 2;
        int64_t tokens[R], capacity[R];
        for (int64_t& t : tokens) t = pick(g, 1, g() % 4 ? 50 : 100000000);
        void* b[6][R];
        if (g() % 3 == 0) {
            rc_route_desc d{};
            d.struct_size = sizeof d;
            d.dtype = dtype;
            d.num_groups = 1 << pick(g, 0, 6);
            d.num_experts = d.num_groups * (int32_t)pick(g, 1, RC_MAX_EXPERTS / d.num_groups);
            d.top_groups = (int32_t)pick(g, 1, d.num_groups);
            d.top_k = (int32_t)pick(g, 1, std::min(RC_MAX_TOP_K, d.top_groups * (d.num_experts / d.num_groups)));
            d.score = (int32_t)(g() % 2);
            d.group_by = (int32_t)(g() % 2);
            d.scale = 2.5f;
            if (g() % 2) d.bias = static_cast<const float*>(sp.take(d.num_experts * 4));
            for (int r = 0; r < R; ++r) {
                b[0][r] = sp.take(tokens[r] * d.num_experts * es);
                b[1][r] = sp.take(tokens[r] * d.top_k * 4);
                b[2][r] = sp.take(tokens[r] * d.top_k * 4);
                b[3][r] = sp.take(tokens[r] * d.num_experts * es);
            }
            if (!valid) {
                if (g() % 2) spoil(g, b[1], b[2]);
                else if (g() % 2) d.top_k = 0;
                else tokens[g() % R] = -1;
            }
            auto w = reinterpret_cast<float* const*>(b[1]);
            auto e = reinterpret_cast<int32_t* const*>(b[2]);
            // of the gradient, which only reads them, weights and experts may share
            if (valid || d.top_k == 0 || g() % 2) check(rc_route(&d, tokens, b[0], w, e, nullptr), valid);
            if (valid) check(rc_route_grad(&d, tokens, b[0], e, w, b[3], nullptr), true);
            continue;
        }
        if (g() % 2) {
            rc_exchange_desc d{};
            d.struct_size = sizeof d;
            d.dtype = dtype;
            d.num_experts = R * (int32_t)pick(g, 1, RC_MAX_EXPERTS / R);
            d.top_k = (int32_t)pick(g, 1, 4);
            d.width = pick(g, 1, 5000);
            for (int r = 0; r < R; ++r) {
                capacity[r] = pick(g, 1, 1000);
                b[0][r] = sp.take(tokens[r] * d.top_k * 4);
                b[1][r] = sp.take(tokens[r] * d.top_k * 4);
                b[2][r] = sp.take(tokens[r] * d.width * es);
                b[3][r] = sp.take(capacity[r] * d.width * es);
                b[4][r] = sp.take(d.num_experts * 4 + 4);
                b[5][r] = sp.take(std::max<int64_t>(d.num_experts, tokens[r] * d.top_k) * 4);
            }
            d.tokens = tokens;
            d.capacity = capacity;
            d.experts = reinterpret_cast<const int32_t* const*>(b[0]);
            d.slots = reinterpret_cast<int32_t* const*>(b[1]);
            if (!valid) {
                switch (g() % 4) {
                    case 0: spoil(g, b[1], b[0]); break;
                    case 1: d.num_experts += 1; break;
                    case 2: capacity[g() % R] = -1; break;
                    default: tokens[g() % R] = std::numeric_limits<int64_t>::max(); break;
                }
            }
            int64_t size = 0;
            const int code = rc_dispatch_plan_workspace(&d, &size);
            if (valid) check(code, true);
            if (code == RC_OK) {
                void* ws = sp.take(size);
                auto o = reinterpret_cast<int32_t* const*>(b[4]);
                auto c = reinterpret_cast<int32_t* const*>(b[5]);
                check(rc_dispatch_plan(&d, o, c, ws, size, nullptr), valid);
                if (valid && size) check(rc_dispatch_plan(&d, o, c, ws, size - 1, nullptr), false);
            }
            auto w = reinterpret_cast<float* const*>(b[5]);
            auto dw = reinterpret_cast<float* const*>(b[1]);  // where slots are read: refused
            if (valid) {
                check(rc_dispatch(&d, b[2], b[3], nullptr), true);
                check(rc_combine(&d, b[3], w, b[2], nullptr), true);
                check(rc_combine(&d, b[3], nullptr, b[2], nullptr), true);
                check(rc_combine_grad(&d, b[2], b[3], w, b[3], dw, nullptr), false);
            }
            continue;
        }
        rc_embedding_desc d{};
        d.struct_size = sizeof d;
        d.dtype = dtype;
        d.id_dtype = g() % 2 ? RC_I32 : RC_I64;
        d.grad_dtype = g() % 2 ? RC_F32 : dtype;
        d.accumulate = (int32_t)(g() % 2);
        d.vocab = pick(g, R, g() % 4 ? 1000 : 2147483646);
        d.width = pick(g, 1, 5000);
        d.scale = 1.0f;
        const int64_t shard = (d.vocab + R - 1) / R;
        for (int r = 0; r < R; ++r) {
            b[0][r] = sp.take(tokens[r] * 8);
            b[1][r] = sp.take(shard * d.width * 4);
            b[2][r] = sp.take(tokens[r] * d.width * es);
        }
        d.tokens = tokens;
        d.ids = b[0];
        if (!valid) {
            switch (g() % 4) {
                case 0: d.width = 0; break;
                case 1: d.vocab = 2147483647; break;
                case 2: d.scale = std::numeric_limits<float>::infinity(); break;
                default: d.id_dtype = RC_F32; break;
            }
        }
        check(rc_embedding(&d, b[1], b[2], nullptr), valid);
        int64_t size = 0;
        check(rc_embedding_grad_workspace(&d, &size), valid);
        if (valid) check(rc_embedding_grad(&d, b[2], b[1], sp.take(size), size, nullptr), true);
    }
}

// Random fields: every call returns a documented status.
void fuzz(int seed, int iters) {
    Rng g(seed);
    auto any32 = [&] { return g() % 3 ? (int32_t)pick(g, -1, 20) : (int32_t)g(); };
    auto any64 = [&] { return g() % 3 ? pick(g, -1, 100) : (int64_t)g(); };
    for (int i = 0; i < iters; ++i) {
        void* b[5][R];
        for (auto& list : b)
            for (void*& p : list) p = g() % 6 ? reinterpret_cast<void*>(g() & 0xfffffffffffull) : nullptr;
        int64_t tokens[R], capacity[R], size = 0;
        for (int r = 0; r < R; ++r) {
            tokens[r] = any64();
            capacity[r] = any64();
        }
        int code = RC_OK;
        if (g() % 3 == 0) {
            rc_route_desc d{};
            d.struct_size = g() % 8 ? sizeof d : any32();
            d.dtype = any32();
            d.num_experts = any32();
            d.top_k = any32();
            d.score = any32();
            d.num_groups = any32();
            d.top_groups = any32();
            d.group_by = any32();
            code = rc_route(&d, tokens, b[0], reinterpret_cast<float* const*>(b[1]), reinterpret_cast<int32_t* const*>(b[2]), nullptr);
        } else if (g() % 2) {
            rc_exchange_desc d{};
            d.struct_size = g() % 8 ? sizeof d : any32();
            d.dtype = any32();
            d.num_experts = any32();
            d.top_k = any32();
            d.width = any64();
            d.tokens = g() % 8 ? tokens : nullptr;
            d.capacity = g() % 8 ? capacity : nullptr;
            d.experts = g() % 8 ? reinterpret_cast<const int32_t* const*>(b[0]) : nullptr;
            d.slots = g() % 8 ? reinterpret_cast<int32_t* const*>(b[1]) : nullptr;
            code = g() % 2 ? rc_dispatch(&d, b[2], b[3], nullptr)
                           : rc_dispatch_plan(&d, reinterpret_cast<int32_t* const*>(b[2]), reinterpret_cast<int32_t* const*>(b[3]),
                                              b[4][0], any64(), nullptr);
        } else {
            rc_embedding_desc d{};
            d.struct_size = g() % 8 ? sizeof d : any32();
            d.dtype = any32();
            d.id_dtype = any32();
            d.grad_dtype = any32();
            d.vocab = any64();
            d.width = any64();
            d.tokens = g() % 8 ? tokens : nullptr;
            d.ids = g() % 8 ? b[0] : nullptr;
            code = g() % 2 ? rc_embedding(&d, b[1], b[2], nullptr) : rc_embedding_grad_workspace(&d, &size);
        }
        CHECK(code == RC_OK || code == RC_ERR_INVALID_ARGUMENT);
    }
}

}  // namespace

int main() {
    CHECK(rc_register(R, nullptr) == RC_OK);
    std::vector<std::thread> ts;
    for (int t = 0; t < 4; ++t) ts.emplace_back(calls, t, 1500);
    ts.emplace_back(fuzz, 9, 6000);
    for (auto& t : ts) t.join();
    CHECK(rc_finish() == RC_OK);
    std::printf("%d launches, %d bad results\n", g_launched.load(), g_bad.load());
    return g_bad != 0 || g_launched < 1000;
}
