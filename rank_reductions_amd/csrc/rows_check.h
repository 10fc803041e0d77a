// Argument checks shared by the entry points of the row exchanges and of the
// block operators.  Host-only C++.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdio>
#include <string>
#include <vector>

#include "rows.h"

namespace rc {

constexpr int64_t kMaxItems = 0x7fffffff;              // counts fit 32 bits
constexpr int64_t kMaxWidth = int64_t(1) << 22;        // elements of a row
constexpr int64_t kMaxCapacity = 0x7fffffff;

inline std::string fmt(const char* f, long long a = 0, long long b = 0, long long c = 0) {
    char buf[256];
    std::snprintf(buf, sizeof buf, f, a, b, c);
    return buf;
}

inline Error bad(const char* what, const std::string& msg) {
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
inline Error spans_of(const char* what, int R, const int64_t* counts, int64_t each, RankSpans* out) {
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

}  // namespace rc
