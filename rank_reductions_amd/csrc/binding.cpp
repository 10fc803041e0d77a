// Python module _rows: argument marshalling of the row exchanges (the block
// operators' is in binding_blocks.cpp).
//
// The calls take R tensors per argument, and a decoding step makes several of
// them on a few tokens, where checking and packing some fifty tensors in
// Python costs more than the kernels take (20 to 60 us against 5 to 15).  Here
// each tensor costs nanoseconds.  rows.py holds the public functions; this
// module checks every tensor (type, shape, device, density), allocates what
// the caller did not give, fills the C ABI's descriptors and calls
// librankred.so on the current stream of the tensors' device.
#include "binding_blocks.h"

using namespace rows_binding;

namespace {

// ---------------------------------------------------------------- routing

// route(logits, top_k, score, bias, groups, top_groups, group_by, renormalize, scale, out)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"route", 10});
        const char* what = "route";
        const Session s;
        Tensors l, w, e;
        l.take(a[0], s.ranks, what);
        l.dims(2, what, "[tokens, experts]");
        const at::Device dev = l.t[0]->device();
        int64_t tokens[RC_MAX_RANKS] = {};
        for (int r = 0; r < s.ranks; ++r) tokens[r] = l.t[r]->size(0);
        const int64_t E = l.t[0]->size(1), K = to_int32(a[1], what);
        rc_route_desc d{};
        d.struct_size = sizeof d;
        d.session = s.id;
        d.dtype = row_type(*l.t[0], what);
        l.expect(l.t[0]->scalar_type(), dev, tokens, E, what);
        if (E > RC_MAX_EXPERTS || K < 1 || K > RC_MAX_TOP_K)
            raise(RC_ERR_INVALID_ARGUMENT, what, "%lld experts, top_k %lld", (long long)E, (long long)K);
        d.num_experts = (int32_t)E;
        d.top_k = (int32_t)K;
        d.score = to_int32(a[2], what);
        Tensors b;
        if (a[3] != Py_None) {
            if (!THPVariable_Check(a[3])) raise(RC_ERR_INVALID_ARGUMENT, what, "bias is not a tensor");
            b.take_one(a[3]);
            b.expect(ScalarType::Float, dev, &E, -1, "route bias");
            d.bias = static_cast<const float*>(b.p[0]);
        }
        d.num_groups = to_int32(a[4], what);
        d.top_groups = to_int32(a[5], what);
        d.group_by = to_int32(a[6], what);
        d.renormalize = to_bool(a[7]);
        d.scale = to_float(a[8]);
        PyObject *wo, *eo;
        if (pair_of(a[9], what, &wo, &eo)) {
            w.take(wo, s.ranks, "route weights");
            e.take(eo, s.ranks, "route experts");
        } else {
            w.make(s.ranks, tokens, K, ScalarType::Float, dev, what);
            e.make(s.ranks, tokens, K, ScalarType::Int, dev, what);
        }
        w.expect(ScalarType::Float, dev, tokens, K, "route weights");
        e.expect(ScalarType::Int, dev, tokens, K, "route experts");
        void* stream = stream_on(s, dev, what);
        call([&] { return rc_route(&d, tokens, l.p, reinterpret_cast<float* const*>(w.p), reinterpret_cast<int32_t* const*>(e.p), stream); });
        PyObject* first = w.give();
        return pack(first, e.give());
    });
}

// route_grad(logits, experts, d_weights, score, renormalize, scale, out)
PyObject* route_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"route_grad", 7});
        const char* what = "route_grad";
        const Session s;
        Tensors l, e, w, o;
        l.take(a[0], s.ranks, what);
        l.dims(2, what, "[tokens, experts]");
        const at::Device dev = l.t[0]->device();
        int64_t tokens[RC_MAX_RANKS] = {};
        for (int r = 0; r < s.ranks; ++r) tokens[r] = l.t[r]->size(0);
        const int64_t E = l.t[0]->size(1);
        rc_route_desc d{};
        d.struct_size = sizeof d;
        d.session = s.id;
        d.dtype = row_type(*l.t[0], what);
        const ScalarType type = l.t[0]->scalar_type();
        l.expect(type, dev, tokens, E, what);
        e.take(a[1], s.ranks, "route_grad experts");
        e.dims(2, "route_grad experts", "[tokens, top_k]");
        const int64_t K = e.t[0]->size(1);
        e.expect(ScalarType::Int, dev, tokens, K, "route_grad experts");
        w.take(a[2], s.ranks, "route_grad d_weights");
        w.expect(ScalarType::Float, dev, tokens, K, "route_grad d_weights");
        if (E > RC_MAX_EXPERTS || K > RC_MAX_TOP_K)
            raise(RC_ERR_INVALID_ARGUMENT, what, "%lld experts, top_k %lld", (long long)E, (long long)K);
        d.num_experts = (int32_t)E;
        d.top_k = (int32_t)K;
        d.score = to_int32(a[3], what);
        d.num_groups = d.top_groups = 1;
        d.renormalize = to_bool(a[4]);
        d.scale = to_float(a[5]);
        if (a[6] != Py_None) {
            o.take(a[6], s.ranks, "route_grad output");
        } else {
            o.make(s.ranks, tokens, E, type, dev, what);
        }
        o.expect(type, dev, tokens, E, "route_grad output");
        void* stream = stream_on(s, dev, what);
        call([&] { return rc_route_grad(&d, tokens, l.p, reinterpret_cast<const int32_t* const*>(e.p),
                            reinterpret_cast<const float* const*>(w.p), o.p, stream); });
        return o.give();
    });
}

// ---------------------------------------------------------------- exchange

// What a plan's users share: its experts, slots and capacities.
struct Plan {
    Tensors experts, slots;
    int64_t tokens[RC_MAX_RANKS] = {}, capacity[RC_MAX_RANKS] = {}, K = 0;
    rc_exchange_desc d{};

    void capacities(PyObject* seq, int ranks, const char* what) {
        if (!PyList_Check(seq) && !PyTuple_Check(seq)) raise(RC_ERR_INVALID_ARGUMENT, what, "capacity is not a list");
        const Py_ssize_t size = PySequence_Fast_GET_SIZE(seq);
        if (size != ranks) raise(RC_ERR_INVALID_ARGUMENT, what, "%lld capacities for %d ranks", (long long)size, ranks);
        for (int r = 0; r < ranks; ++r) capacity[r] = to_int(PySequence_Fast_GET_ITEM(seq, r));
        for (int r = 0; r < ranks; ++r)
            if (capacity[r] < 0) raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d: negative capacity", r);
    }
    void choices(PyObject* seq, int ranks, const char* what) {
        experts.take(seq, ranks, what);
        experts.dims(2, what, "[tokens, top_k]");
        for (int r = 0; r < ranks; ++r) tokens[r] = experts.t[r]->size(0);
        K = experts.t[0]->size(1);
        experts.expect(ScalarType::Int, experts.t[0]->device(), tokens, K, what);
        if (K > RC_MAX_TOP_K) raise(RC_ERR_INVALID_ARGUMENT, what, "top_k %lld", (long long)K);
    }
    void describe(const Session& s, int32_t num_experts, int dtype, int64_t width) {
        d.struct_size = sizeof d;
        d.session = s.id;
        d.dtype = dtype;
        d.num_experts = num_experts;
        d.top_k = (int32_t)K;
        d.width = width;
        d.tokens = tokens;
        d.capacity = capacity;
        d.experts = reinterpret_cast<const int32_t* const*>(experts.p);
        d.slots = reinterpret_cast<int32_t* const*>(slots.p);
    }
    // From (experts, slots, capacity, num_experts), for rows on `dev`.
    void follow(PyObject* const* a, int ranks, const at::Device& dev, const char* what) {
        const std::string ew = std::string(what) + " experts", sw = std::string(what) + " slots";
        choices(a[0], ranks, ew.c_str());
        if (experts.t[0]->device() != dev)
            raise(RC_ERR_INVALID_ARGUMENT, what, "the plan on %s, rows on %s", experts.t[0]->device().str().c_str(), dev.str().c_str());
        slots.take(a[1], ranks, sw.c_str());
        slots.expect(ScalarType::Int, dev, tokens, K, sw.c_str());
        capacities(a[2], ranks, what);
    }
};

// dispatch_plan(experts, num_experts, capacity or None)
// -> (slots, offsets, counts, capacity)
PyObject* dispatch_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"dispatch_plan", 3});
        const char* what = "dispatch_plan";
        const Session s;
        const int R = s.ranks;
        Plan p;
        p.choices(a[0], R, what);
        const at::Device dev = p.experts.t[0]->device();
        const int32_t E = to_int32(a[1], what);
        if (E < 1 || E > RC_MAX_EXPERTS || E % R) raise(RC_ERR_INVALID_ARGUMENT, what, "%d experts over %d ranks", E, R);
        const int64_t per = E / R;
        int64_t entries = 0;
        for (int r = 0; r < R; ++r) entries += p.tokens[r] * p.K;
        if (a[2] == Py_None) {
            for (int r = 0; r < R; ++r) p.capacity[r] = entries;
        } else if (PyLong_Check(a[2])) {
            const int64_t c = to_int(a[2]);
            if (c < 0) raise(RC_ERR_INVALID_ARGUMENT, what, "negative capacity");
            for (int r = 0; r < R; ++r) p.capacity[r] = c;
        } else {
            p.capacities(a[2], R, what);
        }
        void* stream = stream_on(s, dev, what);
        // slots, offsets and counts of all ranks in one piece
        const Tensor all = at::empty({entries + R * (2 * per + 1)}, options(ScalarType::Int, dev));
        p.slots.make(R);
        Tensors offsets, counts;
        offsets.make(R);
        counts.make(R);
        int64_t at_ = 0, one[RC_MAX_RANKS];
        for (int r = 0; r < R; ++r) {
            p.slots.made[r] = part_of(all, at_, {p.tokens[r], p.K});
            at_ += p.tokens[r] * p.K;
        }
        for (int r = 0; r < R; ++r, at_ += per + 1) offsets.made[r] = part_of(all, at_, {per + 1});
        for (int r = 0; r < R; ++r, at_ += per) counts.made[r] = part_of(all, at_, {per});
        p.slots.expect(ScalarType::Int, dev, p.tokens, p.K, what);
        for (int r = 0; r < R; ++r) one[r] = per + 1;
        offsets.expect(ScalarType::Int, dev, one, -1, what);
        for (int r = 0; r < R; ++r) one[r] = per;
        counts.expect(ScalarType::Int, dev, one, -1, what);
        p.describe(s, E, RC_F32, 1);
        int64_t size = 0;
        call([&] { return rc_dispatch_plan_workspace(&p.d, &size); });
        Tensor work;
        if (size) work = at::empty({size}, options(ScalarType::Byte, dev));
        call([&] { return rc_dispatch_plan(&p.d, reinterpret_cast<int32_t* const*>(offsets.p), reinterpret_cast<int32_t* const*>(counts.p),
                               size ? work.data_ptr() : nullptr, size, stream); });
        PyObject* caps = PyList_New(R);
        if (!caps) throw Raised{};
        for (int r = 0; r < R; ++r) PyList_SET_ITEM(caps, r, PyLong_FromLongLong(p.capacity[r]));
        PyObject* out[4] = {p.slots.give(), offsets.give(), counts.give(), caps};
        PyObject* t = PyTuple_Pack(4, out[0], out[1], out[2], out[3]);
        for (PyObject* o : out) Py_DECREF(o);
        if (!t) throw Raised{};
        return t;
    });
}

// dispatch(xs, experts, slots, capacity, num_experts, out)
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"dispatch", 6});
        const char* what = "dispatch";
        const Session s;
        Tensors x, o;
        x.take(a[0], s.ranks, what);
        x.dims(2, what, "[tokens, width]");
        const at::Device dev = x.t[0]->device();
        const ScalarType type = x.t[0]->scalar_type();
        const int64_t D = x.t[0]->size(1);
        Plan p;
        p.follow(a + 1, s.ranks, dev, what);
        x.expect(type, dev, p.tokens, D, what);
        p.describe(s, to_int32(a[4], what), row_type(*x.t[0], what), D);
        if (a[5] != Py_None) {
            o.take(a[5], s.ranks, "dispatch output");
        } else {
            o.make(s.ranks, p.capacity, D, type, dev, what, true);
        }
        o.expect(type, dev, p.capacity, D, "dispatch output");
        void* stream = stream_on(s, dev, what);
        call([&] { return rc_dispatch(&p.d, x.p, o.p, stream); });
        return o.give();
    });
}

// combine(rows, experts, slots, capacity, num_experts, weights or None, out)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"combine", 7});
        const char* what = "combine";
        const Session s;
        Tensors x, w, o;
        x.take(a[0], s.ranks, what);
        x.dims(2, what, "[capacity, width]");
        const at::Device dev = x.t[0]->device();
        const ScalarType type = x.t[0]->scalar_type();
        const int64_t D = x.t[0]->size(1);
        Plan p;
        p.follow(a + 1, s.ranks, dev, what);
        x.expect(type, dev, p.capacity, D, what);
        p.describe(s, to_int32(a[4], what), row_type(*x.t[0], what), D);
        if (a[5] != Py_None) {
            w.take(a[5], s.ranks, "combine weights");
            w.expect(ScalarType::Float, dev, p.tokens, p.K, "combine weights");
        }
        if (a[6] != Py_None) {
            o.take(a[6], s.ranks, "combine output");
        } else {
            o.make(s.ranks, p.tokens, D, type, dev, what);
        }
        o.expect(type, dev, p.tokens, D, "combine output");
        void* stream = stream_on(s, dev, what);
        call([&] { return rc_combine(&p.d, x.p, w.n ? reinterpret_cast<const float* const*>(w.p) : nullptr, o.p, stream); });
        return o.give();
    });
}

// combine_grad(d_outs, rows, experts, slots, capacity, num_experts, weights, out)
PyObject* combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"combine_grad", 8});
        const char* what = "combine_grad";
        const Session s;
        Tensors dy, x, w, dx, dw;
        dy.take(a[0], s.ranks, what);
        dy.dims(2, what, "[tokens, width]");
        const at::Device dev = dy.t[0]->device();
        const ScalarType type = dy.t[0]->scalar_type();
        const int64_t D = dy.t[0]->size(1);
        Plan p;
        p.follow(a + 2, s.ranks, dev, what);
        dy.expect(type, dev, p.tokens, D, what);
        x.take(a[1], s.ranks, "combine_grad rows");
        x.expect(type, dev, p.capacity, D, "combine_grad rows");
        p.describe(s, to_int32(a[5], what), row_type(*dy.t[0], what), D);
        w.take(a[6], s.ranks, "combine_grad weights");
        w.expect(ScalarType::Float, dev, p.tokens, p.K, "combine_grad weights");
        PyObject *xo, *wo;
        if (pair_of(a[7], what, &xo, &wo)) {
            dx.take(xo, s.ranks, "combine_grad d_rows");
            dw.take(wo, s.ranks, "combine_grad d_weights");
        } else {
            dx.make(s.ranks, p.capacity, D, type, dev, what, true);
            dw.make(s.ranks, p.tokens, p.K, ScalarType::Float, dev, what);
        }
        dx.expect(type, dev, p.capacity, D, "combine_grad d_rows");
        dw.expect(ScalarType::Float, dev, p.tokens, p.K, "combine_grad d_weights");
        void* stream = stream_on(s, dev, what);
        call([&] { return rc_combine_grad(&p.d, dy.p, x.p, reinterpret_cast<const float* const*>(w.p), dx.p,
                              reinterpret_cast<float* const*>(dw.p), stream); });
        PyObject* first = dx.give();
        return pack(first, dw.give());
    });
}

// ---------------------------------------------------------------- embedding

void shards(int64_t vocab, int ranks, int64_t* rows) {
    const int64_t s = (vocab + ranks - 1) / ranks;
    for (int64_t c = 0; c < ranks; ++c) rows[c] = std::max<int64_t>(0, std::min((c + 1) * s, vocab) - c * s);
}

struct Ids {
    Tensors ids;
    int64_t tokens[RC_MAX_RANKS] = {};
    rc_embedding_desc d{};
    at::Device dev{at::kCPU};

    Ids(PyObject* seq, const Session& s, const char* what) {
        const int ranks = s.ranks;
        ids.take(seq, ranks, what);
        ids.dims(1, what, "[tokens]");
        dev = ids.t[0]->device();
        const ScalarType type = ids.t[0]->scalar_type();
        if (type != ScalarType::Int && type != ScalarType::Long) {
            PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %s; int32 and int64 are supported", what, type_name(type));
            throw Raised{};
        }
        for (int r = 0; r < ranks; ++r) tokens[r] = ids.t[r]->size(0);
        ids.expect(type, dev, tokens, -1, what);
        d.struct_size = sizeof d;
        d.session = s.id;
        d.id_dtype = type == ScalarType::Long ? (int)RC_I64 : (int)RC_I32;
        d.tokens = tokens;
        d.ids = ids.p;
    }
};

// embedding(ids, tables, scale, out)
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"embedding", 4});
        const char* what = "embedding";
        const Session s;
        Ids i(a[0], s, what);
        Tensors t, o;
        t.take(a[1], s.ranks, "embedding tables");
        t.dims(2, "embedding tables", "[rows, width]");
        const ScalarType type = t.t[0]->scalar_type();
        int64_t rows[RC_MAX_RANKS];
        const int64_t D = t.t[0]->size(1);
        for (int r = 0; r < s.ranks; ++r) i.d.vocab += t.t[r]->size(0);
        shards(i.d.vocab, s.ranks, rows);
        t.expect(type, i.dev, rows, D, "embedding tables");
        i.d.dtype = i.d.grad_dtype = row_type(*t.t[0], what);
        i.d.scale = to_float(a[2]);
        i.d.width = D;
        if (a[3] != Py_None) {
            o.take(a[3], s.ranks, "embedding output");
        } else {
            o.make(s.ranks, i.tokens, D, type, i.dev, what);
        }
        o.expect(type, i.dev, i.tokens, D, "embedding output");
        void* stream = stream_on(s, i.dev, what);
        call([&] { return rc_embedding(&i.d, t.p, o.p, stream); });
        return o.give();
    });
}

// embedding_grad(ids, d_outs, vocab, scale, dtype or None, out, accumulate)
PyObject* embedding_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"embedding_grad", 7});
        const char* what = "embedding_grad";
        const Session s;
        Ids i(a[0], s, what);
        Tensors g, o;
        g.take(a[1], s.ranks, what);
        g.dims(2, what, "[tokens, width]");
        const int64_t D = g.t[0]->size(1);
        const ScalarType type = g.t[0]->scalar_type();
        g.expect(type, i.dev, i.tokens, D, what);
        i.d.dtype = row_type(*g.t[0], what);
        i.d.vocab = to_int(a[2]);
        if (i.d.vocab < 1 || i.d.vocab > INT32_MAX) raise(RC_ERR_INVALID_ARGUMENT, what, "a vocabulary of %lld", (long long)i.d.vocab);
        i.d.scale = to_float(a[3]);
        i.d.width = D;
        i.d.accumulate = to_bool(a[6]);
        int64_t rows[RC_MAX_RANKS];
        shards(i.d.vocab, s.ranks, rows);
        ScalarType out_type = type;
        if (a[4] != Py_None) {
            if (!THPDtype_Check(a[4])) raise(RC_ERR_INVALID_ARGUMENT, what, "dtype is not a torch.dtype");
            out_type = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
        }
        if (a[5] != Py_None) {
            o.take(a[5], s.ranks, "embedding_grad output");
            if (a[4] == Py_None) out_type = o.t[0]->scalar_type();
        } else {
            if (i.d.accumulate) raise(RC_ERR_INVALID_ARGUMENT, what, "accumulate needs the tensors to add to");
            o.make(s.ranks, rows, D, out_type, i.dev, what);
        }
        o.expect(out_type, i.dev, rows, D, "embedding_grad output");
        i.d.grad_dtype = row_type(*o.t[0], what);
        void* stream = stream_on(s, i.dev, what);
        int64_t size = 0;
        call([&] { return rc_embedding_grad_workspace(&i.d, &size); });
        Tensor work;
        if (size) work = at::empty({size}, options(ScalarType::Byte, i.dev));
        call([&] { return rc_embedding_grad(&i.d, g.p, o.p, size ? work.data_ptr() : nullptr, size, stream); });
        return o.give();
    });
}

// device() -> the session's GPU, -1 for none
PyObject* device(PyObject*, PyObject* const*, Py_ssize_t) {
    return guarded([&] { return PyLong_FromLong(Session().device); });
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

#define RC_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    RC_METHOD(route), RC_METHOD(route_grad), RC_METHOD(dispatch_plan), RC_METHOD(dispatch), RC_METHOD(combine),
    RC_METHOD(combine_grad), RC_METHOD(embedding), RC_METHOD(embedding_grad), RC_METHOD(device),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rows(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddFunctions(m, block_methods) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
