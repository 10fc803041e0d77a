// Python module _rows: argument marshalling of the block operators (blocks.py
// holds the public functions).
#include "binding_blocks.h"

#include <c10/hip/HIPCachingAllocator.h>

#include <cstring>
#include <memory>

using namespace rows_binding;

namespace {

constexpr ScalarType kE4M3 = ScalarType::Float8_e4m3fn;

// Counts of R tensors' rows.
void rows_of(const Tensors& x, int64_t* rows) {
    for (int r = 0; r < x.n; ++r) rows[r] = x.t[r]->size(0);
}

// R lists as a tuple, or the only one.
PyObject* lists(std::initializer_list<Tensors*> all) {
    PyObject* out[4];
    int n = 0;
    for (Tensors* t : all)
        if (t) out[n++] = t->give();
    if (n == 1) return out[0];
    PyObject* tuple = PyTuple_New(n);
    for (int i = 0; i < n; ++i) {
        if (tuple) PyTuple_SET_ITEM(tuple, i, out[i]);
        else Py_DECREF(out[i]);
    }
    if (!tuple) throw Raised{};
    return tuple;
}

// ---------------------------------------------------------------- norm

// Rows, weights and what both norm calls are told alike.
struct Norm {
    Tensors x, w;
    int64_t tokens[RC_MAX_RANKS] = {}, width = 0, one[RC_MAX_RANKS];
    at::Device dev{at::kCPU};
    ScalarType type{}, weight_type{};
    rc_norm_desc d{};

    Norm(PyObject* rows, PyObject* weights, PyObject* eps, const Session& s, const char* what) {
        x.take(rows, s.ranks, what);
        x.dims(2, what, "[tokens, width]");
        dev = x.t[0]->device();
        type = x.t[0]->scalar_type();
        rows_of(x, tokens);
        width = x.t[0]->size(1);
        d.struct_size = sizeof d;
        d.session = s.id;
        d.dtype = row_type(*x.t[0], what);
        x.expect(type, dev, tokens, width, what);
        const std::string name = std::string(what) + " weights";
        w.take(weights, s.ranks, name.c_str());
        weight_type = w.t[0]->scalar_type();
        if (weight_type != type && weight_type != ScalarType::Float)
            raise(RC_ERR_DTYPE_MISMATCH, what, "weights of dtype %s, expected %s or Float", type_name(weight_type), type_name(type));
        d.weight_dtype = row_type(*w.t[0], what);
        for (int r = 0; r < s.ranks; ++r) one[r] = width;
        w.expect(weight_type, dev, one, -1, name.c_str());
        d.eps = to_float(eps);
        d.width = width;
        d.tokens = tokens;
    }
};

// rms_norm(xs, weights, eps, residuals or None, quantize, group, ys, scales, sums (each or None))
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"rms_norm", 9});
        const char* what = "rms_norm";
        const Session s;
        Norm m(a[0], a[1], a[2], s, what);
        Tensors res, y, scales, sums;
        const bool with = a[3] != Py_None;
        if (with) {
            res.take(a[3], s.ranks, "rms_norm residuals");
            res.expect(m.type, m.dev, m.tokens, m.width, "rms_norm residuals");
        }
        m.d.quantize = to_int32(a[4], what);
        m.d.group = to_int32(a[5], what);
        const ScalarType type = m.d.quantize ? kE4M3 : m.type;
        if (a[6] != Py_None) y.take(a[6], s.ranks, "rms_norm output");
        else y.make(s.ranks, m.tokens, m.width, type, m.dev, what);
        y.expect(type, m.dev, m.tokens, m.width, "rms_norm output");
        if (m.d.quantize) {
            const int64_t groups = m.d.group > 0 ? (m.width + m.d.group - 1) / m.d.group : 1;
            if (a[7] != Py_None) scales.take(a[7], s.ranks, "rms_norm scales");
            else scales.make(s.ranks, m.tokens, groups, ScalarType::Float, m.dev, what);
            scales.expect(ScalarType::Float, m.dev, m.tokens, groups, "rms_norm scales");
        }
        if (with) {
            if (a[8] != Py_None) sums.take(a[8], s.ranks, "rms_norm sums");
            else sums.make(s.ranks, m.tokens, m.width, m.type, m.dev, what);
            sums.expect(m.type, m.dev, m.tokens, m.width, "rms_norm sums");
        }
        void* stream = stream_on(s, m.dev, what);
        call([&] { return rc_rms_norm(&m.d, m.x.p, with ? res.p : nullptr, m.w.p, y.p,
                               m.d.quantize ? reinterpret_cast<float* const*>(scales.p) : nullptr, with ? sums.p : nullptr, stream); });
        return lists({&y, m.d.quantize ? &scales : nullptr, with ? &sums : nullptr});
    });
}

// rms_norm_grad(d_ys, sums, weights, eps, d_sums or None, out or None)
PyObject* rms_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"rms_norm_grad", 6});
        const char* what = "rms_norm_grad";
        const Session s;
        Norm m(a[1], a[2], a[3], s, what);
        Tensors dy, ds, dx, dw;
        dy.take(a[0], s.ranks, "rms_norm_grad d_ys");
        dy.expect(m.type, m.dev, m.tokens, m.width, "rms_norm_grad d_ys");
        const bool with = a[4] != Py_None;
        if (with) {
            ds.take(a[4], s.ranks, "rms_norm_grad d_sums");
            ds.expect(m.type, m.dev, m.tokens, m.width, "rms_norm_grad d_sums");
        }
        PyObject *xo, *wo;
        if (pair_of(a[5], what, &xo, &wo)) {
            dx.take(xo, s.ranks, "rms_norm_grad d_xs");
            dw.take(wo, s.ranks, "rms_norm_grad d_weights");
        } else {
            dx.make(s.ranks, m.tokens, m.width, m.type, m.dev, what);
            dw.make(s.ranks);
            for (int r = 0; r < s.ranks; ++r) dw.made[r] = at::empty({m.width}, options(m.weight_type, m.dev));
        }
        dx.expect(m.type, m.dev, m.tokens, m.width, "rms_norm_grad d_xs");
        dw.expect(m.weight_type, m.dev, m.one, -1, "rms_norm_grad d_weights");
        void* stream = stream_on(s, m.dev, what);
        int64_t size = 0;
        call([&] { return rc_rms_norm_grad_workspace(&m.d, &size); });
        Tensor work;
        if (size) work = at::empty({size}, options(ScalarType::Byte, m.dev));
        call([&] { return rc_rms_norm_grad(&m.d, dy.p, m.x.p, m.w.p, with ? ds.p : nullptr, dx.p, dw.p,
                               size ? work.data_ptr() : nullptr, size, stream); });
        return lists({&dx, &dw});
    });
}

// ---------------------------------------------------------------- experts

int moe_type(ScalarType t, const char* what) {
    switch (t) {
        case ScalarType::Float: return RC_F32;
        case ScalarType::Half: return RC_F16;
        case ScalarType::BFloat16: return RC_BF16;
        case kE4M3: return RC_E4M3;
        default: break;
    }
    PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %s; float32, float16, bfloat16 and float8_e4m3fn are supported", what, type_name(t));
    throw Raised{};
}

// R lists of weights, [experts, rows, cols] each.
void expect3(Tensors& t, ScalarType type, const at::Device& dev, int64_t experts, int64_t rows, int64_t cols, const char* what) {
    for (int r = 0; r < t.n; ++r) {
        const Tensor& x = *t.t[r];
        if (x.scalar_type() != type)
            raise(RC_ERR_DTYPE_MISMATCH, what, "rank %d has dtype %s, expected %s", r, type_name(x.scalar_type()), type_name(type));
        if (x.dim() != 3 || x.size(0) != experts || x.size(1) != rows || x.size(2) != cols)
            raise(RC_ERR_SHAPE_MISMATCH, what, "rank %d: expected (%lld, %lld, %lld)", r, (long long)experts, (long long)rows, (long long)cols);
        if (x.device() != dev) raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d on %s, others on %s", r, x.device().str().c_str(), dev.str().c_str());
        if (x.layout() != at::kStrided || !x.is_contiguous()) raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d is not contiguous", r);
        t.p[r] = x.data_ptr();
    }
}

// moe_layer(xs, weights, experts, gate_up, down, scales or None, gate_up_scales or None, down_scales or None, dtype or None, out or None)
PyObject* moe_layer(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"moe_layer", 10});
        const char* what = "moe_layer";
        const Session s;
        const int R = s.ranks;
        Tensors x, w, e, up, down, xs, us, ds, y;
        x.take(a[0], R, what);
        x.dims(2, what, "[tokens, width]");
        const at::Device dev = x.t[0]->device();
        const ScalarType type = x.t[0]->scalar_type();
        int64_t tokens[RC_MAX_RANKS] = {}, one[RC_MAX_RANKS];
        rows_of(x, tokens);
        rc_moe_desc d{};
        d.struct_size = sizeof d;
        d.session = s.id;
        d.dtype = moe_type(type, what);
        d.width = x.t[0]->size(1);
        d.tokens = tokens;
        x.expect(type, dev, tokens, d.width, what);
        e.take(a[2], R, "moe_layer experts");
        e.dims(2, "moe_layer experts", "[tokens, top_k]");
        const int64_t K = e.t[0]->size(1);
        if (K > RC_MAX_TOP_K) raise(RC_ERR_INVALID_ARGUMENT, what, "top_k %lld", (long long)K);
        d.top_k = (int32_t)K;
        e.expect(ScalarType::Int, dev, tokens, K, "moe_layer experts");
        w.take(a[1], R, "moe_layer weights");
        w.expect(ScalarType::Float, dev, tokens, K, "moe_layer weights");
        up.take(a[3], R, "moe_layer gate_up");
        up.dims(3, "moe_layer gate_up", "[experts, 2 * inner, width]");
        const int64_t per = up.t[0]->size(0), rows = up.t[0]->size(1);
        if (per > RC_MAX_EXPERTS || rows % 2) raise(RC_ERR_SHAPE_MISMATCH, what, "gate_up of %lld experts, %lld rows", (long long)per, (long long)rows);
        const ScalarType weight_type = up.t[0]->scalar_type();
        d.weight_dtype = moe_type(weight_type, "moe_layer gate_up");
        d.num_experts = (int32_t)(per * R);
        d.inner = rows / 2;
        expect3(up, weight_type, dev, per, rows, d.width, "moe_layer gate_up");
        down.take(a[4], R, "moe_layer down");
        expect3(down, weight_type, dev, per, d.width, d.inner, "moe_layer down");
        if (a[5] != Py_None) {
            xs.take(a[5], R, "moe_layer scales");
            xs.expect(ScalarType::Float, dev, tokens, 1, "moe_layer scales");
        }
        for (int r = 0; r < R; ++r) one[r] = per;
        if (a[6] != Py_None) {
            us.take(a[6], R, "moe_layer gate_up_scales");
            us.expect(ScalarType::Float, dev, one, rows, "moe_layer gate_up_scales");
        }
        if (a[7] != Py_None) {
            ds.take(a[7], R, "moe_layer down_scales");
            ds.expect(ScalarType::Float, dev, one, d.width, "moe_layer down_scales");
        }
        ScalarType out_type = type == kE4M3 ? ScalarType::BFloat16 : type;
        if (a[8] != Py_None) {
            if (!THPDtype_Check(a[8])) raise(RC_ERR_INVALID_ARGUMENT, what, "dtype is not a torch.dtype");
            out_type = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
        }
        if (a[9] != Py_None) {
            y.take(a[9], R, "moe_layer output");
            if (a[8] == Py_None) out_type = y.t[0]->scalar_type();
        }
        d.out_dtype = moe_type(out_type, "moe_layer output");
        int64_t size = 0;
        call([&] { return rc_moe_layer_workspace(&d, &size); });
        if (a[9] == Py_None) y.make(R, tokens, d.width, out_type, dev, what);
        y.expect(out_type, dev, tokens, d.width, "moe_layer output");
        void* stream = stream_on(s, dev, what);
        Tensor work;
        if (size) work = at::empty({size}, options(ScalarType::Byte, dev));
        auto floats = [](const Tensors& t) { return t.n ? reinterpret_cast<const float* const*>(t.p) : nullptr; };
        call([&] { return rc_moe_layer(&d, x.p, floats(xs), reinterpret_cast<const int32_t* const*>(e.p), floats(w), up.p, floats(us), down.p,
                               floats(ds), y.p, size ? work.data_ptr() : nullptr, size, stream); });
        return y.give();
    });
}

// ---------------------------------------------------------------- gradients and AdamW

// Owned references to one map for each rank.
struct Maps {
    PyObject* map[RC_MAX_RANKS] = {};
    int n = 0;
    Maps() = default;
    Maps(const Maps&) = delete;
    Maps& operator=(const Maps&) = delete;
    ~Maps() {
        for (int r = 0; r < n; ++r) Py_DECREF(map[r]);
    }
    void take(PyObject* seq, int ranks, const char* what) {
        if (!PyList_Check(seq) && !PyTuple_Check(seq)) raise(RC_ERR_INVALID_ARGUMENT, what, "not a list of maps");
        const Py_ssize_t size = PySequence_Fast_GET_SIZE(seq);
        if (size != ranks) raise(RC_ERR_INVALID_ARGUMENT, what, "%lld maps for %d ranks", (long long)size, ranks);
        for (int r = 0; r < ranks; ++r) {
            PyObject* m = PySequence_Fast_GET_ITEM(seq, r);
            if (!PyDict_Check(m)) raise(RC_ERR_INVALID_ARGUMENT, what, "no map for rank %d", r);
            Py_INCREF(m);
            map[n++] = m;
        }
    }
};

// A gradient's fields; its tensor has to be dense and on `dev`.
rc_grad grad_of(const Tensor& t, const at::Device& dev, const char* what, int rank) {
    rc_grad g{};
    g.dtype = row_type(t, what);
    if (t.device() != dev)
        raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d: a gradient on %s, others on %s", rank, t.device().str().c_str(), dev.str().c_str());
    if (t.layout() != at::kStrided || !t.is_contiguous()) raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d: a gradient is not contiguous", rank);
    g.count = t.numel();
    g.grad = g.count ? t.data_ptr() : nullptr;
    return g;
}

// A dense tensor of `count` elements on `dev`.
void* data_of(PyObject* o, ScalarType type, int64_t count, const at::Device& dev, const char* what, const char* name) {
    if (!THPVariable_Check(o)) raise(RC_ERR_INVALID_ARGUMENT, what, "%s is not a tensor", name);
    const Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type)
        raise(RC_ERR_DTYPE_MISMATCH, what, "%s has dtype %s, expected %s", name, type_name(t.scalar_type()), type_name(type));
    if (t.numel() != count) raise(RC_ERR_SHAPE_MISMATCH, what, "%s has %lld elements, expected %lld", name, (long long)t.numel(), (long long)count);
    if (t.device() != dev) raise(RC_ERR_INVALID_ARGUMENT, what, "%s on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
    if (t.layout() != at::kStrided || !t.is_contiguous()) raise(RC_ERR_INVALID_ARGUMENT, what, "%s is not contiguous", name);
    return t.data_ptr();
}

// grad_norm(grads, over_all, out or None)
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"grad_norm", 3});
        const char* what = "grad_norm";
        const Session s;
        Maps maps;
        maps.take(a[0], s.ranks, what);
        std::vector<Tensor> held;  // a map may change while the call is made
        std::vector<rc_grad> all;
        int counts[RC_MAX_RANKS] = {};
        for (int r = 0; r < s.ranks; ++r) {
            PyObject *key, *value;
            Py_ssize_t pos = 0;
            while (PyDict_Next(maps.map[r], &pos, &key, &value)) {
                if (value == Py_None) continue;
                if (!THPVariable_Check(value)) raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d: a gradient is not a tensor", r);
                held.push_back(THPVariable_Unpack(value));
                all.push_back(grad_of(held.back(), held.front().device(), what, r));
                ++counts[r];
            }
        }
        const rc_grad* lists[RC_MAX_RANKS];
        for (int r = 0, at_ = 0; r < s.ranks; at_ += counts[r++]) lists[r] = all.data() + at_;
        PyObject* out = a[2];
        at::Device dev(at::kCPU);
        if (out != Py_None) {
            if (!THPVariable_Check(out)) raise(RC_ERR_INVALID_ARGUMENT, what, "out is not a tensor");
            dev = THPVariable_Unpack(out).device();
        } else if (!held.empty()) {
            dev = held.front().device();
        } else {
            raise(RC_ERR_INVALID_ARGUMENT, what, "no gradients, and no out that says which GPU");
        }
        if (!held.empty() && held.front().device() != dev)
            raise(RC_ERR_INVALID_ARGUMENT, what, "out on %s, gradients on %s", dev.str().c_str(), held.front().device().str().c_str());
        Tensor made;
        if (out == Py_None) made = at::empty({s.ranks}, options(ScalarType::Float, dev));
        float* norms = static_cast<float*>(out == Py_None ? made.data_ptr() : data_of(out, ScalarType::Float, s.ranks, dev, what, "out"));
        void* stream = stream_on(s, dev, what);
        rc_grad_norm_desc d{};
        d.struct_size = sizeof d;
        d.session = s.id;
        d.over_all = to_bool(a[1]);
        int64_t size = 0;
        call([&] { return rc_grad_norm_workspace(&d, counts, lists, &size); });
        Tensor work;
        if (size) work = at::empty({size}, options(ScalarType::Byte, dev));
        call([&] { return rc_grad_norm(&d, counts, lists, norms, size ? work.data_ptr() : nullptr, size, stream); });
        if (out == Py_None) return THPVariable_Wrap(made);
        Py_INCREF(out);
        return out;
    });
}

// What steps go by: the parameters' and states' tensors with the addresses that
// the table names, and the table itself.
struct Table {
    int ranks = 0, bits = 0;
    at::Device dev{at::kCPU};
    std::vector<PyObject*> keys, tensors;  // owned
    std::vector<const void*> addresses;
    std::vector<PyObject*> params;         // those of `tensors` that are parameters
    int num[RC_MAX_RANKS] = {};
    std::vector<uint64_t> host;
    Tensor gpu;

    ~Table() {
        for (PyObject* o : keys) Py_DECREF(o);
        for (PyObject* o : tensors) Py_DECREF(o);
    }
    void* hold(PyObject* map, PyObject* key, ScalarType type, int64_t count, const char* what, const char* name) {
        PyObject* o = PyDict_GetItemWithError(map, key);
        if (!o) {
            if (PyErr_Occurred()) throw Raised{};
            raise(RC_ERR_PARAM_MISMATCH, what, "a parameter has no %s", name);
        }
        void* p = data_of(o, type, count, dev, what, name);
        Py_INCREF(o);
        tensors.push_back(o);
        addresses.push_back(p);
        return p;
    }
    // Whether the tensors still are where the table says.
    void check(const char* what) const {
        for (size_t i = 0; i < tensors.size(); ++i)
            if (THPVariable_Unpack(tensors[i]).data_ptr() != addresses[i])
                raise(RC_ERR_INVALID_ARGUMENT, what, "a tensor of the state has been given other memory since the state was made: make it anew");
    }
    // Keeps the table's memory, should the state go, from being given out again
    // before what the current stream holds by now is done: the table is not the
    // caller's to record.  A stream that is not torch's own, whose number is its
    // handle, may be gone by the time the memory is asked for, and stays out.
    void hold_for_stream() const {
        const auto s = c10::hip::getCurrentHIPStream(dev.index());
        if (s.stream() && s.id() == reinterpret_cast<intptr_t>(s.stream())) return;
        c10::hip::HIPCachingAllocator::recordStream(gpu.storage().data_ptr(), s);
    }
};

constexpr const char* kTableName = "rank_reductions_amd.AdamWTable";

Table* table_of(PyObject* capsule) {
    auto* t = static_cast<Table*>(PyCapsule_GetPointer(capsule, kTableName));
    if (!t) throw Raised{};
    return t;
}

// adamw_table(bits, params, master or None, m, v, m_scale or None, v_scale or None)
PyObject* adamw_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"adamw_table", 7});
        const char* what = "adamw_state";
        const Session s;
        Maps params, maps[5];
        params.take(a[1], s.ranks, what);
        for (int i = 0; i < 5; ++i)
            if (a[2 + i] != Py_None) maps[i].take(a[2 + i], s.ranks, what);
        auto table = std::make_unique<Table>();
        Table& t = *table;
        t.ranks = s.ranks;
        t.bits = to_int32(a[0], what);
        if (t.bits != 8 && t.bits != 32) raise(RC_ERR_INVALID_ARGUMENT, what, "states of %d bits, not 32 or 8", t.bits);
        if (!maps[1].n || !maps[2].n || (t.bits == 8 && (!maps[3].n || !maps[4].n))) raise(RC_ERR_INVALID_ARGUMENT, what, "m, v or their scales are missing");
        const ScalarType type = t.bits == 8 ? kE4M3 : ScalarType::Float;
        std::vector<rc_adamw_param> all;
        bool first = true;
        for (int r = 0; r < s.ranks; ++r) {
            PyObject *key, *value;
            Py_ssize_t pos = 0;
            while (PyDict_Next(params.map[r], &pos, &key, &value)) {
                if (!THPVariable_Check(value)) raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d: a parameter is not a tensor", r);
                const Tensor& p = THPVariable_Unpack(value);
                if (first) t.dev = p.device();
                first = false;
                Py_INCREF(key);
                t.keys.push_back(key);
                rc_adamw_param e{};
                e.count = p.numel();
                e.dtype = row_type(p, what);
                e.param = t.hold(params.map[r], key, p.scalar_type(), e.count, what, "param");
                t.params.push_back(t.tensors.back());
                if (e.dtype != RC_F32) {
                    if (!maps[0].n) raise(RC_ERR_INVALID_ARGUMENT, what, "16-bit parameters without master copies");
                    e.master = static_cast<float*>(t.hold(maps[0].map[r], key, ScalarType::Float, e.count, what, "master"));
                }
                e.m = t.hold(maps[1].map[r], key, type, e.count, what, "m");
                e.v = t.hold(maps[2].map[r], key, type, e.count, what, "v");
                if (t.bits == 8) {
                    const int64_t blocks = (e.count + RC_ADAMW_BLOCK - 1) / RC_ADAMW_BLOCK;
                    e.m_scale = static_cast<float*>(t.hold(maps[3].map[r], key, ScalarType::Float, blocks, what, "m_scale"));
                    e.v_scale = static_cast<float*>(t.hold(maps[4].map[r], key, ScalarType::Float, blocks, what, "v_scale"));
                }
                all.push_back(e);
                ++t.num[r];
            }
        }
        if (first) raise(RC_ERR_INVALID_ARGUMENT, what, "no parameters");
        stream_on(s, t.dev, what);
        const rc_adamw_param* lists[RC_MAX_RANKS];
        for (int r = 0, at_ = 0; r < s.ranks; at_ += t.num[r++]) lists[r] = all.data() + at_;
        rc_adamw_table_desc d{};
        d.struct_size = sizeof d;
        d.session = s.id;
        d.state_bits = t.bits;
        int64_t size = 0;
        call([&] { return rc_adamw_table(&d, t.num, lists, nullptr, &size); });
        t.host.resize((size_t)(size + 7) / 8);
        call([&] { return rc_adamw_table(&d, t.num, lists, t.host.data(), &size); });
        Tensor host = at::empty({size}, options(ScalarType::Byte, at::Device(at::kCPU)));
        std::memcpy(host.data_ptr(), t.host.data(), (size_t)size);
        t.gpu = host.to(t.dev);  // returns when the copy is done
        PyObject* capsule = PyCapsule_New(table.get(), kTableName, [](PyObject* c) {
            delete static_cast<Table*>(PyCapsule_GetPointer(c, kTableName));
        });
        if (!capsule) throw Raised{};
        table.release();
        return capsule;
    });
}

// adamw_step(table, steps, out_table, steps_out, grads, lr, beta1, beta2, eps, weight_decay, norms or None, max_norm,
//            grad_scale, seed)
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, {"adamw_step", 14});
        const char* what = "adamw_step";
        const Session s;
        Table &t = *table_of(a[0]), &o = *table_of(a[2]);
        if (t.ranks != s.ranks) raise(RC_ERR_INVALID_ARGUMENT, what, "a state of %d ranks, the session has %d", t.ranks, s.ranks);
        t.check(what);
        if (&o != &t) {
            o.check(what);
            if (o.dev != t.dev || o.keys.size() != t.keys.size()) raise(RC_ERR_PARAM_MISMATCH, what, "out holds other parameters");
            for (size_t i = 0; i < t.keys.size(); ++i) {
                const int same = PyObject_RichCompareBool(t.keys[i], o.keys[i], Py_EQ);
                if (same < 0) throw Raised{};
                if (!same) raise(RC_ERR_PARAM_MISMATCH, what, "out holds other parameters, or in another order");
            }
        }
        Maps grads;
        grads.take(a[4], s.ranks, what);
        std::vector<Tensor> held;
        held.reserve(t.keys.size());
        std::vector<rc_grad> all(t.keys.size());
        const rc_grad* lists[RC_MAX_RANKS];
        size_t i = 0;
        for (int r = 0; r < s.ranks; ++r) {
            lists[r] = all.data() + i;
            Py_ssize_t found = 0;
            for (int k = 0; k < t.num[r]; ++k, ++i) {
                PyObject* g = PyDict_GetItemWithError(grads.map[r], t.keys[i]);
                if (!g && PyErr_Occurred()) throw Raised{};
                if (!g) continue;
                ++found;
                if (g == Py_None) continue;
                if (!THPVariable_Check(g)) raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d: a gradient is not a tensor", r);
                held.push_back(THPVariable_Unpack(g));
                if (held.back().sizes() != THPVariable_Unpack(t.params[i]).sizes())
                    raise(RC_ERR_SHAPE_MISMATCH, what, "rank %d: a gradient of %lld elements has another shape than its parameter", r,
                          (long long)held.back().numel());
                all[i] = grad_of(held.back(), t.dev, what, r);
            }
            if (found != PyDict_GET_SIZE(grads.map[r])) raise(RC_ERR_PARAM_MISMATCH, what, "rank %d: gradients of parameters that the state does not hold", r);
        }
        rc_adamw_desc d{};
        d.struct_size = sizeof d;
        d.session = s.id;
        if (THPVariable_Check(a[5])) {
            d.lr_on_gpu = static_cast<const float*>(data_of(a[5], ScalarType::Float, 1, t.dev, what, "lr"));
        } else {
            d.lr = to_double(a[5]);
        }
        d.beta1 = to_double(a[6]);
        d.beta2 = to_double(a[7]);
        d.eps = to_double(a[8]);
        d.weight_decay = to_double(a[9]);
        if (a[10] != Py_None) d.norms = static_cast<const float*>(data_of(a[10], ScalarType::Float, s.ranks, t.dev, what, "norms"));
        d.max_norm = to_double(a[11]);
        d.grad_scale = to_double(a[12]);
        const long long seed = to_int(a[13]);
        if (seed < 0 || seed > UINT32_MAX) raise(RC_ERR_INVALID_ARGUMENT, what, "seed %lld is no number of 32 bits", seed);
        d.seed = (uint32_t)seed;
        d.steps = static_cast<const int32_t*>(data_of(a[1], ScalarType::Int, s.ranks, t.dev, what, "step"));
        d.steps_out = static_cast<int32_t*>(data_of(a[3], ScalarType::Int, s.ranks, t.dev, what, "step of out"));
        void* stream = stream_on(s, t.dev, what);
        t.hold_for_stream();
        if (&o != &t) o.hold_for_stream();
        call([&] { return rc_adamw_step(&d, t.host.data(), t.gpu.data_ptr(), o.host.data(), o.gpu.data_ptr(), lists, stream); });
        Py_RETURN_NONE;
    });
}

}  // namespace

#define RC_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef rows_binding::block_methods[] = {
    RC_METHOD(rms_norm), RC_METHOD(rms_norm_grad), RC_METHOD(moe_layer), RC_METHOD(grad_norm), RC_METHOD(adamw_table), RC_METHOD(adamw_step),
    {nullptr, nullptr, 0, nullptr},
};
