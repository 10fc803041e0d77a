// Python module _rows: argument marshalling of the block operators (blocks.py
// holds the public functions).
#include "binding_blocks.h"

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

}  // namespace

#define RC_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef rows_binding::block_methods[] = {
    RC_METHOD(rms_norm), RC_METHOD(rms_norm_grad),
    {nullptr, nullptr, 0, nullptr},
};
